"""Tree calls at the edges of what their documentation allows: batches without rows, positions
out of range, q written by the kernel in front.  Tolerances: tests/test_step_ops_gpu.py."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_step_ops_gpu import Trees, _built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- no rows allowed
@pytest.mark.parametrize("kind,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp8", 128), ("fp4", 64), ("fp4", 128),
                                    ("fp4", 256)])
def test_trees_of_a_batch_without_rows(kind, d):
    """max_seqlen_q = 0 with padding tokens: empty sequences are served, others reported."""
    bt = Trees(2000, 8, 2, d, 16, (2, 3), (40, 20), kind=kind).device()
    p = bt.problem()
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    out = torch.full_like(bt.d_q, 7.0)

    def call(cu, sk, most):
        p.forward_tree(bt.d_q, bt.d_k, bt.d_v, bt.d_table, cu, sk, 2, 5, 0, most, ua.UA_FLAG_CAUSAL, mask, out=out)

    for sk, most in ((bt.d_sk, 40), (i32([0, 0]), 40), (i32([0, 0]), 0)):
        call(i32([0, 0, 0]), sk, most)
        assert p.check_device_error() == 0 and bool((out == 7).all())
    call(bt.d_cu, bt.d_sk, 40)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS and bool((out == 0).all())


# ---------------------------------------------------------------- positions out of range
@pytest.mark.parametrize("kind,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp8", 128), ("fp4", 64), ("fp4", 128),
                                    ("fp4", 256)])
@pytest.mark.parametrize("at,moved", [(2000, 39), (-1, 35), (34, 35), (40, 39)])
def test_alibi_positions_outside_the_chunk_are_reported(kind, d, at, moved):
    """With ALiBi alone, as with a window: moved into the chunk and reported.  Good ones are not."""
    bt = Trees(2001, 4, 2, d, 16, (5, 3), (40, 20), kind=kind).device()
    alibi = np.array([0.5, 0.25, 0.125, 1.0], np.float32)
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_ALIBI
    p = bt.problem(flags)
    bt.check(bt.run(p, flags, alibi=alibi), alibi=alibi)
    assert p.check_device_error() == 0
    bt.pos[0][2] = at
    got = bt.run(p, flags, alibi=alibi)
    assert p.check_device_error() == ua.UA_DEVERR_TREE
    bt.pos[0][2] = moved
    bt.check(got, alibi=alibi)
    # Without a window or ALiBi positions are not read.
    bt.pos[0][2] = at
    bt.check(bt.run(p, ua.UA_FLAG_CAUSAL))
    assert p.check_device_error() == 0


# ---------------------------------------------------------------- early starts
@pytest.mark.parametrize("d,words", [(64, 16), (128, 16), (256, 16), (256, 8)])
def test_q_that_the_kernel_in_front_writes(d, words):
    """The same q buffer, written anew in front of every call (words: its alignment in 16-bit
    words, whole or half sectors): each call reads what was written last."""
    bt = Trees(2700 + d, 16, 2, d, 16, (64, 20), (200, 90)).device()
    p = bt.problem()
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    room = torch.zeros(bt.d_q.numel() + 64, dtype=torch.bfloat16, device="cuda")
    q = room[words:words + bt.d_q.numel()].view(bt.d_q.shape)
    assert q.data_ptr() % 32 == 2 * words % 32
    rows = [torch.randn(bt.d_q.shape, device="cuda").to(torch.bfloat16) for _ in range(16)]
    outs = [torch.empty_like(bt.d_q) for _ in rows]

    def call(out):
        p.forward_tree(q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 2, 84, 64, 200, ua.UA_FLAG_CAUSAL, mask, out=out)

    for x, out in zip(rows, outs):
        q.copy_(x)
        call(out)
    torch.cuda.synchronize()
    want = torch.empty_like(bt.d_q)
    for x, out in zip(rows, outs):
        q.copy_(x)
        torch.cuda.synchronize()
        call(want)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert p.check_device_error() == 0
