"""Results that a call on another stream than the current one allocates itself: memory that
kernels of the current stream still use is not handed to it."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_step_ops_gpu import Rope, Trees, _built  # noqa: F401

pytestmark = pytest.mark.gpu


def calls():
    bt = Trees(2100, 8, 2, 128, 16, (9, 20), (300, 90)).device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    w = torch.zeros(2, 2, 300, device="cuda")
    lists = torch.arange(32, dtype=torch.int32, device="cuda").repeat(29, 1)
    lens = torch.full((29,), 32, dtype=torch.int32, device="cuda")
    r = Rope(0).device()
    rp = r.problem()
    caches = [c[1] for c in r.caches()]
    tree = (bt.d_q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 2, 29, 20, 300)
    return dict(
        forward=(bt.d_q, lambda st: p.forward(*tree, ua.UA_FLAG_CAUSAL, stream=st)),
        topk=(bt.d_q, lambda st: p.forward_topk(*tree, lists, lens, ua.UA_FLAG_CAUSAL, stream=st)),
        weights=(bt.d_q, lambda st: p.forward_weights(*tree, ua.UA_FLAG_CAUSAL, None, w, stream=st)),
        tree=(bt.d_q, lambda st: p.forward_tree(*tree, ua.UA_FLAG_CAUSAL, mask, stream=st)),
        rope=(r.d_q, lambda st: rp.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, *caches, stream=st)),
    )


@pytest.mark.parametrize("name", ["forward", "topk", "weights", "tree", "rope"])
@pytest.mark.parametrize("raw", [False, True])
def test_results_of_another_stream(name, raw):
    q, call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call(side)                                            # (kernels loaded)
    torch.cuda.synchronize()
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    other = torch.ones_like(big)
    held = [torch.empty_like(want) for _ in range(8)]
    kept = [torch.empty_like(want) for _ in range(8)]
    torch.cuda.synchronize()
    for x in held:
        x.fill_(3.0)
    for _ in range(60):                                   # about 20 ms of copies
        big.copy_(other)
    for x, y in zip(held, kept):
        y.copy_(x)
    del x, held                                           # the current stream has still to read them
    got = [call(side.cuda_stream if raw else side) for _ in range(8)]
    torch.cuda.synchronize()
    for x, y in zip(got, kept):
        assert bool((y == 3).all()) and torch.equal(x, want) and x.shape == q.shape


def test_results_on_the_default_stream_from_a_side_stream():
    q, call = calls()["tree"]
    want = call(None)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = call(0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_a_result_read_by_the_current_stream_outlives_its_name():
    """Dropped while the current stream has still to read it, it is not handed out again."""
    _, call = calls()["tree"]
    want = call(None)
    side = torch.cuda.Stream()
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    other = torch.ones_like(big)
    torch.cuda.synchronize()
    got = call(side)
    side.synchronize()
    for _ in range(60):
        big.copy_(other)
    late = got.clone()
    del got
    for _ in range(8):
        with torch.cuda.stream(side):
            torch.empty_like(want).fill_(7.0)
    torch.cuda.synchronize()
    assert torch.equal(late, want)


def test_results_inside_a_captured_graph():
    """A captured fork to another stream: the result lies in the graph's memory."""
    _, call = calls()["tree"]
    want = call(None)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    got.fill_(5.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
