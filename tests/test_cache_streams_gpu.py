"""The cache operators on streams and in captured graphs, against the plain 64-bit
implementations of tests/cache_ref.py.  Tolerances: tests/test_cache_ops_gpu.py."""
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_cache_ops_gpu import Batch, _built, check_out, check_weights  # noqa: F401

pytestmark = pytest.mark.gpu


def check_call(bt, out, w):
    """Output and fresh key weights of one call against the reference."""
    got, gw, g = out.double().cpu().numpy(), w.double().cpu().numpy(), bt.hq // bt.hk
    for s in range(bt.n):
        o, a, weights, mag = bt.reference(s)
        check_out(bt, got, s, o, a, mag)
        fresh = weights.reshape(bt.hk, g, bt.sq[s], bt.sk[s]).sum((1, 2))
        check_weights(gw[s, :, :bt.sk[s]], fresh, fresh, mag, bt.d, g * bt.sq[s])


def test_first_call_on_a_side_stream_while_the_default_stream_is_busy():
    """A problem created and used while earlier work of the default stream still runs."""
    bt = Batch(300, "fp4", 8, 2, 128, 16, (1,) * 6, (900, 20, 300, 1, 64, 2000)).device()
    side = torch.cuda.Stream()
    w = torch.zeros(bt.n, bt.hk, max(bt.sk), device="cuda")
    out = torch.zeros_like(bt.d_q)
    big = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda")
    other = torch.ones_like(big)
    torch.cuda.synchronize()
    for _ in range(100):                               # about 30 ms of copies
        big.copy_(other)
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, None, w, out=out, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    assert p.check_device_error() == 0
    check_call(bt, out, w)


def test_host_tensors_are_refused_before_any_launch():
    bt = Batch(301, "fp4", 8, 2, 128, 16, (1, 1), (30, 17)).device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    kn, vn = bt.new_rows("k"), bt.new_rows("v")
    w = torch.zeros(2, 2, 30, device="cuda")
    kept = torch.zeros(2, 2, 10, dtype=torch.int32, device="cuda")
    pages = torch.zeros(bt.blocks, 16, 2, 128, dtype=torch.bfloat16, device="cuda")

    def store(kn=kn, vn=vn):
        p.cache_store(kn, vn, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 2, 2, 1, 30)

    def expand(k=pages, v=pages, table=bt.d_table, begin=bt.d_cu):
        p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 2, 30, k, v, table, begin=begin)

    def weigh(w_in=None, w_out=w):
        p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, w_in, w_out)

    def evict(w_in=w, w_out=w, kept=kept, used=bt.d_sk, dst=bt.d_table):
        p.cache_evict(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 2, 30, w_in, w_out, 10, 2, kept, used, dst_block_table=dst)

    for call, names in ((store, dict(kn=kn, vn=vn)), (weigh, dict(w_in=w, w_out=w)),
                        (expand, dict(k=pages, v=pages, table=bt.d_table, begin=bt.d_cu)),
                        (evict, dict(w_in=w, w_out=w, kept=kept, used=bt.d_sk, dst=bt.d_table))):
        for name, t in names.items():
            with pytest.raises(ValueError):
                call(**{name: t.cpu()})
    assert p.last_launch_count() == 0
