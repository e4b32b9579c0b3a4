"""Calls of the cache operators that the documentation allows beside the usual ones:
padded batches, bias matrices and bf16 partials with key weights, scales at the ends of
fp32, graphs that share a problem.  Against the plain 64-bit implementations of
tests/cache_ref.py; tolerances: tests/test_cache_ops_gpu.py."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests.test_cache_ops_gpu import (  # noqa: F401
    Batch, _built, bits, check_out, check_weights, on_gpu, raw_of, terms, weights_reference)

pytestmark = pytest.mark.gpu


def compare(bt, out, w, softcap=0.0, extra=0.0, bf16_p=False, **kw):
    """Outputs (and key weights that started from zero) of every sequence."""
    got = out.double().cpu().numpy()
    if w is not None:
        want, fresh, mag = weights_reference(bt, None, 0.0, softcap=softcap, **kw)
    for s in range(bt.n):
        if not bt.sq[s]:
            continue
        o, a, _, m = bt.reference(s, softcap=softcap, **kw)
        check_out(bt, got, s, o, a, m, softcap, extra, bf16_p)
        if w is not None:
            sk = bt.sk[s]
            check_weights(w[s, :, :sk].double().cpu().numpy(), want[s, :, :sk], fresh[s, :, :sk], mag, bt.d,
                          bt.hq // bt.hk * bt.sq[s], softcap, extra)


# (kind, hq, hk, d, b, S_q, S_k): each kernel family, one segment and several
SHAPES = [
    ("fp4", 8, 2, 128, 16, (1, 0, 3), (700, 20, 33)),
    ("fp4", 4, 2, 64, 32, (2, 1, 1), (40, 3000, 1)),
    ("fp4", 8, 2, 128, 32, (30, 0, 9), (2000, 5, 9)),
    ("fp4", 16, 2, 256, 64, (9, 12, 1), (130, 900, 70)),
    ("bf16", 8, 2, 128, 16, (1, 0, 2), (1500, 20, 33)),
    ("bf16", 4, 2, 64, 32, (20, 1, 0), (300, 70, 9)),
    ("fp8", 8, 2, 128, 16, (1, 0, 9), (1500, 20, 33)),
]


@pytest.mark.parametrize("case", range(len(SHAPES)))
@pytest.mark.parametrize("partials", [ua.UA_PARTIALS_F32, ua.UA_PARTIALS_BF16])
def test_rows_behind_the_last_sequence_stay_as_they_are(case, partials):
    """A padded batch: total_q, tables and lengths for more than the sequences in use."""
    kind, hq, hk, d, b, sq, sk = SHAPES[case]
    bt = Batch(320 + case, kind, hq, hk, d, b, sq, sk, 0.5, 0.25).device()
    pad = 70
    q = torch.cat([bt.d_q, torch.full((pad, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")])
    flags = ua.UA_FLAG_CAUSAL
    p = bt.problem(flags | ua.UA_FLAG_KEY_WEIGHTS, max_total_q=len(q) + 5, split_partials=partials)
    a = bt.args()
    w = torch.full((bt.n + 2, hk, max(sk) + 1), 9.0, device="cuda")
    out = torch.full_like(q, 3.0)
    bf16_p = kind == "bf16" or partials == ua.UA_PARTIALS_BF16
    for _ in range(2):
        p.forward_weights(q, *a[1:7], len(q), *a[8:], flags, None, w, decay=0.0, out=out)
        assert p.check_device_error() == 0
        compare(bt, out, w, bf16_p=bf16_p)
        assert bool((out[sum(sq):] == 3.0).all()) and bool((w[bt.n:] == 9.0).all())
        for s in range(bt.n):
            assert bool((w[s, :, sk[s] if sq[s] else 0:] == 9.0).all())
    if kind == "fp4":
        out.fill_(3.0)
        p.forward(q, *a[1:7], len(q), *a[8:], flags, out=out)
        compare(bt, out, None, bf16_p=bf16_p)
        assert p.check_device_error() == 0 and bool((out[sum(sq):] == 3.0).all())


@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_qq_bias_with_key_weights(case):
    kind, hq, hk, d, b, sq, sk = SHAPES[case]
    bt = Batch(340 + case, kind, hq, hk, d, b, sq, sk, 0.5, 0.25).device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_QQ_BIAS | ua.UA_FLAG_SINKS
    qq = bt.rng.normal(size=(max(sq), max(sq) + 3)).astype(np.float32)
    sinks = bt.rng.normal(size=hq).astype(np.float32)
    p = bt.problem(flags | ua.UA_FLAG_KEY_WEIGHTS)
    p.set_qq_bias(torch.from_numpy(qq).cuda())
    w = torch.zeros(bt.n, hk, max(sk), device="cuda")
    out = p.forward_weights(*bt.args(), flags, None, w, sinks=on_gpu(sinks))
    assert p.check_device_error() == 0
    compare(bt, out, w, extra=5.0, bf16_p=kind == "bf16", qq=qq.astype(np.float64), sinks=sinks.astype(np.float64))


@pytest.mark.parametrize("nq,sk", [(1, (40, 300)), (20, (40, 300)), (70, (70, 400))])
@pytest.mark.parametrize("window", [0, 9])
def test_scores_whose_factor_underflows(nq, sk, window):
    """scale * k_scale times a row's power of two below fp32: the scores are zero, not NaN,
    and the masks still hold."""
    bt = Batch(360, "fp4", 8, 2, 128, 16, (nq, nq), sk)
    bt.kscale = float(np.float32(2.0 ** -40))
    bt.kc.scale = bt.kscale
    bt.q = bt.q * 2.0 ** -126
    bt.qb, bt.q = bits(bt.q)
    flags = ua.UA_FLAG_CAUSAL | (ua.UA_FLAG_WINDOW if window else 0)
    p = bt.device().problem(flags | ua.UA_FLAG_KEY_WEIGHTS, window=window)
    compare(bt, p.forward(*bt.args(), flags), None, window=window)
    w = torch.zeros(2, 2, max(sk), device="cuda")
    out = p.forward_weights(*bt.args(), flags, None, w)
    assert p.check_device_error() == 0
    compare(bt, out, w, window=window)


def test_graphs_of_one_problem_replayed_in_turn():
    """A decode step, a window call and a plain call of one 4-bit problem, captured apart
    and replayed one after another, give the bits of the eager calls."""
    bt = Batch(370, "fp4", 8, 2, 128, 16, (1, 1, 1, 1), (900, 31, 64, 2000)).device()
    wide = Batch(371, "fp4", 8, 2, 128, 16, (20, 9, 33, 1), (900, 31, 64, 2000))
    wide.table, wide.kc, wide.vc, wide.blocks, wide.width = bt.table, bt.kc, bt.vc, bt.blocks, bt.width
    wide.device()
    p = ua.Problem(8, 2, 128, 16, bt.blocks, 4, bt.width, 63, ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS, bt.scale,
                   kv_dtype=ua.UA_DTYPE_FP4_E2M1)
    calls, results = [], []
    for x, weigh in ((bt, True), (wide, True), (bt, False), (wide, False)):
        w, out = torch.zeros(4, 2, 2000, device="cuda"), torch.zeros_like(x.d_q)

        def call(x=x, weigh=weigh, w=w, out=out, stream=None):
            if weigh:
                p.forward_weights(*x.args(), ua.UA_FLAG_CAUSAL, None, w, out=out, stream=stream)
            else:
                p.forward(*x.args(), ua.UA_FLAG_CAUSAL, out=out, stream=stream)
        calls.append(call)
        results.append((w, out))
    for c in calls:
        c()
    assert p.check_device_error() == 0
    want = [(w.clone(), o.clone()) for w, o in results]
    for x, (w, o) in zip((bt, wide), want):
        compare(x, o, w)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graphs = []
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=stream):
            c(stream=None)
        graphs.append(g)
    for w, o in results:
        w.zero_()
        o.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        for i in (0, 1, 2, 3, 1, 0, 3, 2, 0, 0, 1, 1):
            graphs[i].replay()
    torch.cuda.synchronize()
    assert p.check_device_error() == 0
    for (w, o), (ww, wo) in zip(results, want):
        assert torch.equal(w, ww) and torch.equal(o.view(torch.int16), wo.view(torch.int16))


@pytest.mark.parametrize("kind,nq", [("fp4", 1), ("fp4", 40), ("bf16", 1), ("bf16", 9), ("fp8", 2)])
def test_the_same_calls_on_blocks_past_4_gib(kind, nq):
    """Store, weighed attention, eviction (into other blocks, then in place) and expansion on
    blocks beyond 2^32 bytes of the cache: the bits of the same calls on a small cache."""
    sk = (130, 70, 200)
    bt = Batch(380, kind, 8, 2, 128, 16, (nq,) * 3, sk, 0.5, 0.25, spare=40).device()
    shift = (1 << 32) // (bt.d_k[0].numel() * bt.d_k.element_size()) + 3
    pages = torch.zeros(bt.blocks, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    kn, vn = bt.new_rows("k"), bt.new_rows("v")
    dst = torch.full_like(bt.d_table, -1)
    dst[:, :6] = torch.from_numpy(bt.spare_ids[:18].astype(np.int32)).cuda().view(3, 6)
    results = []
    for off in (0, shift):
        k, v = (torch.zeros(off + bt.blocks, *c.shape[1:], dtype=c.dtype, device="cuda") for c in (bt.d_k, bt.d_v))
        k[off:], v[off:] = bt.d_k, bt.d_v
        move = lambda t: torch.where(t >= 0, t + off, -1).to(torch.int32)     # noqa: E731
        table, to = move(bt.d_table), move(dst)
        p = ua.Problem(8, 2, 128, 16, off + bt.blocks, 3, bt.width, 3 * nq,
                       ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS, bt.scale, kv_dtype=ua_dtype(kind),
                       k_scale=bt.kscale, v_scale=bt.vscale)
        w, kept = torch.zeros(3, 2, 200, device="cuda"), torch.zeros(3, 2, 90, dtype=torch.int32, device="cuda")
        kept2 = torch.zeros(3, 2, 33, dtype=torch.int32, device="cuda")
        used, out = bt.d_sk.clone(), torch.zeros_like(bt.d_q)
        ko, vo = pages.clone(), pages.clone()
        p.cache_store(kn, vn, k, v, table, bt.d_cu, used, 3, 3 * nq, nq, 200)
        p.forward_weights(bt.d_q, k, v, table, bt.d_cu, used, 3, 3 * nq, nq, 200, ua.UA_FLAG_CAUSAL, None, w, out=out)
        p.cache_evict(k, v, table, used, 3, 200, w, w, 90, 7, kept, used, dst_block_table=to)
        p.cache_evict(k, v, to, used, 3, 90, w, w, 33, 5, kept2, used)
        p.cache_expand(k, v, to, used, 3, 33, ko, vo, dst)
        assert p.check_device_error() == 0
        assert not bool(k[:off].view(torch.uint8).any()) and not bool(v[:off].view(torch.uint8).any())
        results.append([t.clone().view(torch.uint8) for t in (k[off:], v[off:], out, w, kept, kept2, used, ko, vo)])
        if off == 0:
            compare(bt, out, None, bf16_p=kind == "bf16")
        del k, v
    for a, b in zip(*results):
        assert torch.equal(a, b)


def ua_dtype(kind):
    return {"bf16": ua.UA_DTYPE_BF16, "fp8": ua.UA_DTYPE_FP8_E4M3, "fp4": ua.UA_DTYPE_FP4_E2M1}[kind]
