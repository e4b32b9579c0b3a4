"""Attention for draft trees over 4-bit and fp8 caches on the GPU, against the 64-bit reference
of tests/step_ref.py on the values that the cache's bytes stand for.  Tolerances:
tests/test_step_ops_gpu.py."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests import step_ref as S
from tests.test_step_ops_gpu import Trees, _built, bits, i32, terms  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = [
    # (hq, hk, d, b, S_q, S_k, terms)
    (8, 2, 128, 16, (1, 5, 9), (1, 40, 700), {}),
    (8, 2, 64, 32, (8, 1, 0, 33), (8, 129, 5, 300), dict(softcap=20.0, window=40, sinks=True)),
    (32, 8, 128, 16, (17, 32), (1200, 33), {}),
    (16, 1, 128, 64, (64, 7), (900, 64), dict(sinks=True)),
    (16, 2, 256, 64, (64, 1, 20), (1500, 65, 20), {}),
    (5, 5, 256, 16, (130, 40), (400, 41), dict(window=9, alibi=True, sinks=True)),
    (6, 2, 128, 16, (50, 3), (177, 128), dict(window=2)),
    (12, 4, 64, 16, (100, 33), (100, 1000), dict(alibi=True)),
    (40, 1, 64, 16, (9, 4), (130, 260), dict(window=1)),
    (128, 1, 128, 32, (3, 2), (50, 515), dict(softcap=5.0)),
    (2, 2, 128, 64, (200, 128), (2000, 128), dict(window=300, softcap=30.0)),
    (8, 8, 128, 16, (1,), (5000,), {}),
    (8, 1, 64, 64, (20,), (12000,), {}),
]


KINDS = [("fp4", c) for c in range(len(CASES))] + [("fp8", c) for c in range(len(CASES)) if CASES[c][2] == 128]
PATH = dict(fp4="fp4_rows", fp8="fp8_tree")


@pytest.mark.parametrize("kind,case", KINDS)
@pytest.mark.parametrize("partials", [ua.UA_PARTIALS_F32, ua.UA_PARTIALS_BF16])
def test_tree_attention(kind, case, partials):
    hq, hk, d, b, sq, sk, kw = CASES[case]
    bt = Trees(1700 + case, hq, hk, d, b, sq, sk, kind=kind, kscale=0.7, vscale=1.3).device()
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    p = bt.problem(flags, softcap=softcap, window=window, split_partials=partials)
    out = torch.full_like(bt.d_q, 3.0)
    got = bt.run(p, flags, sinks, alibi, out=out, pos=bool(window or kw.get("alibi")))
    assert p.check_device_error() == 0 and p.last_path().startswith(PATH[kind])
    bt.check(got, softcap, partials == ua.UA_PARTIALS_BF16, window=window, sinks=sinks, alibi=alibi)
    assert torch.equal(bt.run(p, flags, sinks, alibi, pos=bool(window or kw.get("alibi"))), got)


@pytest.mark.parametrize("kind,hq,hk,d", [("fp4", 8, 2, 128), ("fp4", 4, 4, 64), ("fp4", 8, 1, 256), ("fp8", 8, 2, 128)])
def test_masks_that_are_no_trees(kind, hq, hk, d):
    bt = Trees(1740, hq, hk, d, 16, (40, 33, 5), (40, 90, 5), words=3, kind=kind)
    bt.mask = bt.rng.integers(0, 1 << 32, bt.mask.shape, dtype=np.uint64).astype(np.uint32)
    bt.mask[3] = bt.mask[17] = bt.mask[45] = bt.mask[75] = 0
    bt.device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_SINKS
    p = bt.problem(flags)
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == 0
    bt.check(got)
    assert bool((got[[3, 17, 75]] == 0).all())
    sinks = np.full(hq, 0.5, np.float32)
    sinks[0], sinks[1] = np.inf, -np.inf
    bt.check(bt.run(p, flags, sinks, pos=False), sinks=sinks.astype(np.float64))


@pytest.mark.parametrize("kind,d,window", [("fp4", 64, 0), ("fp4", 128, 0), ("fp4", 256, 0), ("fp4", 128, 25), ("fp4", 64, 7),
                                           ("fp8", 128, 0), ("fp8", 128, 25), ("fp8", 128, 7)])
def test_nan_values_reach_the_rows_that_see_them(kind, d, window):
    """NaN (of a 4-bit cache in groups of 16 dims) in V of nodes and in front of the window,
    and a NaN key: the rows that see them and no others."""
    group = 16 if kind == "fp4" else 1
    bt = Trees(1742, 8, 2, d, 16, (40, 20), (150, 333), store=False, kind=kind)
    bt.trees = [[-1, 0, 0, 1, 1, 2] + [2] * 34, [-1, 0] + [0] * 18]
    bt.mask = np.concatenate([S.mask_of(t, bt.words) for t in bt.trees])
    bt.pos = [np.array(S.depths(t)) + k - len(t) for t, k in zip(bt.trees, bt.sk)]
    for node, dim in ((4, 3), (9, 20), (39, d - 1)):
        bt.v[0][110 + node, 1, dim] = np.nan
    bt.k[0][110 + 12, 0, 1] = np.nan
    if window:
        bt.v[1][:313 - window + 1] = np.nan             # in front of every window
        bt.v[1][313 - window + 1, :, 5] = np.nan        # seen by the root alone
        bt.k[1][:313 - window + 1] = np.nan
    for s in range(2):
        (bt.kb[s], bt.k[s]), (bt.vb[s], bt.v[s]) = bits(bt.k[s]), bits(bt.v[s])
        for j in range(bt.sk[s]):
            bt.put(s, j)
    bt.device()
    flags = ua.UA_FLAG_CAUSAL | (ua.UA_FLAG_WINDOW if window else 0)
    p = bt.problem(flags, window=window)
    got = bt.run(p, flags).double().cpu().numpy()
    assert p.check_device_error() == 0
    want = np.zeros(got.shape, bool)
    for node, dim in ((4, 3), (9, 20), (39, d - 1)):
        want[node, 4:, dim // group * group:dim // group * group + group] = True
    want[12, :4] = True
    if window:
        want[40, :, 5 // group * group:5 // group * group + group] = True
    np.testing.assert_array_equal(np.isnan(got), want)
    assert np.isfinite(got[~want]).all()


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_malformed_sequences_blocks_and_positions(kind):
    bt = Trees(1743, 8, 2, 128, 16, (9, 12, 6, 4), (60, 40, 100, 30), kind=kind).device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_WINDOW
    p = bt.problem(flags, window=1000)
    good = bt.run(p, flags)
    bt.d_sk = i32([60, 5, 100, 30])
    got = bt.run(p, flags)
    assert p.check_device_error() & ua.UA_DEVERR_CONTEXT
    assert bool((got[9:21] == 0).all()) and torch.equal(got[:9], good[:9]) and torch.equal(got[21:], good[21:])
    bt.d_sk = i32(bt.sk)
    bt.d_table[2, 1] = bt.blocks + 5
    got = bt.run(p, flags)
    assert p.check_device_error() == ua.UA_DEVERR_BLOCK_ID
    assert torch.equal(got[:21], good[:21]) and torch.equal(got[27:], good[27:]) and bool(got.isfinite().all())
    bt.d_table.copy_(torch.from_numpy(bt.table))
    bt.pos[0][2] = 2000
    bt.run(p, flags)
    assert p.check_device_error() == ua.UA_DEVERR_TREE


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_stall_hook_gives_up(kind):
    from paged_varlen_flash_gb300 import binding
    bt = Trees(1746, 8, 2, 128, 16, (9, 4), (600, 300), kind=kind).device()
    p = bt.problem()
    good = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert binding.ua_debug_stall_data_waits(p.handle, 1, 2_000_000) == 0
    bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() & ua.UA_DEVERR_TIMEOUT
    assert binding.ua_debug_stall_data_waits(p.handle, 0) == 0
    assert torch.equal(bt.run(p, ua.UA_FLAG_CAUSAL, pos=False), good)
    assert p.check_device_error() == 0


def test_key_weights_and_tree_calls_of_one_problem():
    bt = Trees(1744, 8, 2, 128, 16, (6, 9), (300, 90), kind="fp4").device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    bt.check(bt.run(p, ua.UA_FLAG_CAUSAL, pos=False))
    assert p.check_device_error() == 0


@pytest.mark.parametrize("kind", ["fp4", "fp8"])
def test_captured_and_replayed(kind):
    bt = Trees(1745, 16, 4, 128, 32, (20, 7, 33), (500, 2000, 33), kind=kind).device()
    p = bt.problem()
    mask = torch.from_numpy(bt.mask.view(np.int32)).cuda()
    out = torch.zeros_like(bt.d_q)
    call = lambda: p.forward_tree(bt.d_q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, bt.n, 60, 33, 2000,  # noqa: E731
                                  ua.UA_FLAG_CAUSAL, mask, out=out)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    graph.replay()
    bt.check(out)
    bt.mask[:] = bt.rng.integers(0, 1 << 32, bt.mask.shape, dtype=np.uint64).astype(np.uint32)
    mask.copy_(torch.from_numpy(bt.mask.view(np.int32)))
    graph.replay()
    bt.check(out)
    assert p.check_device_error() == 0


@pytest.mark.parametrize("seed", range(24))
def test_random_trees(seed):
    kind = "fp8" if seed >= 16 else "fp4"
    g = np.random.default_rng(16000 + seed)
    hk, gq = int(g.choice([1, 2, 3, 8])), int(g.choice([1, 2, 3, 4, 8, 16]))
    d, b = int(g.choice([64, 128, 256])) if kind == "fp4" else 128, int(g.choice([16, 32, 64]))
    n = int(g.integers(1, 7))
    sq = [int(x) for x in np.minimum(np.exp(g.uniform(0, 5, n)), 70 if gq < 8 else 40)]
    sk = [a + int(np.exp(g.uniform(0, 7))) - 1 for a in sq]
    softcap, window = float(g.choice([0.0, 0.0, 8.0])), int(g.choice([0, 0, 1, 5, 60, 500]))
    sinks = g.normal(size=gq * hk).astype(np.float32) if g.random() < 0.4 else None
    alibi = (2.0 ** -g.uniform(0, 8, gq * hk)).astype(np.float32) if g.random() < 0.3 else None
    bt = Trees(17000 + seed, gq * hk, hk, d, b, sq, sk, kind=kind, kscale=float(g.uniform(0.3, 3)), vscale=float(g.uniform(0.3, 3)))
    if g.random() < 0.3:
        bt.mask = bt.rng.integers(0, 1 << 32, bt.mask.shape, dtype=np.uint64).astype(np.uint32)
    bt.device()
    flags = ua.flags_of(True, softcap, alibi is not None, window, sinks is not None)
    p = bt.problem(flags, softcap=softcap, window=window)
    got = bt.run(p, flags, sinks, alibi)
    assert p.check_device_error() == 0
    bt.check(got, softcap, window=window, sinks=sinks, alibi=alibi)
