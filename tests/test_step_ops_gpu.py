"""A speculative decoding step on the GPU (blocks and slots, rotary store, attention for
draft trees, accepted branches) against the plain implementations of tests/step_ref.py.

Tolerances.  Attention: with dx the score error bound of ``score_error`` (natural units),
a softmax weight w is off by at most w (2 dx + 2^-18), and a row's output by
    2^-8 |o|                        the final rounding to bf16
  + (2 dx + 2^-10 + 2^-8) sum w|v|  weights, and P rounded to bf16 for the MMA.
bf16 partials round each of a row's pieces once more (2^-8 of at most sum w|v|).  Over a
4-bit cache P is f16 (2^-11, within the 2^-10 above), and the last 2^-8 falls away.

Rotation: cos and sin are off by at most e = 2^-20: the fraction of a turn has 32 bits and
becomes an fp32 number (half a step of a number up to 1 half turns: 2^-25 pi), sincospi
is off by 2 units in the last place at most (2^-23 each), and the product with the magnitude
rounds once (2^-24).  The two products and their sum round to fp32 (3 times 2^-24), the
result to bf16: 2^-8 |y| + magnitude (e + 2^-22)(|x| + |z|).

Everything else (blocks, slots, positions, masks, stored bytes, moved rows) is exact."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests import step_ref as S
from tests.test_cache_ops_gpu import Batch, _built, bits, on_gpu, raw_of, terms, to_gpu  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(np.asarray(x, np.int64).astype(np.int32), device="cuda")


def same(t, want):
    np.testing.assert_array_equal(t.cpu().numpy(), np.asarray(want))


# ---------------------------------------------------------------- blocks, slots, masks
class Planned:
    """Device state of ua_plan_step beside the lists of step_ref.Step."""

    def __init__(self, seed, n, b=16, width=12, num_blocks=200, pool=60, ctx=None, spare=1):
        g = self.g = np.random.default_rng(seed)
        self.n, self.b, self.width, self.num_blocks = n, b, width, num_blocks
        self.ctx = list(ctx) if ctx is not None else [int(g.integers(0, (width - 4) * b)) for _ in range(n)]
        held = [min(width, -(-c // b) + int(g.integers(0, spare + 1))) for c in self.ctx]
        ids = g.permutation(num_blocks)
        assert sum(held) + pool <= num_blocks
        table, off = np.full((n, width), -1, np.int32), 0
        for s in range(n):
            table[s, :held[s]] = ids[off:off + held[s]]
            off += held[s]
        self.ref = S.Step(table.tolist(), held, ids[off:off + pool].tolist(), b, num_blocks)
        self.problem = ua.Problem(2, 1, 64, b, num_blocks, max(n, 1), width, 1 << 20, ua.UA_FLAG_CAUSAL, 0.125)
        self.upload()

    def upload(self):
        self.table = i32(self.ref.table).reshape(self.n, self.width)
        self.held, self.left = i32(self.ref.held), i32([len(self.ref.pool)])
        self.pool = torch.full((self.num_blocks,), -9, dtype=torch.int32, device="cuda")
        self.pool[:len(self.ref.pool)] = i32(self.ref.pool)

    def outputs(self, cap, words=0):
        kw = dict(dtype=torch.int32, device="cuda")
        return dict(granted=torch.full((self.n,), 77, **kw), cu_seqlens_q=torch.full((self.n + 1,), 77, **kw),
                    seqused_k=torch.full((self.n,), 77, **kw), positions=torch.full((cap,), 77, **kw),
                    slots=torch.full((cap,), 77, dtype=torch.int64, device="cuda"),
                    **(dict(tree_mask=torch.full((cap, words), 77, **kw)) if words else {}))

    def step(self, new, cap, trees=None, words=0, want_err=0, stride=None, stream=None):
        out = self.outputs(cap, words)
        parents = None
        if trees is not None:
            wide = stride or max([len(t) for t in trees] + [1])
            parents = i32([list(t) + [-1] * (wide - len(t)) for t in trees]).reshape(self.n, wide)
        self.problem.plan_step(self.table, self.held, self.pool, self.left, i32(self.ctx), i32(new), self.n, cap,
                               parents=parents, stream=stream, **out)
        assert self.problem.last_launch_count() == 1
        assert self.problem.check_device_error() == want_err
        want, err = self.ref.plan(self.ctx, new, cap, trees, words)
        assert err == want_err
        self.check(want, out, cap, words)
        return out, want

    def check(self, want, out, cap, words):
        total = want["cu"][-1]
        same(out["granted"], want["granted"])
        same(out["cu_seqlens_q"], want["cu"])
        same(out["seqused_k"], want["used"])
        same(out["positions"], want["pos"] + [0] * (cap - total))
        same(out["slots"], want["slots"] + [-1] * (cap - total))
        same(self.held, self.ref.held)
        same(self.left, [len(self.ref.pool)])
        same(self.pool[:len(self.ref.pool)], self.ref.pool)
        for s in range(self.n):
            same(self.table[s, :self.ref.held[s]], self.ref.table[s][:self.ref.held[s]])
        if words:
            got = out["tree_mask"].cpu().numpy().view(np.uint32)
            rows = np.concatenate(want["mask"]) if total else np.zeros((0, words), np.uint32)
            np.testing.assert_array_equal(got[:total], rows)
            assert np.all(got[total:] == 77)


@pytest.mark.parametrize("n,b,spare,pool", [(1, 16, 0, 5), (5, 16, 1, 60), (40, 32, 2, 30), (64, 64, 0, 200), (33, 16, 3, 3)])
def test_plan_chains(n, b, spare, pool):
    st = Planned(n + b, n, b, num_blocks=1000, pool=pool, spare=spare)
    for _ in range(3):
        new = [min(int(st.g.integers(0, 3 * b)), st.width * b - c) for c in st.ctx]
        out, want = st.step(new, sum(new) + 9)
        st.ctx = [max(0, u - int(st.g.integers(0, 2 * b))) for u in want["used"]]


@pytest.mark.parametrize("n,words", [(1, 1), (7, 2), (50, 3), (3, 32)])
def test_plan_trees(n, words):
    st = Planned(100 + n, n, 16, width=90, num_blocks=5000, pool=1000, ctx=[37 * s % 301 for s in range(n)])
    for k in range(2):
        trees = [S.grow(st.g, int(st.g.integers(0, 32 * words + 1))) for _ in range(n)]
        if k:
            trees[0] = S.grow(st.g, 32 * words, roots=0.0)
        new = [len(t) for t in trees]
        st.step(new, max(1, sum(new)), trees, words, stride=max(new) + 3)
        st.step([0] * n, 4)


def test_plan_with_a_dry_pool():
    """Sequences are served in their order; those that need no block are always served."""
    st = Planned(7, 6, 16, pool=3, ctx=[16, 30, 16, 5, 16, 15], spare=0)
    out, want = st.step([17, 2, 32, 8, 1, 1], 100)
    assert want["granted"] == [17, 2, 0, 8, 0, 1]
    # A request that ends gives its blocks to the others of the same call.
    st.ctx = want["used"]
    st.ctx[0] = 0
    out, want = st.step([0, 0, 32, 0, 1, 0], 100)
    assert want["granted"] == [0, 0, 32, 0, 1, 0]


def test_plan_then_back_restores_the_pool():
    st = Planned(8, 30, 16, num_blocks=500, pool=90, spare=0)
    before = st.pool.clone(), st.left.clone(), st.held.clone()
    new = [int(st.g.integers(0, 40)) for _ in range(30)]
    st.step(new, sum(new))
    assert int(st.left) < int(before[1])
    st.step([0] * 30, 1)
    for a, b in zip(before, (st.pool, st.left, st.held)):
        assert torch.equal(a, b)


def test_plan_of_many_sequences_and_many_tokens():
    """More sequences than threads, and tokens for more than one CTA; outputs over inputs."""
    n = 3000
    g = np.random.default_rng(9)
    ctx = [int(x) for x in g.integers(0, 40, n)]
    st = Planned(9, n, 16, width=40, num_blocks=90000, pool=20000, ctx=ctx)
    new = [int(x) for x in g.integers(0, 300, n)]
    cap = sum(new)
    d_ctx, d_new = i32(ctx), i32(new)
    out = st.outputs(cap)
    out["seqused_k"], out["granted"] = d_ctx, d_new
    st.problem.plan_step(st.table, st.held, st.pool, st.left, d_ctx, d_new, n, cap, **out)
    assert st.problem.check_device_error() == 0
    want, err = st.ref.plan(ctx, new, cap)
    assert err == 0 and 0 < sum(x == 0 for x in want["granted"]) < n
    st.check(want, out, cap, 0)
    st.ctx = want["used"]
    st.step([1] * n, n)


def test_plan_malformed_lengths_and_ids():
    st = Planned(10, 6, 16, pool=20, ctx=[20, 3, 50, 7, 9, 30], spare=0)
    st.ctx[1] = -1
    st.step([4, 5, -2, 16 * 12, 6, 3], 50, want_err=S.BOUNDS)
    st.ctx[1] = 3
    st.step([4, 5, 2, 7, 30, 3], 12, want_err=S.BOUNDS)              # more tokens than places
    st.ref.held[2] = 13
    st.upload()
    st.step([1, 1, 1, 1, 1, 1], 6, want_err=S.BOUNDS)
    st.ref.held[2] = 4
    st.ref.table[4][0] = 200                                        # a bad id in a table
    st.upload()
    st.step([1, 1, 1, 1, 1, 1], 6, want_err=S.BLOCK_ID)


def test_plan_pool_counts_out_of_range():
    st = Planned(11, 3, 16, num_blocks=40, pool=5, ctx=[20, 3, 0], spare=0)
    for count in (-1, 41):
        st.left = i32([count])
        out = st.outputs(9)
        st.problem.plan_step(st.table, st.held, st.pool, st.left, i32(st.ctx), i32([1, 1, 1]), 3, 9, **out)
        assert st.problem.check_device_error() == S.POOL
        same(out["granted"], [1, 1, 0])                            # only the third lacks a block
        same(st.left, [count])
    # More blocks given back than the pool has room for: they stay where they are.
    st.left = i32([39])
    held = st.held.clone()
    out = st.outputs(9)
    st.problem.plan_step(st.table, st.held, st.pool, st.left, i32([0, 0, 0]), i32([0, 0, 0]), 3, 9, **out)
    assert st.problem.check_device_error() == S.POOL
    assert torch.equal(held, st.held) and int(st.left) == 39


def test_plan_bad_parents_end_their_branch():
    st = Planned(12, 2, 16, pool=20, spare=0)
    out = st.outputs(8, 1)
    st.problem.plan_step(st.table, st.held, st.pool, st.left, i32(st.ctx), i32([3, 3]), 2, 8,
                         parents=i32([[-1, 1, 0], [-1, 0, -7]]), **out)
    assert st.problem.check_device_error() == S.TREE
    same(out["positions"][:6] - i32([st.ctx[0]] * 3 + [st.ctx[1]] * 3), [0, 0, 1, 0, 1, 0])
    same(out["tree_mask"][:6, 0], [1, 2, 5, 1, 3, 4])


def test_plan_without_sequences_or_tokens():
    st = Planned(13, 3, 16, pool=4)
    st.step([0, 0, 0], 5)
    st.step([0, 0, 0], 0)
    p = st.problem
    slots = torch.full((4,), 7, dtype=torch.int64, device="cuda")
    pos, cu = i32([7] * 4), i32([7])
    none = i32([])
    p.plan_step(torch.zeros(0, st.width, dtype=torch.int32, device="cuda"), none, st.pool, st.left, none, none, 0, 4, none,
                cu, none, pos, slots)
    assert p.check_device_error() == 0
    same(slots, [-1] * 4)
    same(pos, [0] * 4)
    same(cu, [0])


# ---------------------------------------------------------------- rotary store
ROPE = [
    # (kv, hq, hk, d, b, rot, pairs, tokens, scaling)
    ("bf16", 8, 2, 128, 16, 128, False, 5, {}),
    ("bf16", 32, 8, 128, 16, 128, True, 1, {}),
    ("bf16", 5, 5, 64, 32, 32, False, 33, dict(scaling="linear", factor=4.0)),
    ("bf16", 6, 2, 64, 16, 16, True, 7, dict(scaling="ntk", factor=8.0)),
    ("bf16", 6, 2, 64, 16, 48, False, 7, {}),
    ("bf16", 16, 1, 256, 64, 256, False, 9, dict(scaling="yarn", factor=16.0, trained=4096, low=1.0, high=32.0)),
    ("bf16", 3, 1, 256, 64, 80, True, 130, dict(scaling="bands", factor=8.0, trained=8192)),
    ("bf16", 128, 16, 64, 16, 64, False, 3, {}),
    ("fp8", 8, 2, 128, 16, 128, False, 40, {}),
    ("fp8", 8, 2, 128, 32, 64, True, 17, {}),
    ("fp4", 8, 2, 128, 16, 128, False, 40, {}),
    ("fp4", 4, 4, 64, 32, 16, False, 17, {}),
    ("fp4", 4, 2, 256, 64, 256, True, 17, {}),
]


class Rope:
    def __init__(self, case, kscale=0.25, vscale=0.5):
        kv, self.hq, self.hk, self.d, self.b, self.rot, self.pairs, n, kw = ROPE[case]
        self.kv, self.n = kv, n
        g = np.random.default_rng(500 + case)
        self.freq, self.magnitude = ua.rope_frequencies(self.rot, **kw)
        self.blocks = n // self.b + 3
        self.kscale, self.vscale = (kscale, vscale) if kv != "bf16" else (1.0, 1.0)
        pos = g.integers(0, 1 << 20, n)
        pos[:min(n, 6)] = [0, 1, 2 ** 31 - 1, 131071, 8191, 3][:n]
        self.pos, self.slots = pos, g.permutation(self.blocks * self.b)[:n]
        _, self.x = bits(g.normal(size=(n, self.hq + 2 * self.hk, self.d)))

    def problem(self):
        kind = dict(bf16=ua.UA_DTYPE_BF16, fp8=ua.UA_DTYPE_FP8_E4M3, fp4=ua.UA_DTYPE_FP4_E2M1)[self.kv]
        p = ua.Problem(self.hq, self.hk, self.d, self.b, self.blocks, 4, 8, self.n, ua.UA_FLAG_CAUSAL, 0.1, kv_dtype=kind,
                       k_scale=self.kscale, v_scale=self.vscale)
        p.set_rope(self.freq, ua.UA_ROPE_PAIRS if self.pairs else ua.UA_ROPE_HALF, self.magnitude)
        return p

    def device(self):
        self.d_x = torch.tensor(self.x, dtype=torch.float32).to(torch.bfloat16).cuda()
        self.d_q, self.d_kn, self.d_vn = self.d_x.split([self.hq, self.hk, self.hk], 1)
        self.d_pos, self.d_slots = i32(self.pos), torch.from_numpy(self.slots).cuda()
        return self

    def caches(self):
        """K's and V's reference cache and device tensor."""
        for scale in (self.kscale, self.vscale):
            c = R.Cache(self.kv, self.blocks, self.b, self.hk, self.d, scale, 0x55)
            yield c, to_gpu(c)


def check_rotated(got, x, pos, freq, pairs, magnitude):
    want = S.rotate(x, pos, freq, pairs, magnitude)
    n = len(freq)
    other = np.zeros_like(x)
    if pairs:
        other[..., 0:2 * n:2], other[..., 1:2 * n:2] = x[..., 1:2 * n:2], x[..., 0:2 * n:2]
    else:
        other[..., :n], other[..., n:2 * n] = x[..., n:2 * n], x[..., :n]
    turned = np.zeros(x.shape[-1], bool)
    turned[:2 * n] = True
    bound = 2.0 ** -8 * np.abs(want) + abs(magnitude) * (2.0 ** -20 + 2.0 ** -22) * (np.abs(x) + np.abs(other))
    err = np.abs(got - want)
    assert np.all(err <= bound), float((err / (bound + 1e-30)).max())
    np.testing.assert_array_equal(got[..., ~turned], x[..., ~turned])


@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_store(case):
    r = Rope(case).device()
    p = r.problem()
    (kc, d_k), (vc, d_v) = r.caches()
    q_out = p.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, d_k, d_v)
    assert p.check_device_error() == 0 and p.last_launch_count() == 1 and p.last_path() == "rope_store"
    check_rotated(q_out.double().cpu().numpy(), r.x[:, :r.hq], r.pos, r.freq, r.pairs, r.magnitude)
    # The rotated keys as bf16: from a bf16 cache.
    r16 = ua.Problem(r.hq, r.hk, r.d, r.b, r.blocks, 4, 8, r.n, ua.UA_FLAG_CAUSAL, 0.1)
    r16.set_rope(r.freq, ua.UA_ROPE_PAIRS if r.pairs else ua.UA_ROPE_HALF, r.magnitude)
    k16 = torch.full((r.blocks, r.b, r.hk, r.d), 9.0, dtype=torch.bfloat16, device="cuda")
    v16 = k16.clone()
    r16.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, k16, v16)
    k_rot = k16.view(-1, r.hk, r.d)[r.d_slots]
    assert torch.equal(v16.view(-1, r.hk, r.d)[r.d_slots], r.d_vn)
    left = torch.ones(r.blocks * r.b, dtype=torch.bool)
    left[r.slots] = False
    assert bool((k16.view(-1, r.hk, r.d).cpu()[left] == 9).all() and (v16.view(-1, r.hk, r.d).cpu()[left] == 9).all())
    check_rotated(k_rot.double().cpu().numpy(), r.x[:, r.hq:r.hq + r.hk], r.pos, r.freq, r.pairs, r.magnitude)
    # What is stored: those values in the cache's format, other rows untouched.
    kb = k_rot.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    vb = r.d_vn.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    for t in range(r.n):
        blk, slot = divmod(int(r.slots[t]), r.b)
        kc.put(blk, slot, R.bf16_values(k_rot[t]), kb[t])
        vc.put(blk, slot, R.bf16_values(r.d_vn[t]), vb[t])
    np.testing.assert_array_equal(raw_of(d_k, r.kv), kc.raw)
    np.testing.assert_array_equal(raw_of(d_v, r.kv), vc.raw)


@pytest.mark.parametrize("case", [8, 10])
def test_rope_store_tensor_scales_that_are_no_powers_of_two(case):
    r = Rope(case, kscale=0.03, vscale=1.7).device()
    p = r.problem()
    (kc, d_k), (vc, d_v) = r.caches()
    p.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, d_k, d_v)
    vb = r.d_vn.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    for t in range(r.n):
        vc.put(*divmod(int(r.slots[t]), r.b), R.bf16_values(r.d_vn[t]), vb[t])
    np.testing.assert_array_equal(raw_of(d_v, r.kv), vc.raw)
    # K against the store of the rotated keys (chains in whole sequences of one block).
    k16 = torch.zeros(r.blocks, r.b, r.hk, r.d, dtype=torch.bfloat16, device="cuda")
    r16 = ua.Problem(r.hq, r.hk, r.d, r.b, r.blocks, 4, 8, r.n, ua.UA_FLAG_CAUSAL, 0.1)
    r16.set_rope(r.freq, int(r.pairs), r.magnitude)
    r16.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, k16, k16.clone())
    rows = k16.view(-1, r.hk, r.d)[r.d_slots]
    raw = rows.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)
    for t in range(r.n):
        kc.put(*divmod(int(r.slots[t]), r.b), R.bf16_values(rows[t]), raw[t])
    np.testing.assert_array_equal(raw_of(d_k, r.kv), kc.raw)


@pytest.mark.parametrize("case", [0, 1, 4])
def test_rope_in_place_and_padding_tokens(case):
    """q rotated over itself inside the fused rows; tokens with slot -1 are not stored, rows
    behind total_q stay; a slot past the cache is reported."""
    r = Rope(case).device()
    p = r.problem()
    want = p.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, *[c[1] for c in r.caches()])
    x = torch.cat([r.d_x, r.d_x])
    q, kn, vn = x.split([r.hq, r.hk, r.hk], 1)
    (_, d_k), (_, d_v) = r.caches()
    before = d_k.clone()
    slots = torch.full_like(r.d_slots, -1)
    out = p.rope_store(q, kn, vn, r.d_pos, slots, r.n, d_k, d_v, q_out=q)
    assert out.data_ptr() == q.data_ptr() and p.check_device_error() == 0
    assert torch.equal(q[:r.n], want) and torch.equal(q[r.n:], r.d_q)
    assert torch.equal(kn, torch.cat([r.d_kn, r.d_kn])) and torch.equal(vn, torch.cat([r.d_vn, r.d_vn]))
    assert torch.equal(d_k.view(torch.int16), before.view(torch.int16))
    slots[0] = r.blocks * r.b
    p.rope_store(q[r.n:], kn, vn, r.d_pos, slots, r.n, d_k, d_v)
    assert p.check_device_error() == S.BLOCK_ID
    assert torch.equal(d_k.view(torch.int16), before.view(torch.int16))


def test_rope_values_that_are_not_finite_stay_with_their_pair():
    r = Rope(0)
    r.x[0, 0, 5], r.x[1, 8, 70], r.x[2, 9, 100] = np.nan, np.inf, -np.inf
    r.device()
    p = r.problem()
    k = torch.zeros(r.blocks, r.b, r.hk, r.d, dtype=torch.bfloat16, device="cuda")
    q = p.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, k, k.clone()).float().cpu().numpy()
    bad = np.argwhere(~np.isfinite(q)).tolist()
    assert bad == [[0, 0, 5], [0, 0, 69]]
    rows = k.view(-1, r.hk, r.d)[r.d_slots].float().cpu().numpy()
    assert np.argwhere(~np.isfinite(rows)).tolist() == [[1, 0, 6], [1, 0, 70], [2, 1, 36], [2, 1, 100]]


def test_rope_frequencies_are_taken_by_value():
    """Frequencies set again do not reach calls that were captured before."""
    r = Rope(0).device()
    p = r.problem()
    k, v = (torch.zeros(r.blocks, r.b, r.hk, r.d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = torch.zeros(r.n, r.hq, r.d, dtype=torch.bfloat16, device="cuda")
    call = lambda: p.rope_store(r.d_q, r.d_kn, r.d_vn, r.d_pos, r.d_slots, r.n, k, v, q_out=out)  # noqa: E731
    want = call().clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    p.set_rope([0.0] * 32, ua.UA_ROPE_PAIRS)
    assert torch.equal(call(), r.d_q)
    graph.replay()
    assert torch.equal(out, want)


# ---------------------------------------------------------------- attention for draft trees
class Trees(Batch):
    """A batch whose chunks are trees."""

    def __init__(self, seed, hq, hk, d, b, sq, sk, words=None, kind="bf16", **kw):
        super().__init__(seed, kind, hq, hk, d, b, sq, sk, **kw)
        self.trees = [S.grow(self.rng, n) for n in sq]
        self.words = words or max(1, -(-max(sq) // 32))
        self.mask = np.concatenate([S.mask_of(t, self.words) for t in self.trees])
        self.pos = [np.array(S.depths(t)) + k - len(t) for t, k in zip(self.trees, sk)]

    def see(self, s):
        a, z = R.tokens_of(self.cu, s)
        m = self.mask[a:z]
        return np.array([[bool(m[i, c // 32] >> np.uint32(c % 32) & np.uint32(1)) for c in range(z - a)]
                         for i in range(z - a)], bool).reshape(z - a, z - a)

    def run(self, p, flags, sinks=None, alibi=None, out=None, stream=None, pos=True):
        return p.forward_tree(self.d_q, self.d_k, self.d_v, self.d_table, self.d_cu, self.d_sk, self.n, sum(self.sq),
                              max(self.sq), max(self.sk), flags, torch.from_numpy(self.mask.view(np.int32)).cuda(),
                              positions=i32(np.concatenate(self.pos)) if pos else None, sinks=on_gpu(sinks),
                              alibi_slopes=on_gpu(alibi), out=out, stream=stream)

    def want(self, s, **kw):
        a, z = R.tokens_of(self.cu, s)
        return S.tree_attention(self.q[a:z], self.kc.rows(self.table[s], self.sk[s]),
                                self.vc.rows(self.table[s], self.sk[s]), self.scale, self.see(s), pos=self.pos[s], **kw)

    def check(self, got, softcap=0.0, bf16_parts=False, only=None, **kw):
        got = got.double().cpu().numpy()
        extra = max(self.sk) if kw.get("alibi") is not None else 0.0
        for s in range(self.n) if only is None else only:
            a, z = R.tokens_of(self.cu, s)
            if a == z:
                continue
            o, total, mag = self.want(s, softcap=softcap, **kw)
            dx = R.score_error(mag, self.d, softcap, extra)
            per = 2 * dx + 2.0 ** -10 + (2.0 ** -8 if self.kind == "bf16" else 0.0) + (2.0 ** -8 if bf16_parts else 0.0)
            ok = np.isfinite(o)
            np.testing.assert_array_equal(ok, np.isfinite(got[a:z]))
            bound = 2.0 ** -8 * np.abs(o[ok]) + per * total[ok] + 1e-30
            err = np.abs(got[a:z][ok] - o[ok])
            assert np.all(err <= bound), (s, float((err / bound).max()))


TREE = [
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
]


@pytest.mark.parametrize("case", range(len(TREE)))
@pytest.mark.parametrize("partials", [ua.UA_PARTIALS_F32, ua.UA_PARTIALS_BF16])
def test_tree_attention(case, partials):
    hq, hk, d, b, sq, sk, kw = TREE[case]
    bt = Trees(700 + case, hq, hk, d, b, sq, sk).device()
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    p = bt.problem(flags, softcap=softcap, window=window, split_partials=partials)
    out = torch.full_like(bt.d_q, 3.0)
    got = bt.run(p, flags, sinks, alibi, out=out, pos=bool(window or kw.get("alibi")))
    assert p.check_device_error() == 0 and p.last_path().startswith("tree")
    bt.check(got, softcap, partials == ua.UA_PARTIALS_BF16, window=window, sinks=sinks, alibi=alibi)


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 4, 64), (8, 1, 256)])
def test_tree_masks_that_are_no_trees(hq, hk, d):
    """Any bits: rows that see nothing of the chunk, or later keys; without context a
    row may see nothing at all."""
    bt = Trees(740, hq, hk, d, 16, (40, 33, 5), (40, 90, 5), words=3)
    bt.mask = bt.rng.integers(0, 1 << 32, bt.mask.shape, dtype=np.uint64).astype(np.uint32)
    bt.mask[3] = bt.mask[17] = bt.mask[45] = bt.mask[75] = 0
    bt.device()
    p = bt.problem()
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == 0
    bt.check(got)
    assert bool((got[[3, 17, 75]] == 0).all())
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_SINKS
    sinks = np.full(hq, 0.5, np.float32)
    sinks[0], sinks[1] = np.inf, -np.inf
    p = bt.problem(flags)
    got = bt.run(p, flags, sinks, pos=False)
    bt.check(got, sinks=sinks.astype(np.float64))


def test_a_chain_gives_what_forward_gives():
    bt = Trees(741, 8, 2, 128, 16, (20, 33, 1), (20, 400, 77))
    bt.trees = [list(range(-1, n - 1)) for n in bt.sq]
    bt.mask = np.concatenate([S.mask_of(t, bt.words) for t in bt.trees])
    bt.pos = [np.arange(k - n, k) for n, k in zip(bt.sq, bt.sk)]
    bt.device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_WINDOW
    p = bt.problem(flags, window=30)
    got = bt.run(p, flags)
    bt.check(got, window=30)
    plain = p.forward(*bt.args(), flags).double().cpu().numpy()
    for s in range(bt.n):
        a, z = R.tokens_of(bt.cu, s)
        o, total, _ = bt.want(s, window=30)
        # Each side is within its bound of the same value.
        assert np.all(np.abs(plain[a:z] - got[a:z].double().cpu().numpy()) <= 2.0 ** -7 * np.abs(o) + 2.0 ** -6 * total + 1e-30)


@pytest.mark.parametrize("d,window", [(64, 0), (128, 0), (256, 0), (128, 25)])
def test_tree_values_that_are_not_finite_reach_the_rows_that_see_them(d, window):
    """NaN and infinities in V and K of nodes, of keys in front of the window, and in
    slots behind the end."""
    bt = Trees(742, 8, 2, d, 16, (40, 20), (150, 333), store=False)
    bt.trees = [[-1, 0, 0, 1, 1, 2] + [2] * 34, [-1, 0] + [0] * 18]
    bt.mask = np.concatenate([S.mask_of(t, bt.words) for t in bt.trees])
    bt.pos = [np.array(S.depths(t)) + k - len(t) for t, k in zip(bt.trees, bt.sk)]
    for node, dim, x in ((4, 3, np.nan), (9, 7, np.inf), (10, 7, -np.inf), (39, d - 1, np.nan)):
        bt.v[0][110 + node, 1, dim] = x
    bt.k[0][110 + 12, 0, 1] = np.nan
    bt.k[0][110 + 13, 0] = np.inf
    if window:
        bt.v[1][:313 - window + 1] = np.nan       # in front of every window
        bt.v[1][313 - window + 1, :, 5] = np.inf  # seen by the root alone
        bt.k[1][:200] = np.nan
    for s in range(2):
        (bt.kb[s], bt.k[s]), (bt.vb[s], bt.v[s]) = bits(bt.k[s]), bits(bt.v[s])
        for j in range(bt.sk[s]):
            bt.put(s, j)
    bt.device()
    flags = ua.UA_FLAG_CAUSAL | (ua.UA_FLAG_WINDOW if window else 0)
    p = bt.problem(flags, window=window)
    got = bt.run(p, flags)
    assert p.check_device_error() == 0
    g = got.double().cpu().numpy()
    seen = lambda s, i: int(bt.cu[s]) + i  # noqa: E731
    # Node 4's NaN stays with node 4 in KV head 1's query heads; nodes 9 and 10 have their own infinity.
    assert np.argwhere(np.isnan(g[:40, 4:])).tolist() == [[4, h, 3] for h in range(4)] + [[39, h, d - 1] for h in range(4)]
    assert (~np.isfinite(g[:40, 4:])).sum() == 16
    assert np.all(g[9, 4:, 7] == np.inf) and np.all(g[10, 4:, 7] == -np.inf)
    # NaN scores make their own rows NaN, and only those.
    rows = {i for i in range(40) if np.isnan(g[i, :4]).all()}
    assert {12} <= rows <= {12, 13} and np.isfinite(np.delete(g[:40, :4], [12, 13], 0)).all()
    if window:
        assert np.all(g[seen(1, 0), :, 5] == np.inf) and np.isfinite(np.delete(g[40:], 0, 0)).all()
    with np.errstate(invalid="ignore", over="ignore"):
        o, total, mag = bt.want(0, window=window)
    keep = np.isfinite(o) & np.isfinite(g[:40])
    keep[12:14] = False
    dx = R.score_error(40.0 * d ** 0.5, d)
    bound = 2.0 ** -8 * np.abs(o[keep]) + (2 * dx + 2.0 ** -10 + 2.0 ** -8) * total[keep] + 1e-30
    assert np.all(np.abs(g[:40][keep] - o[keep]) <= bound)


def test_tree_malformed_sequences_and_blocks():
    bt = Trees(743, 8, 2, 128, 16, (9, 12, 6, 4), (60, 40, 100, 30)).device()
    p = bt.problem()
    good = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    bt.d_sk = i32([60, 5, 100, 30])                  # fewer keys than nodes
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == ua.UA_DEVERR_CONTEXT
    assert bool((got[9:21] == 0).all()) and torch.equal(got[:9], good[:9]) and torch.equal(got[21:], good[21:])
    bt.d_sk = i32(bt.sk)
    bt.d_table[2, 1] = bt.blocks + 5
    got = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() == ua.UA_DEVERR_BLOCK_ID
    assert torch.equal(got[:21], good[:21]) and torch.equal(got[27:], good[27:]) and bool(got.isfinite().all())


def test_tree_positions_outside_the_chunk_are_reported():
    bt = Trees(744, 4, 2, 64, 16, (5, 3), (40, 20)).device()
    bt.pos[0][2] = 2000
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_WINDOW
    p = bt.problem(flags, window=10)
    got = bt.run(p, flags)
    assert p.check_device_error() == ua.UA_DEVERR_TREE
    bt.pos[0][2] = 39
    bt.check(got, window=10)


def test_tree_stall_hook_gives_up():
    from paged_varlen_flash_gb300 import binding
    bt = Trees(745, 8, 2, 128, 16, (9, 4), (600, 300)).device()
    p = bt.problem()
    good = bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert binding.ua_debug_stall_data_waits(p.handle, 1, 2_000_000) == 0
    bt.run(p, ua.UA_FLAG_CAUSAL, pos=False)
    assert p.check_device_error() & ua.UA_DEVERR_TIMEOUT
    assert binding.ua_debug_stall_data_waits(p.handle, 0) == 0
    assert torch.equal(bt.run(p, ua.UA_FLAG_CAUSAL, pos=False), good)
    assert p.check_device_error() == 0


# ---------------------------------------------------------------- accepted branches
ACCEPT = [
    # (kind, hk, d, b, S_q, S_k)
    ("bf16", 2, 128, 16, (9, 1, 0, 30, 64), (40, 17, 20, 30, 500)),
    ("bf16", 8, 256, 64, (20, 33), (20, 100)),
    ("bf16", 1, 64, 32, (200,), (231,)),
    ("bf16", 40, 128, 16, (12, 7), (100, 7)),
    ("fp8", 3, 128, 16, (25, 8), (60, 41)),
    ("fp4", 2, 64, 16, (25, 8, 1), (60, 41, 9)),
    ("fp4", 4, 256, 64, (64, 3), (100, 90)),
]


def accept_reference(bt, trees, last, path_width):
    path = np.full((bt.n, path_width), -1, np.int32)
    count = []
    for s in range(bt.n):
        way = S.branch(trees[s], last[s]) if bt.sq[s] else []
        count.append(len(way))
        path[s, :len(way)] = way
        ctx = bt.sk[s] - bt.sq[s]
        for c in (bt.kc, bt.vc):
            for t, r in enumerate(way):
                if t != r:
                    for h in range(bt.hk):
                        row = c.row_bytes(int(bt.table[s, (ctx + r) // bt.b]), (ctx + r) % bt.b, h)
                        c.set_row_bytes(int(bt.table[s, (ctx + t) // bt.b]), (ctx + t) % bt.b, h, row)
    return path, count


@pytest.mark.parametrize("case", range(len(ACCEPT)))
@pytest.mark.parametrize("shape", ["bushy", "long"])
def test_accept_moves_the_branch(case, shape):
    kind, hk, d, b, sq, sk = ACCEPT[case]
    bt = Batch(900 + case, kind, 2 * hk, hk, d, b, sq, sk).device()
    trees = [S.grow(bt.rng, n, 0.7 if shape == "bushy" else 0.1, 0.02) for n in sq]
    wide = max(sq) + 2
    parents = torch.full((bt.n, wide + 3), -5, dtype=torch.int32, device="cuda")
    for s, t in enumerate(trees):
        parents[s, :len(t)] = i32(t)
    last = [int(bt.rng.integers(-1, n)) if s else n - 1 for s, n in enumerate(sq)]
    path, accepted = torch.full((bt.n, wide), 7, dtype=torch.int32, device="cuda"), i32([7] * bt.n)
    p = bt.problem()
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, parents[:, :wide], i32(last), bt.n, sum(sq), max(sq),
                   max(sk), path, accepted, bt.d_sk)
    assert p.check_device_error() == 0 and p.last_launch_count() == 1 and p.last_path() == "accept"
    want_path, count = accept_reference(bt, trees, last, wide)
    same(path, want_path)
    same(accepted, count)
    same(bt.d_sk, [k - n + c for k, n, c in zip(sk, sq, count)])
    np.testing.assert_array_equal(raw_of(bt.d_k, kind), bt.kc.raw)
    np.testing.assert_array_equal(raw_of(bt.d_v, kind), bt.vc.raw)


def test_accept_of_the_largest_tree_and_a_chain():
    """1024 nodes in one branch that skips a node now and then."""
    bt = Batch(920, "bf16", 2, 1, 64, 16, (1024, 1024), (1030, 1500)).device()
    skip = [-1] + [max(0, i - 1 - (i % 5 == 0)) for i in range(1, 1024)]
    trees = [skip, list(range(-1, 1023))]
    p = bt.problem(max_total_q=2048)
    path, out, used = torch.zeros(2, 1024, dtype=torch.int32, device="cuda"), i32([0, 0]), i32([0, 0])
    before = bt.d_k.clone()
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, i32(trees), i32([1023, 1023]), 2, 2048, 1024, 1500, path,
                   out, used)
    assert p.check_device_error() == 0
    want, count = accept_reference(bt, trees, [1023, 1023], 1024)
    same(path, want)
    same(out, count)
    assert count[1] == 1024 and count[0] < 1024 and not torch.equal(before.view(torch.int16), bt.d_k.view(torch.int16))
    np.testing.assert_array_equal(raw_of(bt.d_k, "bf16"), bt.kc.raw)


def test_accept_refuses_what_is_malformed():
    """Bad parents, nodes, lengths and block ids: nothing of that sequence moves, the
    others are served."""
    bt = Batch(921, "bf16", 2, 1, 64, 16, (6, 6, 6, 6, 6, 6), (30, 30, 30, 30, 30, 30)).device()
    tree = [-1, 0, 0, 1, 2, 4]
    parents = i32([tree] * 6)
    parents[1, 4] = 4
    parents[2, 4] = -2
    last = i32([5, 5, 5, 6, -2, 5])
    path, out, used = torch.zeros(6, 8, dtype=torch.int32, device="cuda"), i32([7] * 6), i32([7] * 6)
    before = bt.d_k.clone()
    p = bt.problem()
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, parents, last, 6, 36, 6, 30, path, out, used)
    assert p.check_device_error() == ua.UA_DEVERR_TREE
    same(out, [4, 0, 0, 0, 0, 4])
    same(used, [28, 24, 24, 24, 24, 28])
    same(path[:, :5], [[0, 2, 4, 5, -1]] + [[-1] * 5] * 4 + [[0, 2, 4, 5, -1]])
    moved = (before.view(torch.int16) != bt.d_k.view(torch.int16)).flatten(1).any(1).nonzero()[:, 0].tolist()
    assert set(moved) == {int(bt.table[s, 24 // 16]) for s in (0, 5)}
    # A path row that is too short, and lengths the call does not allow.
    short = torch.zeros(6, 3, dtype=torch.int32, device="cuda")
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, i32([tree] * 6), i32([1] * 5 + [5]), 6, 36, 6, 30, short,
                   out, used)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS
    same(out, [2] * 5 + [0])
    bt.d_sk = i32([30, 3, 30, 30, 30, 31])
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, i32([tree] * 6), i32([1] * 6), 6, 36, 6, 30, path, out, used)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS | ua.UA_DEVERR_CONTEXT
    same(out, [2, 0, 2, 2, 2, 0])
    same(used, [26, 0, 26, 26, 26, 0])
    bt.d_sk = i32([30] * 6)
    bt.d_table[0, 1] = -4
    p.cache_accept(bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, i32([tree] * 6), i32([5] * 6), 6, 36, 6, 30, path, out, used)
    assert p.check_device_error() == ua.UA_DEVERR_BLOCK_ID
    same(out, [4] * 6)
