"""The cache operators on batches long enough that their persistent kernels reach the
steady state (rings that wrap, several pieces of work per warp or CTA, KV segments, runs
of keys past one CTA's shared memory), against 64-bit torch implementations on the GPU.

Tolerances: tests/test_cache_ops_gpu.py, and one term more.  P = 2^(x - m) goes into the
MMA as f16, whose steps below 2^-14 are 2^-24: a smaller P is off by up to 2^-25, whatever
its size.  m is a maximum over some of the row's keys, so the key with the row's largest
score has P >= 1 and the row sum that divides is >= 1 (joins with other segments or the
sink multiply by at most 1): the output is off by at most 2^-25 sum |v| over the keys the
row sees.  It shows where a dim's only nonzero values have weights below 2^-14."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R
from tests.test_cache_ops_gpu import DT, _built, evict_weights, terms  # noqa: F401

pytestmark = pytest.mark.gpu


class LongBatch:
    """A batch over caches of random codes (4-bit, fp8) or values (bf16)."""

    def __init__(self, seed, kind, hq, hk, d, b, sq, sk, qmax=1.0):
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kind, self.hq, self.hk, self.d, self.b = kind, hq, hk, d, b
        self.sq, self.sk, self.n = list(sq), list(sk), len(sk)
        nblk = [-(-k // b) for k in sk]
        self.width, self.blocks = max(nblk), sum(nblk) + 2
        ids = torch.randperm(self.blocks, generator=self.gen, device="cuda").to(torch.int32)
        self.table = torch.full((self.n, self.width), -1, dtype=torch.int32, device="cuda")
        off = 0
        for s in range(self.n):
            self.table[s, :nblk[s]] = ids[off:off + nblk[s]]
            off += nblk[s]
        self.k, self.v = self.cache(), self.cache()
        self.cu = torch.tensor([0] + self.sq, device="cuda").cumsum(0).to(torch.int32)
        self.used = torch.tensor(self.sk, dtype=torch.int32, device="cuda")
        self.q = (qmax * torch.randn(sum(sq), hq, d, generator=self.gen, device="cuda")).to(torch.bfloat16)
        self.kscale, self.vscale, self.scale = (0.5, 0.25, d ** -0.5) if kind != "bf16" else (1.0, 1.0, d ** -0.5)

    def cache(self):
        shape = ua.cache_shape(self.blocks, self.hk, self.d, self.b, DT[self.kind])
        if self.kind == "bf16":
            return torch.randn(shape, generator=self.gen, device="cuda").to(torch.bfloat16)
        c = torch.randint(0, 256, shape, generator=self.gen, device="cuda", dtype=torch.uint8)
        if self.kind == "fp8":
            return torch.where((c & 0x7f) > 0x48, c & 0x8f, c)        # no NaN, magnitudes up to 4
        n = self.b * self.d // 2
        c[..., n:] = c[..., n:] % 0x18 + 0x28                         # scales 0.25 to 1.875
        return c

    def problem(self, flags, **kw):
        return ua.Problem(self.hq, self.hk, self.d, self.b, self.blocks, self.n, self.width, sum(self.sq), flags,
                          self.scale, kv_dtype=DT[self.kind], k_scale=self.kscale, v_scale=self.vscale, **kw)

    def args(self):
        return (self.q, self.k, self.v, self.table, self.cu, self.used, self.n, sum(self.sq), max(self.sq),
                max(self.sk))

    def rows(self, cache, s, factor):
        """float64 [S_k, H_k, d]."""
        pages = cache[self.table[s, :-(-self.sk[s] // self.b)].long()]
        if self.kind == "fp4":
            n, w, g = self.b * self.d // 2, self.d // 2, self.d // 16
            codes = pages[..., :n].unflatten(-1, (self.b, w))
            codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
            lut = torch.tensor(np.concatenate([R.E2M1, -R.E2M1]), device="cuda")
            sc = pages[..., n:].view(torch.float8_e4m3fn).double().unflatten(-1, (self.b, g))
            x = (lut[codes.int()] * sc.repeat_interleave(16, -1)).permute(0, 2, 1, 3)
        elif self.kind == "fp8":
            x = pages.view(torch.float8_e4m3fn).double()
        else:
            x = pages.double()
        return x.flatten(0, 1)[:self.sk[s]] * factor

    def reference(self, s, causal=True, softcap=0.0, window=0, sinks=None, alibi=None):
        """out, sum of weight |v| and of |v| [S_q, H_q, d], weights [H_k, S_k], mag, all float64."""
        sq, sk, g, ctx = self.sq[s], self.sk[s], self.hq // self.hk, self.sk[s] - self.sq[s]
        q = self.q[int(self.cu[s]):int(self.cu[s + 1])].double()
        keys, values = self.rows(self.k, s, self.kscale), self.rows(self.v, s, self.vscale)
        j, i = torch.arange(sk, device="cuda"), torch.arange(sq, device="cuda")
        see = torch.ones(sq, sk, dtype=torch.bool, device="cuda")
        if causal:
            see &= j <= i[:, None] + ctx
        if window:
            see &= j >= i[:, None] + ctx - window + 1
        out, absout, seen = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q)
        weights, mag = torch.zeros(self.hk, sk, dtype=torch.float64, device="cuda"), 0.0
        for h in range(self.hq):
            kh, vh = keys[:, h // g], values[:, h // g]
            x = q[:, h] @ kh.T * self.scale
            mag = max(mag, float((q[:, h].abs() @ kh.abs().T).max()) * self.scale)
            if softcap:
                x = softcap * torch.tanh(x / softcap)
            if alibi is not None:
                x = x + float(alibi[h]) * (j - ctx)
            x = x.masked_fill(~see, -torch.inf)
            if sinks is not None:
                x = torch.cat([x, torch.full((sq, 1), float(sinks[h]), device="cuda", dtype=torch.float64)], 1)
            p = torch.softmax(x, -1)[:, :sk]
            weights[h // g] += p.sum(0)
            out[:, h], absout[:, h], seen[:, h] = p @ vh, p @ vh.abs(), see.double() @ vh.abs()
        return out, absout, seen, weights, mag


def check(bt, s, got, ref, softcap=0.0, extra=0.0, bf16_p=False):
    out, absout, seen, _, mag = ref
    got = got[int(bt.cu[s]):int(bt.cu[s + 1])].double()
    per = 2 * R.score_error(mag, bt.d, softcap, extra) + 2.0 ** -10 + (2.0 ** -7 + 2.0 ** -8 if bf16_p else 0.0)
    bound = 2.0 ** -8 * out.abs() + per * absout + 2.0 ** -25 * seen + 1e-30
    assert bool(torch.isfinite(got).all())
    assert bool(((got - out).abs() <= bound).all()), (s, float(((got - out).abs() / bound).max()))


def check_weights(bt, s, got, old, ref, softcap=0.0, extra=0.0):
    """got [H_k, S_k] against old (decayed, 0 for the chunk's own keys) + fresh."""
    fresh, mag = ref[3:]
    n_rows = bt.hq // bt.hk * bt.sq[s]
    want = old + fresh
    bound = (fresh * (2 * R.score_error(mag, bt.d, softcap, extra) + 2.0 ** -18 + (n_rows + 4) * 2.0 ** -24) +
             want.abs() * 2.0 ** -22 + 1e-30)
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (s, float((err / bound).max()))


def ragged(seed, n, lo, hi, sq_lo, sq_hi):
    g = np.random.default_rng(seed)
    sq = [int(x) for x in g.integers(sq_lo, sq_hi + 1, n)]
    return sq, [q + int(x) for q, x in zip(sq, g.integers(lo, hi + 1, n))]


# ---------------------------------------------------------------- attention, register kernel
ATTEND = [
    # (hq, hk, d, b, n, keys lo, hi, S_q lo, hi, terms)
    (32, 8, 128, 16, 16, 1000, 12000, 1, 1, {}),                       # about 14 steps a warp
    (32, 8, 128, 32, 200, 1, 400, 1, 1, dict(sinks=True)),             # several jobs a warp
    (32, 8, 128, 64, 90, 1, 3000, 1, 4, dict(softcap=20.0)),           # 16-row tiles
    (8, 2, 64, 16, 60, 100, 20000, 1, 6, dict(window=1500, alibi=True)),
    (16, 2, 256, 64, 6, 20000, 40000, 1, 1, {}),
    (16, 2, 256, 32, 40, 1, 6000, 1, 3, dict(sinks=True)),
    (40, 8, 64, 64, 700, 1, 90, 1, 2, {}),                             # two rounds of the work split
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_long_attention_over_4_bits(case):
    hq, hk, d, b, n, lo, hi, sq_lo, sq_hi, kw = ATTEND[case]
    bt = LongBatch(400 + case, "fp4", hq, hk, d, b, *ragged(case, n, lo, hi, sq_lo, sq_hi))
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    dev = [None if x is None else torch.from_numpy(x).cuda() for x in (sinks, alibi)]
    p = bt.problem(flags, softcap=softcap, window=window)
    got = p.forward(*bt.args(), flags, *dev)
    again = p.forward(*bt.args(), flags, *dev)
    assert p.check_device_error() == 0 and p.last_path() == "fp4+merge"
    assert torch.equal(got.view(torch.int16), again.view(torch.int16))
    # Every sequence is part of some share; a spread of them is compared.
    for s in sorted(set(range(0, n, max(1, n // 24))) | {n - 1, int(np.argmax(bt.sk)), int(np.argmin(bt.sk))}):
        check(bt, s, got, bt.reference(s, softcap=softcap, window=window, sinks=sinks, alibi=alibi), softcap,
              max(bt.sk) if alibi is not None else 0.0)


# ---------------------------------------------------------------- key weights
WEIGHTS = [
    # (kind, hq, hk, d, b, n, keys lo, hi, S_q lo, hi, decay, terms, path)
    ("fp4", 32, 8, 128, 32, 8, 1000, 12000, 8, 32, 0.0, {}, "rows"),
    ("fp4", 32, 8, 128, 16, 7, 1000, 12000, 8, 32, 0.9, dict(window=3000, softcap=20.0), "rows"),
    ("fp4", 16, 8, 128, 64, 10, 8000, 8192, 16, 60, 1.0, dict(sinks=True), "rows"),       # 17 tiles a CTA: two runs
    ("fp4", 32, 8, 64, 16, 12, 1, 9000, 9, 70, 0.5, dict(alibi=True), "rows"),
    ("fp4", 8, 2, 64, 64, 6, 3000, 30000, 40, 300, 0.0, dict(window=700), "rows"),
    ("fp4", 16, 8, 256, 64, 8, 500, 6000, 20, 90, 1.0, {}, "rows"),
    ("fp4", 16, 2, 256, 32, 5, 1000, 20000, 5, 40, 0.9, dict(window=5000, softcap=30.0, sinks=True), "rows"),
    ("fp4", 12, 4, 128, 16, 3, 10, 2500, 400, 700, 0.0, {}, "rows"),
    ("fp4", 8, 2, 128, 16, 3, 300, 5000, 30, 90, 1.0, dict(causal=False), "rows"),
    ("fp4", 32, 8, 128, 16, 24, 500, 8000, 1, 1, 1.0, {}, "merge"),
    ("fp4", 32, 8, 128, 64, 16, 500, 8000, 2, 5, 0.9, dict(window=1000, sinks=True), "merge"),
    ("bf16", 32, 8, 128, 16, 16, 500, 8000, 1, 1, 1.0, {}, "decode"),
    ("bf16", 32, 8, 128, 32, 4, 1000, 6000, 8, 32, 0.9, dict(window=1500), "decode"),
    ("bf16", 16, 2, 256, 64, 3, 1000, 6000, 1, 9, 0.0, dict(softcap=20.0), "decode"),
    ("fp8", 32, 8, 128, 16, 6, 500, 9000, 1, 20, 0.5, dict(sinks=True), "decode"),
]


@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_long_key_weights(case):
    kind, hq, hk, d, b, n, lo, hi, sq_lo, sq_hi, decay, kw, path = WEIGHTS[case]
    bt = LongBatch(430 + case, kind, hq, hk, d, b, *ragged(30 + case, n, lo, hi, sq_lo, sq_hi))
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    dev = [None if x is None else torch.from_numpy(x).cuda() for x in (sinks, alibi)]
    p = bt.problem(flags | ua.UA_FLAG_KEY_WEIGHTS, softcap=softcap, window=window)
    w_in = torch.empty(n, hk, max(bt.sk) + 3, device="cuda").exponential_(generator=bt.gen)
    w = [torch.full_like(w_in, -7.0) for _ in range(2)]
    out = [p.forward_weights(*bt.args(), flags, w_in, x, decay=decay, sinks=dev[0], alibi_slopes=dev[1]) for x in w]
    assert p.check_device_error() == 0 and path in p.last_path()
    assert torch.equal(w[0], w[1]) and torch.equal(out[0].view(torch.int16), out[1].view(torch.int16))
    extra = max(bt.sk) if alibi is not None else 0.0
    for s in range(n):
        ref = bt.reference(s, kw.get("causal", True), softcap, window, sinks, alibi)
        sk, ctx = bt.sk[s], bt.sk[s] - bt.sq[s]
        old = torch.where(torch.arange(sk, device="cuda") < ctx, decay * w_in[s, :, :sk].double(), 0.0)
        check_weights(bt, s, w[0][s, :, :sk], old, ref, softcap, extra)
        assert bool((w[0][s, :, sk:] == -7.0).all())
        check(bt, s, out[0], ref, softcap, extra, bf16_p=kind == "bf16")


# ---------------------------------------------------------------- eviction
EVICT = [
    # (kind, hk, d, b, S_k, budget, recent): clusters of 2, 4 and 8 CTAs, and runs past shared memory
    ("bf16", 3, 64, 64, (8193, 50), 1000, 64),
    ("bf16", 2, 64, 32, (9000, 16384, 8192), 4097, 0),
    ("fp4", 3, 128, 64, (20000, 12345), 8191, 1000),
    ("fp4", 2, 64, 16, (32768,), 32767, 1),
    ("bf16", 3, 64, 64, (40000, 33000), 9999, 9999),
    ("fp8", 2, 128, 64, (65536, 40001), 30000, 17),
    ("bf16", 3, 64, 64, (70000, 66000), 20001, 999),
    ("fp4", 2, 64, 64, (140000, 100), 9000, 4000),
]


@pytest.mark.parametrize("case", range(len(EVICT)))
@pytest.mark.parametrize("dst", ["other", "none", "same"])
def test_long_evictions(case, dst):
    kind, hk, d, b, sk, budget, recent = EVICT[case]
    g = torch.Generator(device="cuda").manual_seed(460 + case)
    n, keep = len(sk), [min(k, budget) for k in sk]
    nblk, kblk = [-(-k // b) for k in sk], [-(-k // b) for k in keep]
    blocks = sum(nblk) + sum(kblk) + 1
    shape = ua.cache_shape(blocks, hk, d, b, DT[kind])
    k = torch.randint(0, 256, shape + ((2,) if kind == "bf16" else ()), generator=g, device="cuda", dtype=torch.uint8)
    k = k.view(torch.bfloat16).squeeze(-1) if kind == "bf16" else k
    v = k.flip(0).clone()
    k0, v0 = k.clone(), v.clone()
    ids = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)
    width = max(nblk) + 2
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    to = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    off = 0
    for s in range(n):
        table[s, :nblk[s]] = ids[off:off + nblk[s]]
        to[s, :kblk[s]] = ids[off + nblk[s]:off + nblk[s] + kblk[s]]
        off += nblk[s] + kblk[s]
    if dst != "other":
        to = table
    w = evict_weights(np.random.default_rng(470 + case), (n, hk, max(sk) + 5))
    dw = torch.from_numpy(w).cuda()
    dwo = dw if dst == "none" else torch.full_like(dw, 5.0)
    before = dwo.clone()
    kept = torch.full((n, hk, budget), 99, dtype=torch.int32, device="cuda")
    used = torch.tensor(sk, dtype=torch.int32, device="cuda")
    p = ua.Problem(hk, hk, d, b, blocks, n, width, 1, ua.UA_FLAG_CAUSAL, 0.1, kv_dtype=DT[kind])
    p.cache_evict(k, v, table, used, n, max(sk), dw, dwo, budget, recent, kept, used,
                  dst_block_table=None if dst == "none" else to)
    assert p.check_device_error() == 0 and used.tolist() == keep
    assert p.last_path() == ("evict" if dst == "other" else "evict_in_place")

    def rows(cache, tab, s, h, pos):
        """The stored bytes of key positions pos."""
        blk, slot = tab[s, pos // b].long(), pos % b
        if kind != "fp4":
            return cache[blk, slot, h].view(torch.uint8)
        c, e = b * d // 2, torch.arange(d // 2, device="cuda")
        codes = cache[blk[:, None], h, slot[:, None] * (d // 2) + e]
        return torch.cat([codes, cache[blk[:, None], h, c + slot[:, None] * (d // 16) + e[:d // 16]]], 1)

    for s in range(n):
        for h in range(hk):
            want = torch.from_numpy(R.evict_choice(w[s, h], sk[s], budget, recent)).cuda()
            m = len(want)
            assert torch.equal(kept[s, h, :m].long(), want) and bool((kept[s, h, m:] == -1).all())
            np.testing.assert_array_equal(dwo[s, h, :m].cpu().numpy(), w[s, h][want.cpu().numpy()])
            assert torch.equal(dwo[s, h, m:].view(torch.int32), before[s, h, m:].view(torch.int32))
            r = torch.arange(m, device="cuda")
            for now, old in ((k, k0), (v, v0)):
                assert torch.equal(rows(now, to, s, h, r), rows(old, table, s, h, want))
    # Blocks that no kept key went to are as they were.
    touched = torch.zeros(blocks, dtype=torch.bool, device="cuda")
    for s in range(n):
        touched[to[s, :kblk[s]].long()] = True
    for now, old in ((k, k0), (v, v0)):
        assert torch.equal(now[~touched].view(torch.uint8), old[~touched].view(torch.uint8))


def test_scores_past_2_to_the_31():
    """A prompt chunk whose stored scores are more elements than 32 bits count."""
    sq, sk, hq = 1000, 140000, 16
    bt = LongBatch(490, "bf16", hq, 4, 64, 64, (sq,), (sk,))
    assert sq * hq * sk > 1 << 31
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    w = torch.full((1, 4, sk), -7.0, device="cuda")
    out = p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, None, w)
    assert p.check_device_error() == 0
    ref = bt.reference(0)
    check(bt, 0, out, ref, bf16_p=True)
    check_weights(bt, 0, w[0], torch.zeros_like(ref[3]), ref)
