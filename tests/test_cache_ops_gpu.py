"""The cache operators on the GPU (store, expand, attention over a 4-bit cache,
attention with key weights, eviction) against the plain 64-bit implementations
of tests/cache_ref.py, through the C ABI.

Tolerances.  With dx the score error bound of ``score_error`` (natural units), a
softmax weight w is off by at most w * (2 dx + 2^-18) (numerator and
denominator each move by e^dx; the base-2 exponentials, their sum over a few
thousand keys and log2 add less than 2^-18), and a row's output by
    2^-8 |o|                     the final rounding to bf16 (half a step)
  + (2 dx + 2^-10 + 2^-8 [bf16 P]) * sum w |v|
                                 weights; P in the MMA's f16 (2^-11) or bf16
                                 (2^-8) operand.
The prefill kernels' and bf16 partials' further roundings are covered by 2^-7
more where they take part.
Stored bytes, moved rows, kept positions and lengths are compared exactly."""
import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import cache_ref as R

pytestmark = pytest.mark.gpu

DT = {"bf16": ua.UA_DTYPE_BF16, "fp8": ua.UA_DTYPE_FP8_E4M3, "fp4": ua.UA_DTYPE_FP4_E2M1}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_varlen_flash_gb300 import build
    build.build()
    ua.load_library()


def bits(x):
    """float64 -> (bf16 bit patterns, their float64 values)."""
    t = torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)
    return t.view(torch.int16).numpy().view(np.uint16), t.float().numpy().astype(np.float64)


def to_gpu(c):
    """A reference cache's bytes as the device tensor the library reads."""
    if c.kind == "bf16":
        return torch.from_numpy(c.raw.view(np.int16).copy()).cuda().view(torch.bfloat16)
    return torch.from_numpy(c.raw.copy()).cuda()


def raw_of(t, kind):
    if kind == "bf16":
        return t.view(torch.int16).cpu().numpy().view(np.uint16)
    return t.cpu().numpy()


class Batch:
    """Seeded lengths, tables and values of one ragged batch; the K/V rows of
    every key are in ``k`` / ``v`` (bf16-valued float64 [S_k, H_k, d] per
    sequence), and cached in ``kc`` / ``vc`` up to ``upto``[s] keys."""

    def __init__(self, seed, kind="fp4", hq=8, hk=2, d=128, b=16, sq=(1,), sk=(40,), kscale=1.0, vscale=1.0,
                 scale=None, spare=4, std=1.0, store=True):
        g = self.rng = np.random.default_rng(seed)
        self.kind, self.hq, self.hk, self.d, self.b = kind, hq, hk, d, b
        self.sq, self.sk, self.n = list(sq), list(sk), len(sk)
        self.kscale, self.vscale = (kscale, vscale) if kind != "bf16" else (1.0, 1.0)
        self.scale = scale or d ** -0.5
        nblk = [-(-k // b) for k in sk]
        self.width = max(max(nblk), 1) + 1
        self.blocks = sum(nblk) + spare
        perm = g.permutation(self.blocks)
        self.table = np.full((self.n, self.width), -1, np.int32)
        off = 0
        for s in range(self.n):
            self.table[s, :nblk[s]] = perm[off:off + nblk[s]]
            off += nblk[s]
        self.spare_ids = perm[off:]
        # Slots no key uses: NaN (bf16), the NaN code (fp8), NaN scales (fp4).
        poison = 0x7fc0 if kind == "bf16" else 0x7f
        self.kc = R.Cache(kind, self.blocks, b, hk, d, kscale, poison)
        self.vc = R.Cache(kind, self.blocks, b, hk, d, vscale, poison)
        self.qb, self.q = bits(g.normal(size=(sum(sq), hq, d)))
        self.k, self.v, self.kb, self.vb = [], [], [], []
        for s in range(self.n):
            for vals, raw in ((self.k, self.kb), (self.v, self.vb)):
                rb, rv = bits(std * g.normal(size=(sk[s], hk, d)))
                vals.append(rv)
                raw.append(rb)
        if store:
            for s in range(self.n):
                for j in range(self.sk[s]):
                    self.put(s, j)
        self.cu = np.concatenate([[0], np.cumsum(sq)]).astype(np.int32)
        self.flags_kw = {}

    def put(self, s, j):
        at = int(self.table[s, j // self.b]), j % self.b
        self.kc.put(*at, self.k[s][j], self.kb[s][j])
        self.vc.put(*at, self.v[s][j], self.vb[s][j])

    def problem(self, flags=ua.UA_FLAG_CAUSAL, max_total_q=None, softcap=0.0, window=0, **kw):
        return ua.Problem(self.hq, self.hk, self.d, self.b, self.blocks, self.n, self.width,
                          max_total_q or max(1, sum(self.sq)), flags, self.scale, softcap, window,
                          kv_dtype=DT[self.kind], k_scale=self.kscale, v_scale=self.vscale, **kw)

    def device(self):
        self.d_table = torch.from_numpy(self.table).cuda()
        self.d_cu = torch.from_numpy(self.cu).cuda()
        self.d_sk = torch.tensor(self.sk, dtype=torch.int32, device="cuda")
        self.d_q = torch.from_numpy(self.qb.view(np.int16)).cuda().view(torch.bfloat16)
        self.d_k, self.d_v = to_gpu(self.kc), to_gpu(self.vc)
        return self

    def args(self):
        return (self.d_q, self.d_k, self.d_v, self.d_table, self.d_cu, self.d_sk, self.n, sum(self.sq),
                max(self.sq), max(self.sk))

    def new_rows(self, which):
        """The chunk's rows of every sequence, packed bf16 [total_q, H_k, d]."""
        raw = np.concatenate([(self.kb if which == "k" else self.vb)[s][self.sk[s] - self.sq[s]:]
                              for s in range(self.n)])
        return torch.from_numpy(raw.view(np.int16).copy()).cuda().view(torch.bfloat16)

    def reference(self, s, **kw):
        a, z = R.tokens_of(self.cu, s)
        return R.attention(self.q[a:z], self.kc.rows(self.table[s], self.sk[s]),
                           self.vc.rows(self.table[s], self.sk[s]), self.scale, **kw)


def terms(hq, softcap=0.0, window=0, sinks=False, alibi=False, causal=True, seed=5):
    """(flags, softcap, window, sinks array or None, slopes or None)."""
    g = np.random.default_rng(seed)
    sk = g.normal(size=hq).astype(np.float32) if sinks else None
    al = np.array([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], np.float32) if alibi else None
    return ua.flags_of(causal, softcap, alibi, window, sinks), softcap, window, sk, al


def on_gpu(x):
    return None if x is None else torch.from_numpy(x).cuda()


def check_out(bt, got, s, o, a, mag, softcap=0.0, extra=0.0, bf16_p=False):
    lo, hi = R.tokens_of(bt.cu, s)
    dx = R.score_error(mag, bt.d, softcap, extra)
    per = 2 * dx + 2.0 ** -10 + (2.0 ** -7 + 2.0 ** -8 if bf16_p else 0.0)
    err = np.abs(got[lo:hi] - o)
    bound = 2.0 ** -8 * np.abs(o) + per * a + 1e-30
    assert np.all(np.isfinite(got[lo:hi]))
    assert np.all(err <= bound), (s, float((err / bound).max()))


def check_weights(got, want, fresh, mag, d, n_rows, softcap=0.0, extra=0.0):
    """want = decayed old + fresh (float64); fp32 sums of n_rows weights."""
    dx = R.score_error(mag, d, softcap, extra)
    bound = fresh * (2 * dx + 2.0 ** -18 + (n_rows + 4) * 2.0 ** -24) + np.abs(want) * 2.0 ** -22 + 1e-30
    assert np.all(np.abs(got - want) <= bound), float((np.abs(got - want) / bound).max())


# ---------------------------------------------------------------- store, expand
STORE = [
    # (kind, hq, hk, d, b, S_q, S_k, k_scale, v_scale)
    ("fp4", 8, 2, 128, 16, (1, 40, 0, 17), (33, 40, 20, 17), 1.0, 0.5),
    ("fp4", 4, 4, 64, 32, (5, 1, 70), (5, 64, 200), 0.05, 3.0),
    ("fp4", 2, 1, 256, 64, (1, 65), (1, 130), 0.25, 1.0),
    ("fp8", 8, 2, 128, 16, (9, 1), (30, 16), 1 / 32, 0.03),
    ("bf16", 6, 3, 64, 16, (20, 1), (20, 49), 1.0, 1.0),
]


@pytest.mark.parametrize("case", range(len(STORE)))
def test_store_writes_the_reference_bytes(case):
    kind, hq, hk, d, b, sq, sk, ks, vs = STORE[case]
    bt = Batch(10 + case, kind, hq, hk, d, b, sq, sk, ks, vs, store=False)
    # Values the rounding can go wrong at, in the first new row of sequence 0.
    for vals, raw in ((bt.k, bt.kb), (bt.v, bt.vb)):
        row = vals[0][sk[0] - sq[0]]
        row[0, :16] = [6.0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, -.25, -5, .2, .3, 0, -0.0, 4.9, 5.1]
        row[0, 16:32] = 0
        row[0, 32] = np.inf
        row[0, 33] = -np.inf
        row[-1, 48] = np.nan
        row[-1, :16] *= 1e-4
        row[-1, 16:32] *= 1e6
        rb, rv = bits(row)
        raw[0][sk[0] - sq[0]], vals[0][sk[0] - sq[0]] = rb, rv
    bt.device()
    for s in range(bt.n):
        for j in range(sk[s] - sq[s], sk[s]):
            bt.put(s, j)
    p = bt.problem()
    # A slice of a fused projection: tokens strided, both in one tensor.
    total = sum(sq)
    fused = torch.zeros(total, 2 * hk + 1, d, dtype=torch.bfloat16, device="cuda")
    fused[:, :hk], fused[:, hk:2 * hk] = bt.new_rows("k"), bt.new_rows("v")
    p.cache_store(fused[:, :hk], fused[:, hk:2 * hk], bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, bt.n, total,
                  max(sq), max(sk))
    assert p.check_device_error() == 0 and p.last_launch_count() == 1
    np.testing.assert_array_equal(raw_of(bt.d_k, kind), bt.kc.raw)
    np.testing.assert_array_equal(raw_of(bt.d_v, kind), bt.vc.raw)


@pytest.mark.parametrize("kind,d,b,ks", [("fp4", 64, 16, 1.0), ("fp4", 128, 32, 0.05), ("fp4", 256, 64, 0.5),
                                         ("fp8", 128, 16, 1 / 32), ("bf16", 128, 16, 1.0)])
def test_expand_writes_the_values_once_rounded(kind, d, b, ks):
    bt = Batch(30, kind, 4, 2, d, b, (1, 1, 1, 1), (75, 1, 2 * b, 40), ks, ks)
    begin = np.array([0, 1, b + 3, 17], np.int32)
    p = bt.device().problem()
    out = [torch.full((bt.blocks + 2, b, 2, d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = np.full((4, bt.width + 3), -1, np.int32)
    perm = bt.rng.permutation(bt.blocks + 2)
    off = 0
    for s in range(4):
        for blk in range(begin[s] // b, -(-bt.sk[s] // b)):
            table[s, blk] = perm[off]
            off += 1
    p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 4, 75, out[0], out[1], torch.from_numpy(table).cuda(),
                   begin=torch.from_numpy(begin).cuda())
    assert p.check_device_error() == 0
    for c, o in ((bt.kc, out[0]), (bt.vc, out[1])):
        want = np.full((bt.blocks + 2, b, 2, d), 7.0)
        for s in range(4):
            rows = c.rows(bt.table[s], bt.sk[s])
            for j in range(begin[s], bt.sk[s]):
                want[table[s, j // b], j % b] = rows[j]
        want32 = want.astype(np.float32)
        if ks == 0.05:   # code * scale is exact, the fp32 product with 0.05 rounds before the bf16 rounding
            assert np.all(np.abs(o.double().cpu().numpy() - want) <= np.abs(want) * (2.0 ** -8 + 2.0 ** -23))
        else:
            np.testing.assert_array_equal(o.cpu().view(torch.int16).numpy(),
                                          torch.from_numpy(want32).to(torch.bfloat16).view(torch.int16).numpy())


def test_store_then_expand_without_begin_feeds_a_prefill():
    """A 4-bit cache expanded to bf16 pages and read by the prefill kernels
    gives what the 4-bit kernel gives on the cache itself."""
    sq, sk = (70, 33, 9), (70, 90, 40)
    bt = Batch(40, "fp4", 8, 2, 128, 32, sq, sk, 0.5, 2.0).device()
    p = bt.problem()
    pages = [torch.zeros(bt.blocks, 32, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 3, 90, pages[0], pages[1], bt.d_table)
    p16 = ua.Problem(8, 2, 128, 32, bt.blocks, 3, bt.width, 200, ua.UA_FLAG_CAUSAL, bt.scale)
    a = bt.args()
    got16 = p16.forward(a[0], pages[0], pages[1], *a[3:], ua.UA_FLAG_CAUSAL)
    got4 = p.forward(*a, ua.UA_FLAG_CAUSAL)
    assert p.check_device_error() == 0 and p16.check_device_error() == 0
    for s in range(3):
        o, ab, _, mag = bt.reference(s)
        check_out(bt, got4.double().cpu().numpy(), s, o, ab, mag)
        check_out(bt, got16.double().cpu().numpy(), s, o, ab, mag, bf16_p=True)


# ---------------------------------------------------------------- attention over 4 bits
ATTEND = [
    # (hq, hk, d, b, S_q, S_k, terms)
    (8, 2, 128, 16, (1, 1, 1, 1), (1, 31, 32, 700), {}),
    (8, 2, 128, 32, (1, 3, 0, 2), (16, 100, 50, 513), dict(softcap=20.0, window=40, sinks=True)),
    (8, 8, 64, 16, (1, 9, 1), (65, 129, 1), dict(alibi=True)),
    (16, 1, 128, 64, (1, 2, 5), (900, 64, 5), dict(window=1)),
    (16, 2, 256, 64, (1, 1, 3), (300, 129, 65), dict(sinks=True)),
    (32, 1, 64, 32, (1, 2), (70, 33), dict(softcap=5.0)),
    (6, 2, 128, 16, (7, 20), (7, 150), {}),
    (5, 5, 256, 16, (1, 30), (40, 31), dict(window=9, alibi=True, sinks=True)),
    (8, 2, 64, 64, (2, 2), (300, 2), dict(causal=False)),
    (12, 4, 128, 16, (1,), (5000,), {}),
    (16, 2, 256, 64, (20, 1, 37), (150, 700, 37), {}),
    (16, 2, 256, 16, (9,), (1400,), dict(softcap=30.0, window=300, sinks=True)),
    (4, 4, 64, 32, (200, 0, 129), (300, 7, 129), dict(alibi=True, sinks=True)),
    (8, 2, 128, 16, (300, 33), (300, 900), dict(window=70)),
    (10, 2, 128, 64, (64, 26), (1300, 26), dict(softcap=10.0)),
    (8, 1, 128, 32, (17, 6), (2100, 129), dict(causal=False)),
]


@pytest.mark.parametrize("case", range(len(ATTEND)))
@pytest.mark.parametrize("partials", [ua.UA_PARTIALS_F32, ua.UA_PARTIALS_BF16])
def test_attention_over_4_bits(case, partials):
    hq, hk, d, b, sq, sk, kw = ATTEND[case]
    bt = Batch(60 + case, "fp4", hq, hk, d, b, sq, sk, 0.5, 2.0).device()
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    p = bt.problem(flags, softcap=softcap, window=window, split_partials=partials)
    out = torch.full_like(bt.d_q, 3.0)
    got = p.forward(*bt.args(), flags, on_gpu(sinks), on_gpu(alibi), out=out).double().cpu().numpy()
    assert p.check_device_error() == 0 and p.last_path().startswith("fp4")
    extra = max(sk) if alibi is not None else 0.0
    for s in range(bt.n):
        if not sq[s]:
            continue
        o, a, _, mag = bt.reference(s, causal=kw.get("causal", True), softcap=softcap, window=window, sinks=sinks,
                                    alibi=alibi)
        check_out(bt, got, s, o, a, mag, softcap, extra, bf16_p=partials == ua.UA_PARTIALS_BF16)


@pytest.mark.parametrize("nq", [1, 20])
def test_query_magnitudes_far_outside_f16(nq):
    bt = Batch(80, "fp4", 4, 2, 128, 16, (nq, nq), (100, 37))
    bt.q[:nq] *= 2.0 ** 60
    bt.q[nq:] *= 2.0 ** -70
    bt.qb, bt.q = bits(bt.q)
    bt.scale = 2.0 ** -62
    p = bt.device().problem()
    got = p.forward(*bt.args(), ua.UA_FLAG_CAUSAL).double().cpu().numpy()
    for s in range(2):
        o, a, _, mag = bt.reference(s)
        check_out(bt, got, s, o, a, mag)


def test_4bit_rows_without_keys_and_infinite_sinks():
    bt = Batch(81, "fp4", 4, 2, 128, 16, (1, 1, 1), (20, 5, 40)).device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_SINKS
    sinks = np.array([np.inf, -np.inf, 0.0, 80.0], np.float32)
    p = bt.problem(flags)
    got = p.forward(*bt.args(), flags, on_gpu(sinks)).double().cpu().numpy()
    assert np.all(got[:, 0] == 0)
    for s in range(3):
        o, a, _, mag = bt.reference(s, sinks=sinks.astype(np.float64))
        check_out(bt, got, s, o, a, mag)


@pytest.mark.parametrize("nq", [1, 10])
def test_nan_in_places_no_row_sees_stays_out(nq):
    """NaN keys before every row's window, and after the end, reach nothing."""
    bt = Batch(82, "fp4", 8, 2, 128, 64, (nq, nq), (100, 130))
    for s, upto in ((0, 61 - nq), (1, 91 - nq)):
        for j in range(upto):
            blk = int(bt.table[s, j // 64])
            n = 64 * 64
            for c in (bt.kc, bt.vc):
                c.raw[blk, :, n + (j % 64) * 8:n + (j % 64 + 1) * 8] = 0x7f
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_WINDOW
    p = bt.device().problem(flags, window=40)
    got = p.forward(*bt.args(), flags).double().cpu().numpy()
    for s in range(2):
        keys, vals = (c.rows(bt.table[s], bt.sk[s]) for c in (bt.kc, bt.vc))
        lo = bt.sk[s] - 39 - nq
        o, a, _, mag = R.attention(bt.q[s * nq:(s + 1) * nq], keys[lo:], vals[lo:], bt.scale, window=40)
        check_out(bt, got, s, o, a, mag)


@pytest.mark.parametrize("d,b,hq,hk,sq,sk,window", [
    (128, 16, 8, 2, (3, 2), (40, 130), 0), (64, 32, 4, 4, (6, 1), (70, 33), 0), (64, 16, 4, 4, (8, 8), (8, 500), 5),
    (256, 64, 16, 2, (2, 2), (100, 65), 20), (128, 16, 8, 2, (40, 33), (40, 1500), 0),
    (256, 64, 4, 2, (90, 20), (200, 150), 30), (64, 32, 8, 1, (70, 9), (70, 300), 0),
    (128, 64, 2, 2, (200, 150), (900, 150), 100)])
def test_nan_values_reach_only_the_rows_that_see_them(d, b, hq, hk, sq, sk, window):
    """NaN in V at keys that the masks hide from some rows of a tile."""
    bt = Batch(90, "fp4", hq, hk, d, b, sq, sk)
    marks = []
    for s in range(2):
        ctx = sk[s] - sq[s]
        for j in {sk[s] - 1, ctx + sq[s] // 2, max(0, ctx - window + 2) if window else sk[s] - 1}:
            h, grp = int(bt.rng.integers(hk)), int(bt.rng.integers(d // 16))
            bt.vc.raw[int(bt.table[s, j // b]), h, b * (d // 2) + (j % b) * (d // 16) + grp] = 0x7f
            marks.append((s, j, h, grp))
    flags = ua.UA_FLAG_CAUSAL | (ua.UA_FLAG_WINDOW if window else 0)
    p = bt.device().problem(flags | ua.UA_FLAG_KEY_WEIGHTS, window=window)
    got = p.forward(*bt.args(), flags).double().cpu().numpy()
    w = torch.zeros(2, hk, max(sk), device="cuda")
    again = p.forward_weights(*bt.args(), flags, None, w).double().cpu().numpy()
    assert p.check_device_error() == 0 and bool(torch.isfinite(w).all())
    for s in range(2):
        nan = np.zeros((sq[s], hk, d), bool)
        for t, j, h, grp in marks:
            pos = np.arange(sq[s]) + sk[s] - sq[s]
            see = (j <= pos) & ((j > pos - window) if window else True)
            if t == s:
                nan[see, h, 16 * grp:16 * grp + 16] = True
        nan = np.repeat(nan, hq // hk, 1)
        lo, hi = R.tokens_of(bt.cu, s)
        keys, vals = (c.rows(bt.table[s], sk[s]) for c in (bt.kc, bt.vc))
        o, a, _, mag = R.attention(bt.q[lo:hi], keys, np.nan_to_num(vals), bt.scale, window=window)
        for x in (got, again):
            np.testing.assert_array_equal(np.isnan(x[lo:hi]), nan)
            x[lo:hi][nan] = o[nan]
            check_out(bt, x, s, o, a, mag)


@pytest.mark.parametrize("kind,d,sq,sk", [("fp4", 128, (1, 2), (1, 40)), ("fp4", 64, (1, 3), (900, 300)),
                                          ("fp4", 128, (40, 30), (40, 2000)), ("fp4", 256, (1, 26), (33, 700)),
                                          ("bf16", 128, (1, 2), (1, 1500)), ("bf16", 64, (4, 1), (4, 40)),
                                          ("fp8", 128, (1, 3), (300, 3))])
def test_nan_keys_make_the_rows_that_see_them_nan(kind, d, sq, sk):
    """A NaN key (the chunk's last, of one KV head) and a segment of nothing but
    NaN keys: the rows that see one, and their weights, are NaN; others are not."""
    bt = Batch(95, kind, 4, 2, d, 16, sq, sk)
    for s, js in ((0, [sk[0] - 1]), (1, range(0, min(256, sk[1])))):
        for j in js:
            blk, slot = int(bt.table[s, j // 16]), j % 16
            if kind == "fp4":
                bt.kc.raw[blk, 1, 16 * (d // 2) + slot * (d // 16):][:d // 16] = 0x7f
            else:
                bt.kc.raw[blk, slot, 1] = 0x7fc0 if kind == "bf16" else 0x7f
    bt.device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    w = torch.zeros(2, 2, max(sk), device="cuda")
    out = p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, None, w).float().cpu().numpy()
    if kind == "fp4":
        same = p.forward(*bt.args(), ua.UA_FLAG_CAUSAL).float().cpu().numpy()
        np.testing.assert_array_equal(np.isnan(same), np.isnan(out))
    assert p.check_device_error() == 0
    nan = np.zeros(out.shape, bool)
    nan[sq[0] - 1, 2:] = True
    nan[sq[0]:, 2:] = True
    np.testing.assert_array_equal(np.isnan(out), nan)
    w = w.cpu().numpy()
    for s in range(2):
        assert np.isfinite(w[s, 0]).all() and np.isnan(w[s, 1, :sk[s]]).all() and np.isfinite(w[s, 1, sk[s]:]).all()


def test_4bit_batch_of_more_sequences_than_one_scan_covers():
    """1,300 short sequences, some empty, some malformed: the work split takes three rounds."""
    g = np.random.default_rng(91)
    n = 1300
    sk = [int(x) for x in g.integers(1, 70, n)]
    sq = [int(x) for x in np.minimum(sk, g.integers(0, 3, n))]
    bt = Batch(92, "fp4", 4, 2, 64, 16, sq, sk, store=False)
    for s in range(0, n, 37):
        for j in range(sk[s]):
            bt.put(s, j)
    bt.device()
    bad = [600, 1299]
    for s in bad:
        bt.d_sk[s] = 1000
    p = bt.problem()
    # Sequences that were not filled hold NaN scales: only the checked ones are finite.
    out = torch.full_like(bt.d_q, 5.0)
    got = p.forward(*bt.args(), ua.UA_FLAG_CAUSAL, out=out).double().cpu().numpy()
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS
    for s in range(n):
        lo, hi = R.tokens_of(bt.cu, s)
        if s in bad:
            assert np.all(got[lo:hi] == 0)
        elif s % 37 == 0 and sq[s]:
            o, a, _, mag = bt.reference(s)
            check_out(bt, got, s, o, a, mag)
        elif sq[s]:
            assert np.all(np.isnan(got[lo:hi]))


def test_two_problems_on_two_streams_do_not_touch_each_other():
    a = Batch(93, "fp4", 8, 2, 128, 16, (1,) * 8, (900, 20, 300, 1, 64, 512, 33, 700)).device()
    c = Batch(94, "fp4", 8, 2, 128, 16, (20,) * 3, (700, 20, 100)).device()
    probs = [bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS) for bt in (a, c)]
    ws = [torch.zeros(bt.n, 2, max(bt.sk), device="cuda") for bt in (a, c)]
    outs = [torch.empty_like(bt.d_q) for bt in (a, c)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, bt, w, o, st in zip(probs, (a, c), ws, outs, streams):
            p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, None, w, out=o, stream=st)
    torch.cuda.synchronize()
    for p, bt, w, o in zip(probs, (a, c), ws, outs):
        assert p.check_device_error() == 0
        got, gw = o.double().cpu().numpy(), w.double().cpu().numpy()
        for s in range(bt.n):
            want, ab, weights, mag = bt.reference(s)
            check_out(bt, got, s, want, ab, mag)
            fresh = weights.reshape(2, 4, bt.sq[s], bt.sk[s]).sum((1, 2))
            check_weights(gw[s, :, :bt.sk[s]], fresh, fresh, mag, bt.d, 4 * bt.sq[s])


@pytest.mark.parametrize("g,sq", [(4, (3, 20)), (4, (3, 4)), (1, (3, 2)), (2, (50, 17))])
def test_4bit_qq_bias(g, sq):
    bt = Batch(83, "fp4", 2 * g, 2, 128, 16, sq, (90, 20)).device()
    flags = ua.UA_FLAG_CAUSAL | ua.UA_FLAG_QQ_BIAS
    qq = bt.rng.normal(size=(max(sq), max(sq) + 4)).astype(np.float32)
    p = bt.problem(flags)
    p.set_qq_bias(torch.from_numpy(qq).cuda())
    got = p.forward(*bt.args(), flags).double().cpu().numpy()
    for s in range(2):
        o, a, _, mag = bt.reference(s, qq=qq.astype(np.float64))
        check_out(bt, got, s, o, a, mag, extra=5.0)


@pytest.mark.parametrize("nq", [1, 40])
def test_4bit_bad_blocks_and_lengths_are_reported(nq):
    bt = Batch(84, "fp4", 4, 2, 128, 16, (nq, nq, nq), (40, 40, 40))
    bt.table[0, 1] = bt.blocks + 9
    p = bt.device().problem()
    bt.d_sk[2] = 0                                  # S_k < S_q
    got = p.forward(*bt.args(), ua.UA_FLAG_CAUSAL).double().cpu().numpy()
    assert p.check_device_error() == ua.UA_DEVERR_BLOCK_ID | ua.UA_DEVERR_CONTEXT
    assert np.all(got[2 * nq:] == 0) and np.all(np.isfinite(got))
    # The bad block's keys read as zeros.
    keys, vals = [np.zeros((40, 2, 128)) for _ in range(2)]
    for j in list(range(16)) + list(range(32, 40)):
        keys[j] = bt.kc.row(int(bt.table[0, j // 16]), j % 16)
        vals[j] = bt.vc.row(int(bt.table[0, j // 16]), j % 16)
    o, a, _, mag = R.attention(bt.q[:nq], keys, vals, bt.scale)
    check_out(bt, got, 0, o, a, mag)
    o, a, _, mag = bt.reference(1)
    check_out(bt, got, 1, o, a, mag)


@pytest.mark.parametrize("sq", [(1, 1), (40, 9)])
def test_4bit_bounded_wait_gives_up_and_recovers(sq):
    bt = Batch(85, "fp4", 8, 2, 128, 16, sq, (600, 300)).device()
    p = bt.problem()
    assert ua.binding.ua_debug_stall_data_waits(p.handle, 1) == 0
    p.forward(*bt.args(), ua.UA_FLAG_CAUSAL)
    assert p.check_device_error() == ua.UA_DEVERR_TIMEOUT
    assert ua.binding.ua_debug_stall_data_waits(p.handle, 0) == 0
    got = p.forward(*bt.args(), ua.UA_FLAG_CAUSAL).double().cpu().numpy()
    assert p.check_device_error() == 0
    for s in range(2):
        o, a, _, mag = bt.reference(s)
        check_out(bt, got, s, o, a, mag)


def test_4bit_cache_past_4_gib():
    """Offsets into a cache of more than 2^32 bytes."""
    hk, d, b = 8, 256, 64
    page = b * (d // 2 + d // 16)
    blocks = (1 << 32) // (hk * page) + 40
    bt = Batch(86, "fp4", 8, 8, d, b, (1,), (70,))
    k = torch.full((blocks, hk, page), 0x7f, dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, 0x7f)
    table = np.array([[blocks - 1, blocks - 30, -1]], np.int32)
    bt.device()
    for i in range(2):
        k[int(table[0, i])] = bt.d_k[int(bt.table[0, i])]
        v[int(table[0, i])] = bt.d_v[int(bt.table[0, i])]
    p = ua.Problem(8, 8, d, b, blocks, 1, 3, 1, ua.UA_FLAG_CAUSAL, bt.scale, kv_dtype=DT["fp4"])
    a = bt.args()
    got = p.forward(a[0], k, v, torch.from_numpy(table).cuda(), *a[4:], ua.UA_FLAG_CAUSAL)
    o, ab, _, mag = bt.reference(0)
    check_out(bt, got.double().cpu().numpy(), 0, o, ab, mag)


# ---------------------------------------------------------------- key weights
WEIGHTS = [
    # (kind, hq, hk, d, b, S_q, S_k, decay, terms)
    ("bf16", 8, 2, 128, 16, (1, 1, 1), (1, 300, 129), 1.0, {}),
    ("bf16", 8, 2, 64, 32, (3, 9, 0, 20), (130, 9, 30, 50), 0.5, dict(softcap=20.0, window=30, sinks=True)),
    ("bf16", 6, 2, 256, 64, (1, 12), (200, 140), 0.0, dict(alibi=True)),
    ("bf16", 16, 1, 128, 16, (2, 1), (1500, 77), 1.0, dict(sinks=True)),
    ("fp8", 8, 1, 128, 32, (1, 5), (400, 133), 0.9, {}),
    ("fp4", 8, 2, 128, 16, (1, 1, 1), (1, 300, 1100), 1.0, {}),
    ("fp4", 8, 8, 64, 32, (4, 0, 21), (130, 12, 50), 0.5, dict(softcap=20.0, window=30, sinks=True)),
    ("fp4", 16, 1, 256, 64, (2, 3), (200, 3), 0.0, dict(alibi=True)),
    ("fp4", 40, 2, 128, 16, (1, 2), (90, 33), 1.0, {}),
    ("bf16", 8, 2, 128, 16, (2, 2), (60, 2), 1.0, dict(causal=False)),
    ("fp4", 8, 2, 128, 32, (32, 8, 0, 33), (700, 8, 5, 140), 0.9, {}),
    ("fp4", 16, 2, 256, 16, (10, 5), (300, 130), 1.0, dict(window=40, sinks=True)),
    ("fp4", 4, 2, 64, 64, (140, 1), (140, 260), 0.0, dict(softcap=20.0, alibi=True)),
]


def weights_reference(bt, w_in, decay, **kw):
    """(want, fresh, mag) [n, H_k, max S_k]; NaN where nothing is written."""
    n, hk, g = bt.n, bt.hk, bt.hq // bt.hk
    want = np.full((n, hk, max(bt.sk)), np.nan)
    fresh, mags = np.zeros_like(want), 0.0
    for s in range(n):
        if not bt.sq[s]:
            continue
        _, _, w, mag = bt.reference(s, **kw)
        mags = max(mags, mag)
        sk = bt.sk[s]
        fresh[s, :, :sk] = w.reshape(hk, g, bt.sq[s], sk).sum((1, 2))
        old = np.zeros((hk, sk))
        if w_in is not None and decay:
            old = np.where(np.arange(sk) < sk - bt.sq[s], decay * w_in[s, :, :sk].astype(np.float64), 0.0)
        want[s, :, :sk] = old + fresh[s, :, :sk]
    return want, fresh, mags


@pytest.mark.parametrize("case", range(len(WEIGHTS)))
@pytest.mark.parametrize("alias", [False, True])
def test_key_weights(case, alias):
    kind, hq, hk, d, b, sq, sk, decay, kw = WEIGHTS[case]
    bt = Batch(120 + case, kind, hq, hk, d, b, sq, sk, 1 / 32 if kind == "fp8" else 0.5, 1 / 32,
               std=1.0).device()
    flags, softcap, window, sinks, alibi = terms(hq, **kw)
    p = bt.problem(flags | ua.UA_FLAG_KEY_WEIGHTS, softcap=softcap, window=window)
    stride = max(sk) + 5
    w_in = bt.rng.exponential(size=(bt.n, hk, stride)).astype(np.float32)
    for s in range(bt.n):                      # entries that must not be read
        w_in[s, :, sk[s] - sq[s]:] = np.nan
    din = torch.from_numpy(w_in).cuda()
    dout = din if alias else torch.full_like(din, -3.0)
    before = dout.cpu().numpy().copy()
    out = p.forward_weights(*bt.args(), flags, din if decay else (din if alias else None), dout, decay=decay,
                            sinks=on_gpu(sinks), alibi_slopes=on_gpu(alibi))
    assert p.check_device_error() == 0 and p.last_launch_count() == 3
    got, got_o = dout.cpu().numpy(), out.double().cpu().numpy()
    args = dict(causal=kw.get("causal", True), softcap=softcap, window=window, sinks=sinks, alibi=alibi)
    extra = max(sk) if alibi is not None else 0.0
    want, fresh, mag = weights_reference(bt, w_in, decay, **args)
    for s in range(bt.n):
        if not sq[s]:
            np.testing.assert_array_equal(got[s], before[s])
            continue
        np.testing.assert_array_equal(got[s, :, sk[s]:], before[s, :, sk[s]:])
        check_weights(got[s, :, :sk[s]].astype(np.float64), want[s, :, :sk[s]], fresh[s, :, :sk[s]], mag, d,
                      hq // hk * sq[s], softcap, extra)
        o, a, _, m = bt.reference(s, **args)
        check_out(bt, got_o, s, o, a, m, softcap, extra, bf16_p=kind == "bf16")


def test_key_weights_match_plain_forward_and_repeat_bit_for_bit():
    bt = Batch(140, "bf16", 8, 2, 128, 16, (1,) * 6, (2000, 31, 700, 1500, 5, 4000)).device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    w = [torch.zeros(6, 2, 4000, device="cuda") for _ in range(2)]
    for x in w:
        p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, None, x)
    assert torch.equal(w[0], w[1])
    # Each row's weights sum to 1, so each KV head's to g = 4 rows (fp32 terms).
    total = w[0].double().sum(-1).cpu().numpy()
    assert np.all(np.abs(total - 4) <= 4 * (2.0 ** -16))


def test_key_weights_refusals():
    bt = Batch(141, "bf16", 8, 2, 128, 16, (1, 1), (40, 50)).device()
    w = torch.zeros(2, 2, 50, device="cuda")

    def status(p, stride=50, decay=1.0, wo=w, flags=ua.UA_FLAG_CAUSAL):
        out = torch.empty_like(bt.d_q)
        return ua.ua_forward_weights(p.handle, *bt.args(), flags, None, None, None, wo, stride, decay, out)

    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    assert status(p) == 0
    assert status(bt.problem()) == 1                               # no key weights at creation
    assert status(p, stride=49) == 1 and status(p, decay=-0.5) == 1
    assert status(p, decay=float("nan")) == 1 and status(p, wo=None) == 1
    assert status(p, flags=ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS) == 1
    with pytest.raises(ua.UAError):
        p.forward(*bt.args(), ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    forced = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS, path=ua.UA_PATH_SPLIT_KV)
    assert status(forced) == 2
    wide = Batch(142, "bf16", 40, 2, 128, 16, (1,), (20,)).device()
    pw = wide.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS)
    with pytest.raises(ua.UAError) as e:
        pw.forward_weights(*wide.args(), ua.UA_FLAG_CAUSAL, None, torch.zeros(1, 2, 20, device="cuda"))
    assert e.value.status == 2                                     # g = 20 on a bf16 cache
    with pytest.raises(ValueError):
        p.forward_weights(*bt.args(), ua.UA_FLAG_CAUSAL, torch.zeros(2, 2, 60, device="cuda"), w)


# ---------------------------------------------------------------- eviction
EVICT = [
    # (kind, hk, d, b, S_k, budget, recent)
    ("bf16", 2, 64, 16, (50, 10, 40, 0, 41), 40, 7),
    ("bf16", 3, 128, 32, (700, 65, 300), 33, 33),
    ("fp4", 2, 128, 16, (100, 1, 37), 20, 0),
    ("fp4", 1, 64, 64, (300, 129), 100, 5),
    ("fp4", 2, 256, 32, (90, 31), 31, 1),
    ("fp8", 2, 128, 16, (60, 33), 1, 0),
    ("bf16", 1, 256, 16, (2100,), 1500, 64),
    ("bf16", 2, 64, 16, (30, 20), 64, 3),
]


def evict_reference(bt, w, budget, recent, dst):
    n, hk = bt.n, bt.hk
    kept = np.full((n, hk, budget), -1, np.int32)
    w_out = {}
    rows = []
    for s in range(n):
        for h in range(hk):
            idx = R.evict_choice(w[s, h], bt.sk[s], budget, recent)
            kept[s, h, :len(idx)] = idx
            w_out[s, h] = w[s, h, idx]
            for r, j in enumerate(idx):
                src = int(bt.table[s, j // bt.b]), int(j) % bt.b
                to = int(dst[s, r // bt.b]), r % bt.b
                for c in (bt.kc, bt.vc):
                    rows.append((c, to, h, c.row_bytes(*src, h)))
    for c, to, h, data in rows:
        c.set_row_bytes(*to, h, data)
    return kept, w_out


def evict_weights(rng, shape):
    w = rng.exponential(size=shape).astype(np.float32)
    w = np.where(rng.random(shape) < 0.5, np.floor(w * 4) / 4, w).astype(np.float32)
    flat = w.reshape(-1)
    for v in (np.nan, np.inf, -np.inf, -0.0, -1.5, np.float32(3.4e38), np.float32(1e-40)):
        flat[rng.integers(0, flat.size, 4)] = v
    return w


@pytest.mark.parametrize("case", range(len(EVICT)))
@pytest.mark.parametrize("in_place", [False, True])
def test_evict(case, in_place):
    kind, hk, d, b, sk, budget, recent = EVICT[case]
    need = sum(-(-min(k, budget) // b) for k in sk)
    bt = Batch(160 + case, kind, 2 * hk, hk, d, b, (0,) * len(sk), sk, 0.5, 0.5, spare=need + 3).device()
    p = bt.problem()
    stride = max(sk) + 3
    w = evict_weights(bt.rng, (bt.n, hk, stride))
    dw = torch.from_numpy(w).cuda()
    dwo = dw if in_place else torch.full_like(dw, 5.0)
    before = dwo.cpu().numpy().copy()
    dst = bt.table.copy()
    if not in_place:
        dst[:] = -1
        off = 0
        for s in range(bt.n):
            m = -(-min(sk[s], budget) // b)
            dst[s, :m] = bt.spare_ids[off:off + m]
            off += m
    kept = torch.full((bt.n, hk, budget), 99, dtype=torch.int32, device="cuda")
    used = bt.d_sk if in_place else torch.full_like(bt.d_sk, 77)
    p.cache_evict(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, bt.n, max(sk), dw, dwo, budget, recent, kept, used,
                  dst_block_table=None if in_place else torch.from_numpy(dst).cuda())
    assert p.check_device_error() == 0 and p.last_launch_count() == 2
    want_kept, want_w = evict_reference(bt, w, budget, recent, dst)
    np.testing.assert_array_equal(kept.cpu().numpy(), want_kept)
    assert used.cpu().tolist() == [min(k, budget) for k in sk]
    got_w = dwo.cpu().numpy()
    for s in range(bt.n):
        for h in range(hk):
            m = len(want_w[s, h])
            np.testing.assert_array_equal(got_w[s, h, :m], want_w[s, h])
            np.testing.assert_array_equal(got_w[s, h, m:], before[s, h, m:])
    np.testing.assert_array_equal(raw_of(bt.d_k, kind), bt.kc.raw)
    np.testing.assert_array_equal(raw_of(bt.d_v, kind), bt.vc.raw)


def test_evict_long_sequences_of_equal_weights():
    """All weights equal: the oldest candidates stay; 70,000 keys, in place."""
    hk, d, b, sk, budget, recent = 1, 64, 64, 70000, 20001, 999
    blocks = -(-sk // b)
    g = torch.Generator(device="cuda").manual_seed(3)
    k = torch.randint(0, 1 << 15, (blocks, b, hk, d), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16)
    v = k.flip(0).clone()
    k0, v0 = k.clone(), v.clone()
    table = torch.randperm(blocks, generator=g, device="cuda").to(torch.int32)[None]
    p = ua.Problem(hk, hk, d, b, blocks, 1, blocks, 1, ua.UA_FLAG_CAUSAL, 0.1)
    w = torch.full((1, hk, sk), 0.25, device="cuda")
    kept = torch.zeros(1, hk, budget, dtype=torch.int32, device="cuda")
    used = torch.tensor([sk], dtype=torch.int32, device="cuda")
    p.cache_evict(k, v, table, used, 1, sk, w, w, budget, recent, kept, used)
    assert p.check_device_error() == 0 and used.item() == budget
    want = torch.cat([torch.arange(budget - recent), torch.arange(sk - recent, sk)]).cuda()
    assert torch.equal(kept[0, 0].long(), want)
    j = torch.arange(budget, device="cuda")
    for a, a0 in ((k, k0), (v, v0)):
        new = a[table[0, j // b].long(), j % b].view(torch.int16)
        old = a0[table[0, want // b].long(), want % b].view(torch.int16)
        assert torch.equal(new, old)


def test_evict_malformed_lengths_and_blocks():
    bt = Batch(180, "bf16", 4, 2, 64, 16, (0, 0, 0), (40, 40, 40), spare=6)
    bt.table[1, 0] = -1
    p = bt.device().problem()
    bt.d_sk[0] = 41
    w = torch.rand(3, 2, 40, device="cuda")
    wo = torch.full_like(w, 5.0)
    kept = torch.zeros(3, 2, 20, dtype=torch.int32, device="cuda")
    used = torch.zeros(3, dtype=torch.int32, device="cuda")
    dst = torch.full_like(bt.d_table, -1)
    for s in range(3):
        dst[s, :2] = torch.from_numpy(bt.spare_ids[2 * s:2 * s + 2].astype(np.int32))
    dst[2, 1] = bt.blocks
    p.cache_evict(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 3, 40, w, wo, 20, 4, kept, used, dst_block_table=dst)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS | ua.UA_DEVERR_BLOCK_ID
    assert used.tolist() == [0, 20, 20]
    assert torch.all(kept[0] == -1) and torch.all(wo[0] == 5.0)
    wn = w.cpu().numpy()
    for s in (1, 2):
        for h in range(2):
            idx = R.evict_choice(wn[s, h], 40, 20, 4)
            np.testing.assert_array_equal(kept[s, h].cpu().numpy(), idx)
            for r, j in enumerate(idx):
                to = int(dst[s, r // 16])
                if to >= bt.blocks:
                    continue
                want = (bt.kc.row_bytes(int(bt.table[s, j // 16]), j % 16, h) if bt.table[s, j // 16] >= 0
                        else np.full(64, 0x7fc0, np.uint16))
                np.testing.assert_array_equal(raw_of(bt.d_k, "bf16")[to, r % 16, h], want)


def test_store_and_expand_report_bad_metadata():
    bt = Batch(181, "fp4", 4, 2, 128, 16, (2, 2, 2), (20, 20, 20), store=False)
    bt.table[1, 1] = bt.blocks
    p = bt.device().problem()
    bt.d_sk[0] = 1                                   # S_k < S_q: skipped
    kn, vn = bt.new_rows("k"), bt.new_rows("v")
    p.cache_store(kn, vn, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 3, 6, 2, 20)
    assert p.check_device_error() == ua.UA_DEVERR_CONTEXT | ua.UA_DEVERR_BLOCK_ID
    for j in (18, 19):
        bt.put(2, j)
    np.testing.assert_array_equal(raw_of(bt.d_k, "fp4"), bt.kc.raw)
    out = [torch.zeros(bt.blocks, 16, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    begin = torch.tensor([0, 18, 21], dtype=torch.int32, device="cuda")
    p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 3, 5, out[0], out[1], bt.d_table, begin=begin)
    assert p.check_device_error() == ua.UA_DEVERR_BOUNDS | ua.UA_DEVERR_BLOCK_ID
    begin[2] = 2                                     # 18 keys, above the bound of 5
    p.cache_expand(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 3, 5, out[0], out[1], bt.d_table, begin=begin)
    assert p.check_device_error() & ua.UA_DEVERR_BOUNDS
    assert all(not o[bt.d_table[2, 0].long()].any() for o in out)


def test_cache_call_refusals():
    bt = Batch(182, "fp4", 4, 2, 128, 16, (1, 1), (20, 30)).device()
    p = bt.problem()
    kn, vn = bt.new_rows("k"), bt.new_rows("v")

    def store(stride=256, n=2, total=2, mq=1, mk=30, kn=kn):
        return ua.ua_cache_store(p.handle, kn, vn, stride, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, n, total,
                                 mq, mk)

    assert store() == 0 and store(n=0) == 0 and store(total=0) == 0
    assert [store(stride=255), store(stride=260), store(n=3), store(total=3), store(mk=0),
            store(mk=16 * bt.width + 1), store(kn=None), store(kn=kn.data_ptr() + 2)] == [1] * 8

    out = torch.zeros(8, 16, 2, 128, dtype=torch.bfloat16, device="cuda")

    def expand(n=2, keys=30, stride=bt.width, blocks=8, o=out):
        return ua.ua_cache_expand(p.handle, bt.d_k, bt.d_v, bt.d_table, bt.d_sk, None, n, keys, o, out,
                                  torch.zeros_like(bt.d_table), stride, blocks)

    assert expand(n=0) == 0 and expand(keys=0) == 0
    assert [expand(n=3), expand(keys=-1), expand(stride=0), expand(blocks=0), expand(o=None)] == [1] * 5

    w = torch.ones(2, 2, 30, device="cuda")
    kept = torch.zeros(2, 2, 10, dtype=torch.int32, device="cuda")

    def evict(n=2, mk=30, stride=30, budget=10, recent=2, wi=w, kept=kept):
        return ua.ua_cache_evict(p.handle, bt.d_k, bt.d_v, bt.d_table, None, bt.d_sk, n, mk, wi, w, stride, budget,
                                 recent, kept, torch.zeros_like(bt.d_sk))

    assert evict(n=0) == 0
    assert [evict(n=3), evict(mk=31), evict(budget=0), evict(recent=11), evict(recent=-1), evict(wi=None),
            evict(kept=None), evict(mk=16 * bt.width + 1, stride=1000)] == [1] * 8
    with pytest.raises(ValueError):
        p.cache_evict(bt.d_k, bt.d_v, bt.d_table, bt.d_sk, 2, 30, w, w, 9, 2, kept, bt.d_sk)
    with pytest.raises(ValueError):
        p.cache_store(kn.transpose(1, 2), vn, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, bt.d_sk, 2, 2, 1, 30)


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["fp4", "bf16"])
@pytest.mark.parametrize("graph", [False, True])
def test_a_decode_loop_that_stores_weighs_and_evicts(kind, graph):
    """Prompts stored, then decode steps: store the token, attend with weights;
    every third step evict in place.  The whole step sequence also as replays
    of captured graphs on another stream."""
    hq, hk, d, b, budget, recent = 8, 2, 128, 16, 24, 5
    prompt, steps = [30, 9, 50], 6
    bt = Batch(200, kind, hq, hk, d, b, (1, 1, 1), [n + steps for n in prompt], 0.5, 0.5, store=False)
    bt.device()
    p = bt.problem(ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS, max_total_q=sum(prompt))
    stream = torch.cuda.Stream()
    pcu = torch.tensor(np.concatenate([[0], np.cumsum(prompt)]), dtype=torch.int32, device="cuda")
    psk = torch.tensor(prompt, dtype=torch.int32, device="cuda")

    def gather(raw, lo, hi):
        return torch.from_numpy(np.concatenate([raw[s][lo[s]:hi[s]] for s in range(3)]).view(np.int16).copy()
                                ).cuda().view(torch.bfloat16)

    zero = [0, 0, 0]
    p.cache_store(gather(bt.kb, zero, prompt), gather(bt.vb, zero, prompt), bt.d_k, bt.d_v, bt.d_table, pcu, psk, 3,
                  sum(prompt), max(prompt), max(prompt))
    max_k = max(prompt) + steps
    w = torch.zeros(3, hk, max_k, device="cuda")
    used = psk.clone()
    kept = torch.zeros(3, hk, budget, dtype=torch.int32, device="cuda")
    kn = torch.zeros(3, hk, d, dtype=torch.bfloat16, device="cuda")
    vn, q, out = torch.zeros_like(kn), torch.zeros_like(bt.d_q), torch.zeros_like(bt.d_q)
    qs = [bits(bt.rng.normal(size=(3, hq, d))) for _ in range(steps)]

    def step():
        used.add_(1)
        p.cache_store(kn, vn, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, used, 3, 3, 1, max_k)
        p.forward_weights(q, bt.d_k, bt.d_v, bt.d_table, bt.d_cu, used, 3, 3, 1, max_k, ua.UA_FLAG_CAUSAL, w, w,
                          decay=0.5, out=out)

    def evict():
        p.cache_evict(bt.d_k, bt.d_v, bt.d_table, used, 3, max_k, w, w, budget, recent, kept, used)

    torch.cuda.synchronize()
    graphs = {}
    if graph:
        saved = [t.clone() for t in (bt.d_k, bt.d_v, w, used)]
        with torch.cuda.stream(stream):
            for f in (step, evict):
                f()                                  # warm-up
                torch.cuda.synchronize()
                gr = torch.cuda.CUDAGraph()
                with torch.cuda.graph(gr, stream=stream):
                    f()
                graphs[f] = gr
        torch.cuda.synchronize()
        for t, x in zip((bt.d_k, bt.d_v, w, used), saved):
            t.copy_(x)

    # The same in 64 bits: per sequence and KV head the cached keys' indexes.
    held = [[list(range(prompt[s])) for _ in range(hk)] for s in range(3)]
    kq = R.Cache(kind, 1, b, hk, d, 0.5)
    cached = []                                      # the values a stored row reads back as
    for s in range(3):
        per = []
        for vals, raw in ((bt.k, bt.kb), (bt.v, bt.vb)):
            rows = []
            for j in range(bt.sk[s]):
                kq.put(0, 0, vals[s][j], raw[s][j])
                rows.append(kq.row(0, 0))
            per.append(np.stack(rows))
        cached.append(per)
    wref = [np.zeros((hk, prompt[s])) for s in range(3)]
    for i in range(steps):
        kn.copy_(gather(bt.kb, [n + i for n in prompt], [n + i + 1 for n in prompt]))
        vn.copy_(gather(bt.vb, [n + i for n in prompt], [n + i + 1 for n in prompt]))
        q.copy_(torch.from_numpy(qs[i][0].view(np.int16).copy()).cuda().view(torch.bfloat16))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            (graphs[step].replay() if graph else step())
        stream.synchronize()
        got_o, got_w = out.double().cpu().numpy(), w.double().cpu().numpy()
        g = hq // hk
        for s in range(3):
            n = len(held[s][0]) + 1
            new_w = np.zeros((hk, n))
            for h in range(hk):
                held[s][h].append(prompt[s] + i)
                kk, vv = (cached[s][x][held[s][h], h][:, None] for x in (0, 1))
                o, a, wt, mag = R.attention(qs[i][1][s:s + 1, h * g:(h + 1) * g], kk, vv, bt.scale)
                dx = R.score_error(mag, d)
                per = 2 * dx + 2.0 ** -10 + (2.0 ** -7 + 2.0 ** -8 if kind == "bf16" else 0)
                err = np.abs(got_o[s, h * g:(h + 1) * g] - o[0])
                assert np.all(err <= 2.0 ** -8 * np.abs(o[0]) + per * a[0])
                fresh = wt.sum((0, 1))
                new_w[h] = fresh
                new_w[h, :-1] += 0.5 * wref[s][h]
                # Errors of earlier steps are carried along (halved each step).
                assert np.all(np.abs(got_w[s, h, :n] - new_w[h]) <= new_w[h] * (4 * dx + 2.0 ** -16) + 1e-30)
            wref[s] = new_w
        if i % 3 == 2:
            # Choices follow the GPU's own weights (a near tie may go either way).
            exact_w = w.cpu().numpy().copy()
            with torch.cuda.stream(stream):
                (graphs[evict].replay() if graph else evict())
            stream.synchronize()
            for s in range(3):
                n = len(held[s][0])
                m = min(n, budget)
                nw = np.zeros((hk, m))
                for h in range(hk):
                    idx = R.evict_choice(exact_w[s, h], n, budget, recent)
                    np.testing.assert_array_equal(kept[s, h, :m].cpu().numpy(), idx)
                    held[s][h] = [held[s][h][j] for j in idx]
                    nw[h] = wref[s][h][idx]
                wref[s] = nw
                assert used[s].item() == m
    assert p.check_device_error() == 0
