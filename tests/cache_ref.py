"""Plain 64-bit implementations of the cache operators (store formats, expand,
attention with key weights, eviction), from their definitions, on numpy arrays.
They share no code with the library or the oracle."""
import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9) if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def bf16_values(t):
    """A torch bf16 tensor as float64."""
    return t.detach().cpu().float().numpy().astype(np.float64)


def nearest(x, table):
    """Index of the nearest entry of an ascending table (x >= 0), ties to the
    even index, saturating at the last."""
    hi = np.clip(np.searchsorted(table, x), 1, len(table) - 1)
    lo = hi - 1
    below, above = x - table[lo], table[hi] - x
    return np.where((above < below) | ((above == below) & (hi % 2 == 0)), hi, lo)


def e4m3_codes(y):
    """e4m3 codes of float values: nearest even, saturating, NaN = 0x7f."""
    c = nearest(np.minimum(np.abs(y), 448.0), E4M3).astype(np.uint8)
    c = np.where(np.signbit(y), c | 0x80, c)
    return np.where(np.isnan(y), 0x7f, c).astype(np.uint8)


def e4m3_values(c):
    c = c.astype(np.int64)
    mag = np.append(E4M3, np.nan)[c & 0x7f]
    return np.where(c & 0x80, -mag, mag)


def quantise_fp4(x, tensor_scale):
    """[..., d] float64 -> (codes [..., d], scale bytes [..., d / 16])."""
    with np.errstate(all="ignore"):
        y = (x.astype(np.float32) / np.float32(tensor_scale)).astype(np.float64)
        y = y.reshape(*x.shape[:-1], -1, 16)
        nan = np.isnan(y).any(-1)
        amax = np.where(nan, 0.0, np.abs(y).max(-1))
        s8 = np.where(nan, 0x7f, e4m3_codes(amax / 6.0))
        s = np.where(nan, 0.0, E4M3[np.where(nan, 0, s8)])[..., None]
        ratio = np.where(s > 0, np.abs(y) / np.where(s > 0, s, 1.0), 0.0)
        code = nearest(np.minimum(np.where(np.isnan(ratio), 0.0, ratio), 6.0), E2M1)
    code = np.where((s > 0) & (code > 0), code + 8 * np.signbit(y), 0)
    return code.reshape(x.shape).astype(np.uint8), s8.astype(np.uint8)


class Cache:
    """One K or V cache as numpy bytes / bf16 bit patterns, by kv type."""

    def __init__(self, kind, num_blocks, b, hk, d, scale=1.0, fill=None):
        self.kind, self.b, self.hk, self.d, self.scale = kind, b, hk, d, scale
        if kind == "fp4":
            self.raw = np.zeros((num_blocks, hk, b * (d // 2 + d // 16)), np.uint8)
        else:
            self.raw = np.zeros((num_blocks, b, hk, d), np.uint16 if kind == "bf16" else np.uint8)
        if fill is not None:
            self.raw[...] = fill

    def put(self, block, slot, rows, bits):
        """rows: float64 [hk, d]; bits: their bf16 bit patterns."""
        if self.kind == "bf16":
            self.raw[block, slot] = bits
        elif self.kind == "fp8":
            with np.errstate(all="ignore"):
                y = (rows.astype(np.float32) / np.float32(self.scale)).astype(np.float64)
            self.raw[block, slot] = e4m3_codes(y)
        else:
            codes, s8 = quantise_fp4(rows, self.scale)
            packed = codes[:, 0::2] | (codes[:, 1::2] << 4)
            n, w, g = self.b * self.d // 2, self.d // 2, self.d // 16
            self.raw[block, :, slot * w:(slot + 1) * w] = packed
            self.raw[block, :, n + slot * g:n + (slot + 1) * g] = s8

    def row_bytes(self, block, slot, h):
        """The row's stored bytes, as one array (for moves)."""
        if self.kind != "fp4":
            return self.raw[block, slot, h].copy()
        n, w, g = self.b * self.d // 2, self.d // 2, self.d // 16
        r = self.raw[block, h]
        return np.concatenate([r[slot * w:(slot + 1) * w], r[n + slot * g:n + (slot + 1) * g]])

    def set_row_bytes(self, block, slot, h, row):
        if self.kind != "fp4":
            self.raw[block, slot, h] = row
            return
        n, w, g = self.b * self.d // 2, self.d // 2, self.d // 16
        self.raw[block, h, slot * w:(slot + 1) * w] = row[:w]
        self.raw[block, h, n + slot * g:n + (slot + 1) * g] = row[w:]

    def row(self, block, slot):
        """float64 [hk, d] values."""
        if self.kind == "bf16":
            return (self.raw[block, slot].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        if self.kind == "fp8":
            return e4m3_values(self.raw[block, slot]) * np.float64(np.float32(self.scale))
        rows = np.stack([self.row_bytes(block, slot, h) for h in range(self.hk)])
        w = self.d // 2
        codes = np.stack([rows[:, :w] & 15, rows[:, :w] >> 4], -1).reshape(self.hk, self.d)
        mag = E2M1[codes & 7]
        s = np.repeat(e4m3_values(rows[:, w:]), 16, -1)
        return np.where(codes & 8, -mag, mag) * s * np.float64(np.float32(self.scale))

    def rows(self, table_row, n):
        """float64 [n, hk, d] of keys 0 .. n - 1."""
        if n == 0:
            return np.zeros((0, self.hk, self.d))
        return np.stack([self.row(int(table_row[j // self.b]), j % self.b) for j in range(n)])


def attention(q, keys, values, scale, *, causal=True, softcap=0.0, window=0, sinks=None, alibi=None, qq=None):
    """One sequence: q [S_q, H_q, d], keys / values [S_k, H_k, d] (float64).
    Returns out, abs_out (sum of weight times |v|), the weights [H_q, S_q, S_k]
    and mag, the largest sum |q||k| * scale of a row."""
    sq, hq, d = q.shape
    sk, hk = keys.shape[:2]
    g, ctx = hq // hk, sk - sq
    j, i = np.arange(sk), np.arange(sq)
    out, absout = np.zeros((sq, hq, d)), np.zeros((sq, hq, d))
    weights, mag = np.zeros((hq, sq, sk)), 0.0
    for h in range(hq):
        kh, vh = keys[:, h // g], values[:, h // g]
        x = q[:, h] @ kh.T * scale
        if x.size:
            mag = max(mag, float((np.abs(q[:, h]) @ np.abs(kh).T).max()) * scale)
        if softcap:
            x = softcap * np.tanh(x / softcap)
        if alibi is not None:
            x = x + alibi[h] * (j - ctx)[None]
        if qq is not None:
            for a in range(sq):
                x[a, ctx:] += qq[a, :sk - ctx]
        see = np.ones((sq, sk), bool)
        if causal:
            see &= j[None] <= i[:, None] + ctx
        if window:
            see &= j[None] >= i[:, None] + ctx - window + 1
        x = np.where(see, x, -np.inf)
        m = x.max(-1, initial=-np.inf)
        if sinks is not None:
            m = np.maximum(m, sinks[h])
        m = np.where(np.isfinite(m), m, np.where(m > 0, m, 0.0))
        with np.errstate(invalid="ignore"):
            p = np.where(see, np.exp(x - m[:, None]), 0.0)
            total = p.sum(-1) + (np.exp(sinks[h] - m) if sinks is not None else 0.0)
        if sinks is not None and sinks[h] == np.inf:
            p, total = np.zeros_like(p), np.ones(sq)
        p = p / np.where(total == 0, 1.0, total)[:, None]
        weights[h] = p
        out[:, h], absout[:, h] = p @ vh, p @ np.abs(vh)
    return out, absout, weights, mag


def evict_choice(w, sk, budget, recent):
    """Kept positions, ascending."""
    if sk <= budget:
        return np.arange(sk)
    n = sk - recent
    key = np.where(np.isnan(w[:n]), -np.inf, w[:n].astype(np.float64))
    nan = np.isnan(w[:n])
    # Descending weight, NaN after everything else, ties by position.
    order = sorted(range(n), key=lambda j: (bool(nan[j]), -key[j], j))
    return np.concatenate([np.sort(np.array(order[:budget - recent], dtype=np.int64)),
                           np.arange(n, sk)]).astype(np.int64)


def score_error(mag, d, softcap=0.0, largest=0.0):
    """Bound on the error of a score x (natural units) computed with exact 16-bit
    operands: fp32 accumulation of d products in d / 16 steps of 16 (each step
    and product sum off by at most 2^-22 of the running magnitude, truncation
    allowed), then a handful of fp32 roundings (2^-24 each) of numbers no larger
    than mag + softcap + largest (the other terms)."""
    steps = d / 16 + 4
    return steps * 2.0 ** -22 * mag + 8 * 2.0 ** -24 * (mag + largest) + (4e-6 * softcap if softcap else 0.0)


def tokens_of(cu, s):
    return int(cu[s]), int(cu[s + 1])


def log2(x):
    return math.log2(x)
