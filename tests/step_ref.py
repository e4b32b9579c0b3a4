"""Plain implementations of a speculative decoding step (blocks and slots, rotary
positions, attention for draft trees, accepted branches), from their definitions, on
lists and 64-bit numpy arrays.  They share no code with the library."""
import math

import numpy as np

BOUNDS, BLOCK_ID, TREE, POOL = 8, 2, 32, 64


def grow(rng, n, branching=0.5, roots=0.05):
    """Parents of a random tree of n nodes, parents in front of their children."""
    return [-1 if i == 0 or rng.random() < roots else i - 1 if rng.random() > branching else int(rng.integers(0, i))
            for i in range(n)]


def branch(parents, i):
    """Node numbers from the root to node i (none for -1)."""
    path = []
    while i >= 0:
        path.append(i)
        i = parents[i]
    return path[::-1]


def depths(parents):
    return [len(branch(parents, i)) - 1 for i in range(len(parents))]


def mask_of(parents, words):
    """uint32 [nodes, words]."""
    m = np.zeros((len(parents), words), np.uint32)
    for i in range(len(parents)):
        for c in branch(parents, i):
            m[i, c // 32] |= np.uint32(1 << c % 32)
    return m


class Step:
    """The state of ua_plan_step as lists, and one step on it."""

    def __init__(self, table, held, pool, b, num_blocks):
        self.table, self.held, self.pool = [list(r) for r in table], list(held), list(pool)
        self.b, self.num_blocks, self.width = b, num_blocks, len(table[0]) if len(table) else 0

    def plan(self, ctx, new, max_tokens, trees=None, words=0):
        b, err, n = self.b, 0, len(ctx)
        need, bad = [], []
        for s in range(n):
            end = ctx[s] + new[s]
            wrong = (ctx[s] < 0 or new[s] < 0 or not 0 <= self.held[s] <= self.width or end > self.width * b
                     or (words and new[s] > 32 * words))
            bad.append(wrong)
            need.append(self.held[s] if wrong else -(-end // b))
            err |= BOUNDS if wrong else 0
        back = []
        for s in range(n):
            back += self.table[s][need[s]:self.held[s]]
        if len(self.pool) + len(back) > self.num_blocks:
            err |= POOL
            back = []
        else:
            for s in range(n):
                self.held[s] = min(self.held[s], need[s]) if not bad[s] else self.held[s]
        self.pool += back[::-1]
        budget, asked, tokens = len(self.pool), 0, 0
        out = dict(granted=[], cu=[0], used=[], pos=[], slots=[], mask=[])
        for s in range(n):
            c, k = (0, 0) if bad[s] else (ctx[s], new[s])
            more = max(need[s] - self.held[s], 0)
            asked += more
            tokens += k
            if tokens > max_tokens:
                err |= BOUNDS if k else 0
            if tokens > max_tokens or (more and asked > budget):
                k = more = 0
            for _ in range(more):
                self.table[s][self.held[s]] = self.pool.pop()
                self.held[s] += 1
            tree = trees[s][:k] if trees is not None else list(range(-1, k - 1))
            for i, dep in enumerate(depths(tree)):
                blk = self.table[s][(c + i) // b]
                if not 0 <= blk < self.num_blocks:
                    err |= BLOCK_ID
                out["slots"].append(blk * b + (c + i) % b if 0 <= blk < self.num_blocks else -1)
                out["pos"].append(c + dep)
            if words:
                out["mask"].append(mask_of(tree, words))
            out["granted"].append(k)
            out["cu"].append(out["cu"][-1] + k)
            out["used"].append(c + k)
        return out, err


def rotate(x, pos, freq, pairs, magnitude=1.0):
    """x [tokens, heads, d] float64 rotated by positions [tokens] (python ints)."""
    n = len(freq)
    # Whole turns dropped in integer arithmetic of 200 bits, far beyond what is compared.
    angle = np.array([[math.fmod(int(p) * f, 2 * math.pi) if abs(int(p) * f) < 1e5 else _fraction(int(p), f)
                       for f in freq] for p in pos]).reshape(len(pos), n)[:, None]
    c, s = np.cos(angle) * magnitude, np.sin(angle) * magnitude
    y = x.copy()
    a, z = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if pairs else (x[..., :n], x[..., n:2 * n])
    u, v = a * c - z * s, a * s + z * c
    if pairs:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = u, v
    else:
        y[..., :n], y[..., n:2 * n] = u, v
    return y


def _fraction(p, f):
    """p * f modulo 2 pi for large products: f is the double, pi has 60 digits."""
    from fractions import Fraction
    pi = Fraction(314159265358979323846264338327950288419716939937510582097494, 10 ** 59)
    x = Fraction(f) * p
    k = x // (2 * pi)
    return float(x - k * 2 * pi)


def tree_attention(q, keys, values, scale, see, *, pos=None, softcap=0.0, window=0, sinks=None, alibi=None):
    """One sequence: q [S_q, H_q, d], keys / values [S_k, H_k, d] (float64), see bool
    [S_q, S_q] of the chunk's keys, pos [S_q] positions of the rows.  Returns out, the sum
    of weight times |v| (values that are not finite count as 0), and the largest
    sum |q||k| * scale of a visible pair."""
    sq, hq, d = q.shape
    sk, hk = keys.shape[:2]
    g, ctx = hq // hk, sk - sq
    at = np.arange(sk)
    if pos is not None:
        at = np.concatenate([at[:ctx], np.asarray(pos)])
    vis = np.concatenate([np.ones((sq, ctx), bool), see], 1)
    if window:
        vis &= at[None] > at[ctx:, None] - window
    out, absout, mag = np.zeros((sq, hq, d)), np.zeros((sq, hq, d)), 0.0
    for h in range(hq):
        for i in range(sq):
            j = np.nonzero(vis[i])[0]
            k, v = keys[j, h // g], values[j, h // g]
            if not len(j):
                continue
            x = k @ q[i, h] * scale
            mag = max(mag, float((np.abs(k) @ np.abs(q[i, h])).max()) * scale)
            if softcap:
                x = softcap * np.tanh(x / softcap)
            if alibi is not None:
                x = x + alibi[h] * (at[j] - ctx)
            m = x.max() if sinks is None else max(x.max(), sinks[h])
            if m == np.inf:
                continue
            p = np.exp(x - m) if m > -np.inf else np.zeros_like(x)
            total = p.sum() + (math.exp(sinks[h] - m) if sinks is not None and m > -np.inf else 0.0)
            p = p / total if total else p
            with np.errstate(invalid="ignore"):
                out[i, h] = (p[:, None] * v).sum(0)
            absout[i, h] = p @ np.where(np.isfinite(v), np.abs(v), 0.0)
    return out, absout, mag
