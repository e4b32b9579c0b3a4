"""The cache operators as timed cases: quantised stores, attention over a 4-bit
cache, attention that accumulates key weights, and eviction by those weights.

Each case names one operator by ``kind``:

* ``store``    a chunk's K/V rows written into the paged cache (4-bit or fp8) and
               the same keys expanded to bf16 pages again, as a prompt does
               before its tensor-core prefill reads them;
* ``attend``   ``ua_forward`` over a 4-bit cache;
* ``weights``  ``ua_forward_weights``: attention plus the accumulated weight of
               every cached key;
* ``evict``    ``ua_cache_evict``: the heaviest and the most recent keys of every
               (sequence, KV head) compacted into other blocks.

Lengths are drawn from the case's own ``lens`` seed, so a case's work does not
depend on the seed of its values.  With ``own`` false the plain forms run:
padded batches, elementary torch operations in fp32, one rounding at the end.
"""
import math
import random

import torch

own = False

PAIRS = {"8/2": (8, 2), "16/1": (16, 1), "16/2": (16, 2), "32/8": (32, 8), "8/8": (8, 8)}
# Padded K or V elements a plain pass may hold at once (its fp32 copies).
MOST_PADDED = 600_000_000
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _case(kind, *, kv="fp4", heads="32/8", d=128, b=16, seqs=1, sq=(1, 1), ctx=(0, 0), lens=0,
          softcap=0.0, window=0, sinks=False, alibi=False, kscale=1.0, decay=1.0, budget=0, recent=0,
          name=None):
    c = dict(kind=kind, kv=kv, heads=heads, d=d, b=b, seqs=seqs, sq_min=sq[0], sq_max=sq[1],
             ctx_min=ctx[0], ctx_max=ctx[1], lens=lens, softcap=softcap, window=window, sinks=sinks,
             alibi=alibi, kscale=kscale, decay=decay, budget=budget, recent=recent)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # One request's next token: launch and split latency.
        _case("attend", name="attend_one_request", ctx=(999, 999)),
        # The 64-request decode batch of the benchmark, cache in 4 bits.
        _case("attend", name="attend_decode_batch", seqs=64, ctx=(511, 8191), lens=1),
        # Speculative steps of 1 to 4 tokens with every mask and a capped score, d = 64.
        _case("attend", name="attend_draft_tokens_d64", heads="8/2", d=64, b=32, seqs=32, sq=(1, 4),
              ctx=(200, 4095), lens=2, softcap=50.0, window=1024, sinks=True),
        # Few very long requests, wide heads.
        _case("attend", name="attend_long_d256", heads="16/2", d=256, b=64, seqs=4, ctx=(30000, 65535),
              lens=3, kscale=0.5),
        # A decode step's tokens appended to 64 requests.
        _case("store", name="store_decode_step", seqs=64, ctx=(511, 8191), lens=1),
        # The chunked-prefill batch's prompts, appended after their context.
        _case("store", name="store_chunks", b=32, seqs=16, sq=(1, 512), ctx=(0, 4096), lens=4, kscale=0.25),
        # Whole prompts of 8192 tokens.
        _case("store", name="store_prompts", b=64, seqs=8, sq=(8192, 8192), lens=5),
        # One small request on a bf16 cache, weights decayed.
        _case("weights", name="weights_one_request", kv="bf16", heads="8/2", d=64, ctx=(600, 600), decay=0.9),
        # The decode batch on its bf16 cache, weights of every key accumulated.
        _case("weights", name="weights_decode_batch", kv="bf16", seqs=64, ctx=(511, 8191), lens=1),
        # An observation window of the last 8 to 32 prompt tokens over a 4-bit cache.
        _case("weights", name="weights_window_fp4", b=32, seqs=8, sq=(8, 32), ctx=(1000, 12000), lens=6,
              decay=0.0),
        # The decode batch thinned to 2048 keys, bf16 cache.
        _case("evict", name="evict_decode_batch", kv="bf16", seqs=64, ctx=(511, 8191), lens=1,
              budget=2048, recent=256),
        # Few long requests on a 4-bit cache thinned to an odd budget.
        _case("evict", name="evict_long_fp4", heads="16/2", b=64, seqs=4, ctx=(30000, 65535), lens=3,
              budget=8191, recent=1000),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "attend", "weights", "evict"])
    heads = rng.choice(list(PAIRS))
    d = rng.choice([64, 128, 128, 256])
    kv = {"store": ["fp4", "fp4", "fp8"], "attend": ["fp4"], "weights": ["bf16", "fp4", "fp8"],
          "evict": ["bf16", "fp4"]}[kind]
    kv = rng.choice(kv)
    if kv == "fp8":
        d = 128   # the head size an fp8 cache has
    c = _case(kind, kv=kv, heads=heads, d=d, b=rng.choice([16, 32, 64]), seqs=_log_int(rng, 1, 64),
              lens=rng.randrange(1 << 30), kscale=rng.choice([1.0, 1.0, 0.5, 0.0625]) if kv != "bf16" else 1.0)
    hi = _log_int(rng, 100, 65535)
    c["ctx_max"], c["ctx_min"] = hi, rng.randrange(1, hi)
    if kind == "store":
        c["sq_max"] = rng.choice([1, _log_int(rng, 2, 4096)])
        c["ctx_min"] = rng.choice([0, c["ctx_min"]])
    elif kind in ("attend", "weights"):
        c["sq_max"] = rng.choice([1, 1, 1, rng.randint(2, 5), rng.randint(6, 32)])
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
        c["window"] = rng.choice([0, 0, _log_int(rng, 8, 4096)])
        c["sinks"] = rng.random() < 0.3
        c["alibi"] = rng.random() < 0.2
        c["decay"] = rng.choice([1.0, 0.95, 0.0]) if kind == "weights" else 1.0
    else:
        c["budget"] = rng.randint(1, max(1, hi // 2))
        c["recent"] = rng.randint(0, c["budget"])
    most = {"bytes": 0, "flops": 0}
    for x in listed():
        if x["kind"] == kind:
            most = {m: max(v, work(x)[m]) for m, v in most.items()}
    while True:
        sq, sk = _lengths(c)
        hq, hk = PAIRS[c["heads"]]
        padded = len(sk) * max(sk) * hk * c["d"]
        rows = len(sk) * hq * max(sq) * max(sk) if kind in ("attend", "weights") else 0
        if all(v <= most[m] for m, v in work(c).items()) and padded <= MOST_PADDED and rows <= MOST_PADDED // 2:
            return c
        if c["seqs"] > 1:
            c["seqs"] = (c["seqs"] + 1) // 2
        else:
            c["ctx_max"] = max(1, c["ctx_max"] // 2)
            c["ctx_min"] = min(c["ctx_min"], c["ctx_max"])
            c["sq_max"] = max(1, c["sq_max"] // 2)
            c["budget"] = min(c["budget"], c["ctx_max"])
            c["recent"] = min(c["recent"], c["budget"])


def _lengths(case):
    rng = random.Random(case["lens"])
    sq = [rng.randint(case["sq_min"], case["sq_max"]) for _ in range(case["seqs"])]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return sq, [a + c for a, c in zip(sq, ctx)]


def _row_bytes(case):
    """Bytes of one (key, KV head) row of the cache."""
    d = case["d"]
    return {"fp4": d // 2 + d // 16, "fp8": d, "bf16": 2 * d}[case["kv"]]


def work(case):
    hq, hk = PAIRS[case["heads"]]
    d, rb = case["d"], _row_bytes(case)
    sq, sk = _lengths(case)
    if case["kind"] == "store":
        n = sum(sq) * hk * 2
        # bf16 in, cache rows out and in again, bf16 out; scale, compare, multiply per element
        return {"bytes": n * (2 * d + 2 * rb + 2 * d), "flops": n * d * 4}
    if case["kind"] == "evict":
        bytes_ = flops = 0
        for k in sk:
            keep = min(k, case["budget"])
            bytes_ += hk * (keep * (2 * 2 * rb + 4 + 4) + (4 * k if k > keep else 4 * keep))
            if case["kv"] == "fp4":   # the kept rows expanded to bf16
                bytes_ += hk * keep * 2 * (rb + 2 * d)
            flops += hk * k
        return {"bytes": bytes_, "flops": flops}
    pairs = keys = 0
    for q, k in zip(sq, sk):
        w = case["window"] or k
        for i in range(q):
            pairs += min(i + k - q + 1, w)
        keys += min(k, w + q - 1)
    bytes_ = keys * hk * 2 * rb + 2 * sum(sq) * hq * d * 2
    if case["kind"] == "weights":
        bytes_ += sum(sk) * hk * 4 * (2 if case["decay"] else 1)
    return {"bytes": bytes_, "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ the 4-bit format
def _quantise_fp4(x, tensor_scale):
    """[..., d] values -> ([..., d] codes 0..15, [..., d / 16] e4m3 scale bytes)."""
    y = (x.float() / tensor_scale).unflatten(-1, (-1, 16))
    amax = y.abs().amax(-1)
    s8 = (amax.double() / 6.0).clamp(max=448.0).float().to(torch.float8_e4m3fn)
    s = s8.float().unsqueeze(-1)
    a = y.abs()
    # Midpoints between neighbouring magnitudes times s are exact in fp32; a
    # value on one goes to the even code.
    code = ((a > 0.25 * s).int() + (a >= 0.75 * s).int() + (a > 1.25 * s).int() + (a >= 1.75 * s).int()
            + (a > 2.5 * s).int() + (a >= 3.5 * s).int() + (a > 5.0 * s).int())
    code = torch.where(s > 0, code + 8 * torch.signbit(y).int(), torch.zeros_like(code))
    return code.to(torch.uint8).flatten(-2), s8.view(torch.uint8)


def _pages_fp4(codes, scales):
    """[n, b, hk, d] codes and [n, b, hk, d / 16] scales -> uint8 pages [n, hk, bytes]."""
    codes = codes.permute(0, 2, 1, 3)
    packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
    return torch.cat([packed.flatten(2), scales.permute(0, 2, 1, 3).flatten(2)], -1)


def _values_fp4(pages, b, d, tensor_scale):
    """uint8 pages [..., bytes] -> fp32 values [..., b, d]."""
    codes = pages[..., :b * d // 2].unflatten(-1, (b, d // 2))
    s = pages[..., b * d // 2:].view(torch.float8_e4m3fn).float().unflatten(-1, (b, d // 16))
    codes = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=pages.device)
    v = lut[codes.int()].unflatten(-1, (d // 16, 16)) * s.unsqueeze(-1)
    return v.flatten(-2) * tensor_scale


# ------------------------------------------------------------------ inputs
def _cache(case, blocks, gen, dev):
    """One cache of `blocks` blocks holding normal values; K-like channel magnitudes."""
    hk, d, b = PAIRS[case["heads"]][1], case["d"], case["b"]
    chan = torch.exp(0.4 * torch.randn(hk, d, generator=gen, device=dev))
    parts = []
    step = max(1, (64 << 20) // (b * hk * d))
    for i in range(0, blocks, step):
        x = (torch.randn(min(step, blocks - i), b, hk, d, generator=gen, device=dev) * chan).to(torch.bfloat16)
        if case["kv"] == "fp4":
            x = _pages_fp4(*_quantise_fp4(x, case["kscale"]))
        elif case["kv"] == "fp8":
            x = (x.float() / case["kscale"]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        parts.append(x)
    return torch.cat(parts)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hk = PAIRS[case["heads"]]
    d, b = case["d"], case["b"]
    sq, sk = _lengths(case)
    n = len(sk)
    nblk = [-(-k // b) for k in sk]
    width = max(nblk)
    kept = [-(-min(k, case["budget"]) // b) for k in sk] if case["kind"] == "evict" else [0] * n
    pool = sum(nblk) + sum(kept) + 3
    ids = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    dst = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    off = 0
    for s in range(n):
        table[s, :nblk[s]] = ids[off:off + nblk[s]]
        off += nblk[s]
        dst[s, :kept[s]] = ids[off:off + kept[s]]
        off += kept[s]
    cu = torch.tensor([0] + sq, device=dev).cumsum(0).to(torch.int32)
    st = dict(case=case, hq=hq, hk=hk, d=d, b=b, n=n, width=width, max_q=max(sq), max_k=max(sk),
              total_q=sum(sq), table=table, cu=cu, used=torch.tensor(sk, dtype=torch.int32, device=dev),
              scale=1.0 / math.sqrt(d), blocks=pool)
    if case["kind"] == "store":
        for name in ("k", "v"):
            chan = torch.exp(0.4 * torch.randn(hk, d, generator=gen, device=dev))
            st[name + "_new"] = (torch.randn(st["total_q"], hk, d, generator=gen, device=dev) * chan).to(torch.bfloat16)
            shape = (pool, hk, b * _row_bytes(case)) if case["kv"] == "fp4" else (pool, b, hk, d)
            st[name + "_cache"] = torch.zeros(shape, dtype=torch.uint8, device=dev)
        # bf16 pages for the new keys alone: page p of a sequence is table entry p.
        first = [(k - q) // b for q, k in zip(sq, sk)]
        need = [m - f for m, f in zip(nblk, first)]
        out_table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
        perm = torch.randperm(sum(need), generator=gen, device=dev).to(torch.int32)
        off = 0
        for s in range(n):
            out_table[s, first[s]:nblk[s]] = perm[off:off + need[s]]
            off += need[s]
        st["out_table"] = out_table
        st["begin"] = torch.tensor([k - q for q, k in zip(sq, sk)], dtype=torch.int32, device=dev)
        for name in ("k", "v"):
            st[name + "_out"] = torch.zeros(sum(need), b, hk, d, dtype=torch.bfloat16, device=dev)
    else:
        st["k_cache"] = _cache(case, pool, gen, dev)
        st["v_cache"] = _cache(case, pool, gen, dev)
    if case["kind"] in ("attend", "weights"):
        st["q"] = torch.randn(st["total_q"], hq, d, generator=gen, device=dev).to(torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])
        st["sinks"] = torch.randn(hq, generator=gen, device=dev) if case["sinks"] else None
        st["alibi"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=dev)
                       if case["alibi"] else None)
    if case["kind"] in ("weights", "evict"):
        # Accumulated weights have a long tail; some keys tie, some were never attended to.
        w = torch.empty(n, hk, st["max_k"], device=dev).exponential_(generator=gen)
        w = torch.where(w < 0.3, torch.floor(w * 64) / 64, w * w)
        st["w_in"] = w
        st["w_out"] = torch.zeros_like(w)
    if case["kind"] == "evict":
        st["dst"] = dst
        st["kept"] = torch.full((n, hk, case["budget"]), -7, dtype=torch.int32, device=dev)
        st["used_out"] = torch.zeros(n, dtype=torch.int32, device=dev)
        if case["kv"] == "fp4":
            # bf16 pages of the kept keys: page p of sequence s is page p * n + s.
            pages = -(-case["budget"] // b)
            grid = torch.arange(pages, device=dev)[None] * n + torch.arange(n, device=dev)[:, None]
            out_table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
            m = min(width, pages)
            out_table[:, :m] = grid[:, :m].to(torch.int32)
            st["out_table"] = out_table
            for name in ("k", "v"):
                st[name + "_out"] = torch.zeros(pages * n, b, hk, d, dtype=torch.bfloat16, device=dev)
    if own:
        import paged_varlen_flash_gb300 as ua
        flags = ua.flags_of(True, case["softcap"], case["alibi"], case["window"], case["sinks"])
        st["flags"] = flags
        kind = {"fp4": "UA_DTYPE_FP4_E2M1", "fp8": "UA_DTYPE_FP8_E4M3", "bf16": "UA_DTYPE_BF16"}[case["kv"]]
        st["problem"] = ua.Problem(
            hq, hk, d, b, pool, n, width, max(1, st["total_q"]),
            flags | (ua.UA_FLAG_KEY_WEIGHTS if case["kind"] == "weights" else 0), st["scale"],
            case["softcap"], case["window"], kv_dtype=getattr(ua, kind), k_scale=case["kscale"],
            v_scale=case["kscale"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return globals()["_" + state["case"]["kind"]](state)


def _store(st):
    if own:
        p = st["problem"]
        p.cache_store(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"], st["cu"],
                      st["used"], st["n"], st["total_q"], st["max_q"], st["max_k"])
        p.cache_expand(st["k_cache"], st["v_cache"], st["table"], st["used"], st["n"], st["max_q"],
                       st["k_out"], st["v_out"], st["out_table"], begin=st["begin"])
        return [st["k_out"], st["v_out"]]
    s, pos = _token_place(st)
    block, slot = st["table"][s, pos // st["b"]].long(), pos % st["b"]
    to = st["out_table"][s, pos // st["b"]].long()
    for name in ("k", "v"):
        x, cache = st[name + "_new"], st[name + "_cache"]
        if st["case"]["kv"] == "fp4":
            codes, scales = _quantise_fp4(x, st["case"]["kscale"])
            packed = codes[..., 0::2] | (codes[..., 1::2] << 4)
            n_codes = st["b"] * st["d"] // 2
            code_rows = cache[..., :n_codes].unflatten(-1, (st["b"], st["d"] // 2))
            scale_rows = cache[..., n_codes:].unflatten(-1, (st["b"], st["d"] // 16))
            code_rows[block, :, slot] = packed
            scale_rows[block, :, slot] = scales
            rows = torch.cat([code_rows[block, :, slot], scale_rows[block, :, slot]], -1)
            vals = _values_fp4(rows, 1, st["d"], st["case"]["kscale"])[..., 0, :]
        else:
            y = (x.float() / st["case"]["kscale"]).clamp(-448.0, 448.0)
            cache[block, slot] = y.to(torch.float8_e4m3fn).view(torch.uint8)
            vals = cache[block, slot].view(torch.float8_e4m3fn).float() * st["case"]["kscale"]
        st[name + "_out"][to, slot] = vals.to(torch.bfloat16)
    return [st["k_out"], st["v_out"]]


def _token_place(st):
    """Per packed token: its sequence and its key position."""
    cu = st["cu"].long()
    t = torch.arange(st["total_q"], device=cu.device)
    s = torch.searchsorted(cu, t, right=True) - 1
    return s, st["used"].long()[s] - (cu[s + 1] - t)


def _rows_fp32(st, name):
    """The batch's cached rows, padded: fp32 [n, hk, max_k, d]."""
    pages = st[name + "_cache"][st["table"].clamp(min=0).long()]
    if st["case"]["kv"] == "fp4":
        v = _values_fp4(pages, st["b"], st["d"], st["case"]["kscale"])      # n, width, hk, b, d
        v = v.permute(0, 2, 1, 3, 4)
    elif st["case"]["kv"] == "fp8":
        v = (pages.view(torch.float8_e4m3fn).float() * st["case"]["kscale"]).permute(0, 3, 1, 2, 4)
    else:
        v = pages.float().permute(0, 3, 1, 2, 4)
    return v.flatten(2, 3)[:, :, :st["max_k"]]


def _attention(st):
    """(out [total_q, hq, d] fp32, weights summed over each group [n, hk, max_k])."""
    case, n, hk, g, mq, mk = st["case"], st["n"], st["hk"], st["hq"] // st["hk"], st["max_q"], st["max_k"]
    dev = st["q"].device
    cu, used = st["cu"].long(), st["used"].long()
    ctx = used - (cu[1:] - cu[:-1])
    i = torch.arange(mq, device=dev)
    tok = (cu[:-1, None] + i).clamp(max=st["total_q"] - 1)
    q = st["q"][tok].float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4)   # n, hk, g, mq, d
    x = torch.matmul(q.flatten(2, 3) * st["scale"], _rows_fp32(st, "k").transpose(-1, -2))
    x = x.unflatten(2, (g, mq))
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    j = torch.arange(mk, device=dev)
    if case["alibi"]:
        x = x + st["alibi"].view(1, hk, g, 1, 1) * (j - ctx[:, None]).view(n, 1, 1, 1, mk)
    last = ctx[:, None] + i
    see = (j <= last[..., None]) & (i < (cu[1:] - cu[:-1])[:, None])[..., None]
    if case["window"]:
        see = see & (j > last[..., None] - case["window"])
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    if case["sinks"]:
        sink = st["sinks"].view(1, hk, g, 1, 1)
        m = torch.maximum(m, sink)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if case["sinks"]:
        total = total + torch.exp(sink - m)
    p = p / total.masked_fill(total == 0, 1.0)
    o = torch.matmul(p.flatten(2, 3), _rows_fp32(st, "v")).unflatten(2, (g, mq))
    s, pos = _token_place(st)
    o = o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s, pos - ctx[s]]
    return o, p.sum((2, 3))


def _attend(st):
    if own:
        return st["problem"].forward(
            st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["used"], st["n"],
            st["total_q"], st["max_q"], st["max_k"], st["flags"], st["sinks"], st["alibi"], out=st["out"])
    return _attention(st)[0].to(torch.bfloat16)


def _weights(st):
    if own:
        out = st["problem"].forward_weights(
            st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["used"], st["n"],
            st["total_q"], st["max_q"], st["max_k"], st["flags"], st["w_in"], st["w_out"],
            decay=st["case"]["decay"], sinks=st["sinks"], alibi_slopes=st["alibi"], out=st["out"])
        return [out, st["w_out"]]
    o, p = _attention(st)
    cu, used = st["cu"].long(), st["used"].long()
    ctx = used - (cu[1:] - cu[:-1])
    j = torch.arange(st["max_k"], device=cu.device)
    old = st["w_in"] * (j < ctx[:, None])[:, None] * st["case"]["decay"]
    st["w_out"].copy_(torch.where((j < used[:, None])[:, None], old + p, st["w_out"]))
    return [o.to(torch.bfloat16), st["w_out"]]


def _evict(st):
    case = st["case"]
    if own:
        p = st["problem"]
        p.cache_evict(st["k_cache"], st["v_cache"], st["table"], st["used"], st["n"], st["max_k"],
                      st["w_in"], st["w_out"], case["budget"], case["recent"], st["kept"], st["used_out"],
                      dst_block_table=st["dst"])
        if case["kv"] != "fp4":
            return [st["k_cache"], st["v_cache"], st["w_out"], st["kept"], st["used_out"]]
        p.cache_expand(st["k_cache"], st["v_cache"], st["dst"], st["used_out"], st["n"],
                       min(st["max_k"], case["budget"]), st["k_out"], st["v_out"], st["out_table"])
        return [st["k_out"], st["v_out"], st["w_out"], st["kept"], st["used_out"]]
    n, hk, b, budget, recent = st["n"], st["hk"], st["b"], case["budget"], case["recent"]
    used = st["used"].long()
    j = torch.arange(st["max_k"], device=used.device)
    here = (j < used[:, None])[:, None].expand(n, hk, -1)
    tail = (j >= (used - recent)[:, None])[:, None] & here
    full = (used <= budget)[:, None, None] & here
    # Weights are at least 0: everything that is not a candidate sorts behind.
    w = torch.where(here & ~tail, st["w_in"], torch.full_like(st["w_in"], -1.0))
    order = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, j.expand_as(order).contiguous())
    keep = full | tail | (here & (rank < budget - recent))
    m = min(budget, st["max_k"])
    idx = torch.sort((~keep).to(torch.int8), dim=-1, stable=True).indices[..., :m]
    count = torch.minimum(used, torch.full_like(used, budget))
    live = (torch.arange(m, device=used.device) < count[:, None])[:, None].expand(n, hk, m)
    st["kept"].fill_(-1)
    st["kept"][..., :m] = torch.where(live, idx, -1).to(torch.int32)
    st["w_out"][..., :m] = torch.where(live, st["w_in"].gather(-1, idx), st["w_out"][..., :m])
    st["used_out"].copy_(count)
    s, h, to = torch.nonzero(live, as_tuple=True)
    src = idx[s, h, to]
    sb, db = st["table"][s, src // b].long(), st["dst"][s, to // b].long()
    for name in ("k", "v"):
        cache = st[name + "_cache"]
        if case["kv"] == "fp4":
            n_codes = b * st["d"] // 2
            for part in (cache[..., :n_codes].unflatten(-1, (b, -1)), cache[..., n_codes:].unflatten(-1, (b, -1))):
                part[db, h, to % b] = part[sb, h, src % b]
            rows = torch.cat([cache[..., :n_codes].unflatten(-1, (b, -1))[db, h, to % b],
                              cache[..., n_codes:].unflatten(-1, (b, -1))[db, h, to % b]], -1)
            vals = _values_fp4(rows, 1, st["d"], case["kscale"])[..., 0, :]
            st[name + "_out"][st["out_table"][s, to // b].long(), to % b, h] = vals.to(torch.bfloat16)
        else:
            cache[db, to % b, h] = cache[sb, src % b, h]
    first = [st["k_out"], st["v_out"]] if case["kv"] == "fp4" else [st["k_cache"], st["v_cache"]]
    return first + [st["w_out"], st["kept"], st["used_out"]]


# ------------------------------------------------------------------ 64 bits
def _e4m3_64(byte):
    """e4m3 bytes -> float64, from the bits."""
    c = byte.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    mag = torch.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * torch.exp2((e - 7).double()))
    return torch.where(c >= 128, -mag, mag)


def _nearest(x, table):
    """Nearest entry of an ascending table of magnitudes (x >= 0), ties to the even index."""
    hi = torch.searchsorted(table, x).clamp(1, len(table) - 1)
    lo = hi - 1
    below, above = x - table[lo], table[hi] - x
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return torch.where(up, hi, lo)


def _row_64(case, cache, block, slot, hk):
    """fp64 values [len(block), hk, d] of cached rows."""
    d, b = case["d"], case["b"]
    if case["kv"] == "bf16":
        return cache[block, slot].double()
    if case["kv"] == "fp8":
        return _e4m3_64(cache[block, slot]) * case["kscale"]
    h = torch.arange(hk, device=cache.device)[None, :, None]
    e = torch.arange(d, device=cache.device)[None, None]
    blk, at = block[:, None, None], slot[:, None, None]
    byte = cache[blk, h, at * (d // 2) + e // 2].long()
    code = (byte >> (4 * (e % 2))) & 15
    ex, m = (code >> 1) & 3, (code & 1).double()
    mag = torch.where(ex == 0, m / 2, (1 + m / 2) * torch.exp2((ex - 1).double()))
    s = _e4m3_64(cache[blk, h, b * d // 2 + at * (d // 16) + e // 16])
    return torch.where(code >= 8, -mag, mag) * s * case["kscale"]


def exact(case, seed):
    st = prepare(case, seed)
    sq, sk = _lengths(case)
    hq, hk, d, b = st["hq"], st["hk"], st["d"], st["b"]
    g = hq // hk
    dev = st["table"].device
    if case["kind"] == "store":
        e4m3 = _e4m3_64(torch.arange(127, device=dev))
        e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=dev)
        outs = []
        for name in ("k", "v"):
            res = st[name + "_out"].double()
            t0 = 0
            for s in range(len(sk)):
                y = (st[name + "_new"][t0:t0 + sq[s]].float() / case["kscale"]).double()
                t0 += sq[s]
                if case["kv"] == "fp4":
                    y = y.reshape(sq[s], hk, d // 16, 16)
                    sc = e4m3[_nearest((y.abs().amax(-1) / 6).clamp(max=448), e4m3)][..., None]
                    r = torch.where(sc > 0, y.abs() / sc.clamp(min=2.0 ** -9), torch.zeros_like(y))
                    val = torch.sign(y) * e2m1[_nearest(r.clamp(max=6), e2m1)] * sc
                else:
                    val = torch.sign(y) * e4m3[_nearest(y.abs().clamp(max=448), e4m3)]
                pos = torch.arange(sk[s] - sq[s], sk[s], device=dev)
                res[st["out_table"][s, pos // b].long(), pos % b] = val.reshape(sq[s], hk, d) * case["kscale"]
            outs.append(res)
        return outs
    if case["kind"] == "evict":
        kept = torch.full_like(st["kept"], -1)
        w_out = st["w_out"].double()
        used_out = torch.zeros_like(st["used_out"])
        fp4 = case["kv"] == "fp4"
        outs = [st[x + ("_out" if fp4 else "_cache")].double() for x in ("k", "v")]
        for s in range(len(sk)):
            n = min(sk[s], case["budget"])
            used_out[s] = n
            for h in range(hk):
                old = sk[s] - case["recent"]
                if sk[s] <= case["budget"]:
                    idx = torch.arange(n, device=dev)
                else:
                    w = st["w_in"][s, h, :old].double()
                    best = torch.sort(-w, stable=True).indices[:n - case["recent"]]
                    idx = torch.cat([torch.sort(best).values, torch.arange(old, sk[s], device=dev)])
                kept[s, h, :n] = idx.to(torch.int32)
                w_out[s, h, :n] = st["w_in"][s, h, idx].double()
                to = torch.arange(n, device=dev)
                for o, x in zip(outs, ("k", "v")):
                    rows = _row_64(case, st[x + "_cache"], st["table"][s, idx // b].long(), idx % b, hk)[:, h]
                    o[(st["out_table"] if fp4 else st["dst"])[s, to // b].long(), to % b, h] = rows
        return outs + [w_out, kept, used_out]
    out = torch.zeros(st["total_q"], hq, d, dtype=torch.float64, device=dev)
    w_out = st["w_out"].double() if case["kind"] == "weights" else None
    t0 = 0
    for s in range(len(sk)):
        j = torch.arange(sk[s], device=dev)
        block, slot = st["table"][s, j // b].long(), j % b
        k = _row_64(case, st["k_cache"], block, slot, hk)
        v = _row_64(case, st["v_cache"], block, slot, hk)
        ctx = sk[s] - sq[s]
        i = torch.arange(sq[s], device=dev)
        see = j[None] <= ctx + i[:, None]
        if case["window"]:
            see &= j[None] > ctx + i[:, None] - case["window"]
        for h in range(hq):
            x = st["q"][t0:t0 + sq[s], h].double() @ k[:, h // g].T * st["scale"]
            if case["softcap"]:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            if case["alibi"]:
                x = x + st["alibi"][h].double() * (j - ctx)[None]
            x = x.masked_fill(~see, -math.inf)
            lse = torch.logsumexp(x, -1)
            if case["sinks"]:
                lse = torch.logaddexp(lse, st["sinks"][h].double().expand_as(lse))
            p = torch.exp(x - lse[:, None])
            out[t0:t0 + sq[s], h] = p @ v[:, h // g]
            if w_out is not None:
                if h % g == 0:
                    old = st["w_in"][s, h // g, :sk[s]].double() * case["decay"]
                    w_out[s, h // g, :sk[s]] = torch.where(j < ctx, old, torch.zeros_like(old))
                w_out[s, h // g, :sk[s]] += p.sum(0)
        t0 += sq[s]
    return out if w_out is None else [out, w_out]
