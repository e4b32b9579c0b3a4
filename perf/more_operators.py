"""The operators of a speculative decoding step as timed cases: blocks and slots given
out on the GPU, rotary positions fused with the cache's store, attention for a tree of
drafted tokens, and the accepted branch's rows moved to their final positions.

Each case names one operator by ``kind``:

* ``plan``    ``ua_plan_step`` twice: a step's tokens get their blocks, slots, positions
              and ancestor masks, then the step is taken back (all drafts rejected) and
              its blocks return to the pool, so that every pass starts alike;
* ``rope``    ``ua_rope_store``: q rotated, k rotated and stored with v;
* ``tree``    ``ua_forward_tree``;
* ``accept``  ``ua_cache_accept``.

Lengths, trees and accepted branches come from the case's own ``lens`` seed, so a case's
work does not depend on the seed of its values.  With ``own`` false the plain forms run:
elementary torch operations in fp32 (angles in fp64), one rounding at the end.
"""
import math
import random

import torch

own = False

PAIRS = {"8/2": (8, 2), "16/1": (16, 1), "16/2": (16, 2), "32/8": (32, 8), "8/8": (8, 8)}
# Elements of padded K or V, and of scores, that a plain pass may hold at once.
MOST_PADDED = 600_000_000


# ------------------------------------------------------------------ cases
def _case(kind, *, heads="32/8", d=128, b=16, seqs=1, sq=(1, 1), ctx=(0, 0), lens=0, tree=False, pool=1.0,
          kv="bf16", kscale=1.0, rot=0, layout="half", scaling="none", softcap=0.0, window=0, sinks=False,
          alibi=False, name=None):
    c = dict(kind=kind, heads=heads, d=d, b=b, seqs=seqs, sq_min=sq[0], sq_max=sq[1], ctx_min=ctx[0],
             ctx_max=ctx[1], lens=lens, tree=tree, pool=pool, kv=kv, kscale=kscale, rot=rot or d, layout=layout,
             scaling=scaling, softcap=softcap, window=window, sinks=sinks, alibi=alibi)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # The 64-request decode batch of the benchmark: one token each.
        _case("plan", name="plan_decode_step", seqs=64, sq=(1, 1), ctx=(511, 8191), lens=1),
        # Draft trees of up to 64 nodes for 256 requests, with their ancestor masks; the pool
        # lacks a tenth of what the step asks for.
        _case("plan", name="plan_draft_trees", b=32, seqs=256, sq=(1, 64), ctx=(0, 8191), lens=2, tree=True,
              pool=0.9),
        # A wave of new prompts: about a million tokens.
        _case("plan", name="plan_prompts", b=64, seqs=128, sq=(1, 16384), ctx=(0, 0), lens=3),
        # The decode batch's tokens rotated and appended.
        _case("rope", name="rope_decode_step", seqs=64, sq=(1, 1), ctx=(511, 8191), lens=1),
        # Draft trees into an fp8 cache: neighbouring dims rotated, half of the head.
        _case("rope", name="rope_draft_trees_fp8", heads="16/2", b=32, seqs=256, sq=(1, 64), ctx=(0, 8191), lens=2,
              tree=True, kv="fp8", kscale=0.0625, rot=64, layout="pairs"),
        # Whole prompts of 8192 tokens behind a long context, frequencies scaled for it.
        _case("rope", name="rope_prompts", b=64, seqs=8, sq=(8192, 8192), ctx=(0, 65536), lens=5, scaling="bands"),
        # One request's small draft: launch and split latency.
        _case("tree", name="tree_one_request", heads="8/2", d=64, seqs=1, sq=(8, 8), ctx=(991, 991), lens=6, tree=True),
        # The decode batch with draft trees of 16 to 32 nodes.
        _case("tree", name="tree_decode_batch", seqs=64, sq=(16, 32), ctx=(511, 8191), lens=7, tree=True),
        # Ragged trees up to 64 nodes with every mask and a capped score, d = 64.
        _case("tree", name="tree_masked_d64", heads="8/2", d=64, b=32, seqs=48, sq=(1, 64), ctx=(0, 4095), lens=8,
              tree=True, softcap=50.0, window=1024, sinks=True),
        # Few very long requests, wide heads, 64 nodes for eight query heads per KV head.
        _case("tree", name="tree_long_d256", heads="16/2", d=256, b=64, seqs=4, sq=(64, 64), ctx=(30000, 65535),
              lens=9, tree=True),
        # The accepted branches of the decode batch's trees.
        _case("accept", name="accept_decode_batch", seqs=64, sq=(16, 32), ctx=(511, 2047), lens=7, tree=True),
        # Many requests, wide heads without grouping.
        _case("accept", name="accept_many_d256", heads="8/8", d=256, b=32, seqs=256, sq=(32, 64), ctx=(1, 511),
              lens=10, tree=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["plan", "rope", "tree", "accept"])
    d = rng.choice([64, 128, 128, 256])
    c = _case(kind, heads=rng.choice(list(PAIRS)), d=d, b=rng.choice([16, 32, 64]), seqs=_log_int(rng, 1, 256),
              lens=rng.randrange(1 << 30), tree=True)
    hi = _log_int(rng, 8, 65535)
    c["ctx_max"], c["ctx_min"] = hi, rng.randrange(0, hi)
    c["sq_max"] = _log_int(rng, 1, 64)
    c["sq_min"] = rng.randint(1, c["sq_max"])
    if kind == "plan":
        c["tree"] = rng.random() < 0.5
        if not c["tree"]:
            c["sq_max"], c["sq_min"] = _log_int(rng, 1, 16384), 0
        c["pool"] = rng.choice([1.0, 1.5, 0.7])
    elif kind == "rope":
        c["tree"] = rng.random() < 0.5
        if not c["tree"]:
            c["sq_max"] = _log_int(rng, 1, 8192)
            c["sq_min"] = rng.randint(1, c["sq_max"])
        c["rot"] = rng.choice([d, d, d // 2, d // 4])
        c["layout"] = rng.choice(["half", "pairs"])
        c["scaling"] = rng.choice(["none", "linear", "bands", "yarn"])
        if d == 128 and rng.random() < 0.4:
            c["kv"], c["kscale"] = "fp8", rng.choice([1.0, 0.25, 0.0625])
    elif kind == "accept":
        c["ctx_max"] = _log_int(rng, 8, 2047)
        c["ctx_min"] = rng.randrange(0, c["ctx_max"])
    else:
        c["softcap"] = rng.choice([0.0, 0.0, 30.0])
        c["window"] = rng.choice([0, 0, _log_int(rng, 8, 4096)])
        c["sinks"] = rng.random() < 0.3
        c["alibi"] = rng.random() < 0.2
    most = {"bytes": 0, "flops": 0}
    for x in listed():
        if x["kind"] == kind:
            most = {m: max(v, work(x)[m]) for m, v in most.items()}
    while True:
        sq, ctx = _lengths(c)
        hq, hk = PAIRS[c["heads"]]
        keys = max(a + x for a, x in zip(sq, ctx))
        padded = len(sq) * keys * hk * c["d"] if kind in ("tree", "accept") else 0
        rows = len(sq) * hq * max(sq) * keys if kind == "tree" else 0
        if all(v <= most[m] for m, v in work(c).items()) and padded <= MOST_PADDED and rows <= MOST_PADDED:
            return c
        if c["seqs"] > 1:
            c["seqs"] = (c["seqs"] + 1) // 2
        else:
            c["ctx_max"] = c["ctx_max"] // 2
            c["ctx_min"] = min(c["ctx_min"], c["ctx_max"])
            c["sq_max"] = max(1, c["sq_max"] // 2)
            c["sq_min"] = min(c["sq_min"], c["sq_max"])


def _lengths(case):
    rng = random.Random(case["lens"])
    sq = [rng.randint(case["sq_min"], case["sq_max"]) for _ in range(case["seqs"])]
    ctx = [rng.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    return sq, ctx


def _trees(case):
    """Parents of every sequence's nodes, level by level (a parent stands before its
    children; -1 is a first token), each node with up to about three children."""
    rng = random.Random(case["lens"] + 1)
    trees = []
    for n in _lengths(case)[0]:
        if not case["tree"]:
            trees.append(range(-1, n - 1))
            continue
        parents, at = [], -1
        for i in range(n):
            if i and (at < 0 or rng.random() < 0.5):
                at = min(at + 1 + (rng.random() < 0.2), i - 1)
            parents.append(at)
        trees.append(parents)
    return trees


def _branches(case):
    """The accepted branch of every sequence, as node numbers from the first token on.  None of
    its rows is overwritten before a second pass reads it again."""
    rng = random.Random(case["lens"] + 2)
    out = []
    for parents in _trees(case):
        best = []
        for _ in range(8):
            i, path = rng.randrange(-1, len(parents)), []
            while i >= 0:
                path.append(i)
                i = parents[i]
            path.reverse()
            if len(path) > len(best) and all(r == t or r >= len(path) for t, r in enumerate(path)):
                best = path
        out.append(best)
    return out


def _words(case):
    return -(-case["sq_max"] // 32)


def _blocks(case):
    """Per sequence: blocks held before the step, and blocks that it needs."""
    sq, ctx = _lengths(case)
    b = case["b"]
    return [-(-x // b) for x in ctx], [-(-(a + x) // b) for a, x in zip(sq, ctx)]


def _pool(case):
    held, need = _blocks(case)
    return int(case["pool"] * sum(n - h for h, n in zip(held, need)))


def work(case):
    hq, hk = PAIRS[case["heads"]]
    d = case["d"]
    sq, ctx = _lengths(case)
    if case["kind"] == "plan":
        held, need = _blocks(case)
        left, tokens, blocks = _pool(case), 0, 0
        for a, n in zip(sq, (n - h for h, n in zip(held, need))):
            left -= n
            if left >= 0 or n == 0:
                tokens += a
                blocks += n
        row = 12 + (4 * _words(case) + 4 if case["tree"] else 0)
        # a token's outputs, a taken block's id in and out, and out again; lengths, holdings and results
        return {"bytes": tokens * row + (sum(sq) - tokens) * 12 + blocks * 12 + 2 * len(sq) * 28, "flops": 4 * tokens}
    if case["kind"] == "rope":
        n = sum(sq)
        kept = 2 * d if case["kv"] == "bf16" else d
        return {"bytes": n * ((2 * hq + 2 * hk) * d * 2 + 2 * hk * kept + 12), "flops": n * (hq + hk) * case["rot"] * 3}
    if case["kind"] == "accept":
        row = 2 * hk * 2 * d
        moved = sum(sum(r != t for t, r in enumerate(path)) for path in _branches(case))
        return {"bytes": moved * 2 * row + sum(sq) * 4 + len(sq) * (16 + 4 * case["sq_max"]), "flops": sum(sq)}
    keys = pairs = 0
    for a, x in zip(sq, ctx):
        seen = min(x, case["window"]) if case["window"] else x
        keys += a + seen
        pairs += a * (seen + 1)
    return {"bytes": keys * hk * 2 * 2 * d + 2 * sum(sq) * hq * d * 2 + 4 * sum(sq) * _words(case),
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Angles per position (radians, as Python floats) and the factor on cos and sin."""
    n = case["rot"] // 2
    freq = [10000.0 ** (-i / n) for i in range(n)]
    if case["scaling"] == "linear":
        return [f / 4.0 for f in freq], 1.0
    if case["scaling"] == "bands":
        # Wavelengths beyond the trained 8192 positions stretched by 8, short ones kept.
        out = []
        for f in freq:
            turns = 8192.0 * f / (2.0 * math.pi)
            keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            out.append(f * (keep + (1.0 - keep) / 8.0))
        return out, 1.0
    if case["scaling"] == "yarn":
        turns = [4096.0 * f / (2.0 * math.pi) for f in freq]
        keep = [min(1.0, max(0.0, (t - 1.0) / 31.0)) for t in turns]
        return [f * (k + (1.0 - k) / 16.0) for f, k in zip(freq, keep)], 0.1 * math.log(16.0) + 1.0
    return freq, 1.0


def _depths(parents):
    depth = []
    for q in parents:
        depth.append(0 if q < 0 else depth[q] + 1)
    return depth


def _mask_words(case):
    """int32 [tokens, words]: the bits of every node's ancestors and of itself."""
    rows, words = [], _words(case)
    for parents in _trees(case):
        bits = []
        for i, q in enumerate(parents):
            bits.append((bits[q] if q >= 0 else 0) | 1 << i)
        rows += [[(x >> 32 * w & 0xffffffff) for w in range(words)] for x in bits]
    return torch.tensor(rows, dtype=torch.int64).to(torch.int32)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    hq, hk = PAIRS[case["heads"]]
    d, b = case["d"], case["b"]
    sq, ctx = _lengths(case)
    sk = [a + x for a, x in zip(sq, ctx)]
    n, total = len(sq), sum(sq)
    held, need = _blocks(case)
    width = max(max(need), 1)
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    table = torch.full((n, width), -1, dtype=torch.int32, device=dev)
    given = held if case["kind"] == "plan" else need
    free = _pool(case) if case["kind"] == "plan" else 0
    blocks = sum(given) + free + 3
    ids = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    owner = torch.arange(width, device=dev) < ints(given)[:, None]
    table[owner] = ids[:sum(given)]
    st = dict(case=case, hq=hq, hk=hk, d=d, b=b, n=n, total=total, max_q=max(sq), max_k=max(sk), blocks=blocks,
              table=table, scale=1.0 / math.sqrt(d), sq=ints(sq), ctx=ints(ctx), used=ints(sk),
              cu=torch.tensor([0] + sq, device=dev).cumsum(0).to(torch.int32))
    if case["tree"]:
        trees = _trees(case)
        st["parents"] = ints([list(p) + [-1] * (case["sq_max"] - len(p)) for p in trees])
    if case["kind"] == "plan":
        pool = torch.full((blocks,), -1, dtype=torch.int32, device=dev)
        pool[:free] = ids[sum(given):sum(given) + free]
        st.update(held=ints(held), pool=pool, left=ints([free]), none=torch.zeros_like(st["sq"]))
        for name in ("step", "back"):
            st[name] = dict(granted=ints([0] * n), cu=ints([0] * (n + 1)), used=ints([0] * n),
                            pos=torch.zeros(max(1, total), dtype=torch.int32, device=dev),
                            slots=torch.zeros(max(1, total), dtype=torch.int64, device=dev))
        st["mask"] = torch.zeros(max(1, total), _words(case), dtype=torch.int32, device=dev) if case["tree"] else None
    elif case["kind"] == "accept":
        paths = _branches(case)
        st.update(last=ints([p[-1] if p else -1 for p in paths]), used_out=torch.zeros_like(st["used"]),
                  accepted=torch.zeros_like(st["used"]),
                  path=torch.zeros(n, case["sq_max"], dtype=torch.int32, device=dev))
    elif case["tree"]:
        depth = ints([x for p in _trees(case) for x in _depths(p)])
        st["pos"] = depth + torch.repeat_interleave(st["ctx"], st["sq"].long())
        st["mask"] = _mask_words(case).to(dev)
    else:
        s, pos = _token_place(st)
        st["pos"] = pos.to(torch.int32)
    if case["kind"] == "rope":
        # A fused projection's rows: q, k and v of a token behind each other.
        st["qkv"] = torch.randn(total, hq + 2 * hk, d, generator=gen, device=dev, dtype=torch.bfloat16)
        st["q"], st["k_new"], st["v_new"] = st["qkv"].split([hq, hk, hk], 1)
        st["q_out"] = torch.zeros(total, hq, d, dtype=torch.bfloat16, device=dev)
        s, at = _token_place(st)
        st["slots"] = st["table"][s, at // b].long() * b + at % b
        st["freq"], st["magnitude"] = _frequencies(case)
        st["freq_dev"] = torch.tensor(st["freq"], dtype=torch.float64, device=dev)
        for name in ("k_cache", "v_cache"):
            st[name] = torch.zeros(blocks, b, hk, d, device=dev,
                                   dtype=torch.bfloat16 if case["kv"] == "bf16" else torch.uint8)
    elif case["kind"] in ("tree", "accept"):
        for name in ("k_cache", "v_cache"):
            st[name] = torch.randn(blocks, b, hk, d, generator=gen, device=dev, dtype=torch.bfloat16)
    if case["kind"] == "tree":
        st["q"] = torch.randn(total, hq, d, generator=gen, device=dev, dtype=torch.bfloat16)
        st["out"] = torch.zeros_like(st["q"])
        st["sinks"] = torch.randn(hq, generator=gen, device=dev) if case["sinks"] else None
        st["alibi"] = (torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], device=dev)
                       if case["alibi"] else None)
    if own:
        import paged_varlen_flash_gb300 as ua
        flags = ua.flags_of(True, case["softcap"], case["alibi"], case["window"], case["sinks"])
        st["flags"] = flags
        st["problem"] = p = ua.Problem(
            hq, hk, d, b, blocks, n, width, max(1, total), flags, st["scale"], case["softcap"], case["window"],
            kv_dtype=ua.UA_DTYPE_BF16 if case["kv"] == "bf16" else ua.UA_DTYPE_FP8_E4M3, k_scale=case["kscale"],
            v_scale=case["kscale"])
        if case["kind"] == "rope":
            p.set_rope(st["freq"], ua.UA_ROPE_HALF if case["layout"] == "half" else ua.UA_ROPE_PAIRS, st["magnitude"])
    return st


def _token_place(st):
    """Per packed token: its sequence and its key position."""
    s = torch.repeat_interleave(torch.arange(st["n"], device=st["sq"].device), st["sq"].long())
    t = torch.arange(st["total"], device=s.device)
    return s, st["ctx"].long()[s] + t - st["cu"].long()[s]


# ------------------------------------------------------------------ one pass
def run(state):
    return globals()["_" + state["case"]["kind"]](state)


def _plan(st):
    step, back, parents = st["step"], st["back"], st.get("parents")
    if own:
        p = st["problem"]
        p.plan_step(st["table"], st["held"], st["pool"], st["left"], st["ctx"], st["sq"], st["n"], st["total"],
                    step["granted"], step["cu"], step["used"], step["pos"], step["slots"], parents=parents,
                    tree_mask=st["mask"])
        p.plan_step(st["table"], st["held"], st["pool"], st["left"], st["ctx"], st["none"], st["n"], st["total"],
                    back["granted"], back["cu"], back["used"], back["pos"], back["slots"])
    else:
        _plan_plain(st, step, st["sq"], parents, st["mask"])
        _plan_plain(st, back, st["none"], None, None)
    return [step, st["table"], back, st["held"], st["pool"], st["left"]] + ([st["mask"]] if st["mask"] is not None else [])


def _ancestors(st):
    """bool [n, m, m], m whole words of 32: node i's ancestors and itself."""
    m = 32 * _words(st["case"])
    up = torch.nn.functional.pad(st["parents"], (0, m - st["parents"].shape[1]), value=-1)
    eye = torch.eye(m, dtype=torch.float64, device=up.device)
    # Steps to a parent or none: after m of them every ancestor has been reached.
    return torch.linalg.matrix_power((up[..., None] == torch.arange(m, device=up.device)).double() + eye, m) > 0


def _starts(x):
    return torch.cumsum(x, 0) - x


def _plan_plain(st, out, new, parents, mask):
    b, table, dev = st["b"], st["table"], st["table"].device
    ctx, new, held, left = st["ctx"].long(), new.long(), st["held"].long(), st["left"].long()
    need = (ctx + new + b - 1) // b
    more, back = (need - held).clamp(min=0), (held - need).clamp(min=0)
    ok = (more == 0) | (torch.cumsum(more, 0) <= left + back.sum())
    more, new = more * ok, new * ok
    # Returned blocks, the last one lowest, on top of the pool; taken ones from the top down.
    order = torch.arange(st["n"], device=dev)
    s = torch.repeat_interleave(order, back)
    i = torch.arange(len(s), device=dev)
    returned = table[s, need[s] + i - _starts(back)[s]]
    stack = torch.cat([st["pool"][:left], returned.flip(0)])
    s = torch.repeat_interleave(order, more)
    i = torch.arange(len(s), device=dev)
    table[s, held[s] + i - _starts(more)[s]] = stack[len(stack) - 1 - i]
    rest = len(stack) - len(s)
    st["pool"][:rest] = stack[:rest]
    st["left"].fill_(rest)
    st["held"].copy_(held + more - back)
    out["granted"].copy_(new)
    out["cu"][1:] = torch.cumsum(new, 0)
    out["used"].copy_(ctx + new)
    s = torch.repeat_interleave(order, new)
    i = torch.arange(len(s), device=dev) - _starts(new)[s]
    depth = i
    if parents is not None:
        line = _ancestors(st)[s, i]                                 # a token's nodes
        depth = line.sum(-1) - 1
        mask[:len(s)] = (line.long().unflatten(-1, (-1, 32)) << torch.arange(32, device=dev)).sum(-1).to(torch.int32)
    at = ctx[s] + i
    out["pos"].zero_()
    out["pos"][:len(s)] = (ctx[s] + depth).to(torch.int32)
    out["slots"].fill_(-1)
    out["slots"][:len(s)] = table[s, at // b].long() * b + at % b


def _rope(st):
    if own:
        st["problem"].rope_store(st["q"], st["k_new"], st["v_new"], st["pos"], st["slots"], st["total"], st["k_cache"],
                                 st["v_cache"], q_out=st["q_out"])
    else:
        angle = st["pos"].double()[:, None] * st["freq_dev"]
        c, s = (x.float()[:, None] * st["magnitude"] for x in (torch.cos(angle), torch.sin(angle)))
        st["q_out"].copy_(_rotated(st, st["q"].float(), c, s))
        for x, cache in ((_rotated(st, st["k_new"].float(), c, s).to(torch.bfloat16), st["k_cache"]), (st["v_new"], st["v_cache"])):
            if cache.dtype == torch.uint8:
                x = (x.float() / st["case"]["kscale"]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
            cache.view(-1, st["hk"], st["d"])[st["slots"]] = x
    kind = torch.float8_e4m3fn if st["case"]["kv"] == "fp8" else torch.bfloat16
    return [st["q_out"], st["k_cache"].view(kind), st["v_cache"].view(kind)]


def _rotated(st, x, c, s):
    rot = st["case"]["rot"]
    if st["case"]["layout"] == "half":
        a, z = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * c - z * s, a * s + z * c], -1)
    else:
        a, z = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - z * s, a * s + z * c], -1).flatten(-2)
    return torch.cat([turned, x[..., rot:]], -1)


def _rows_fp32(st, name):
    """The batch's cached rows, padded: fp32 [n, hk, max_k, d]."""
    pages = st[name][st["table"].clamp(min=0).long()].float()
    return pages.permute(0, 3, 1, 2, 4).flatten(2, 3)[:, :, :st["max_k"]]


def _tree(st):
    if own:
        return st["problem"].forward_tree(
            st["q"], st["k_cache"], st["v_cache"], st["table"], st["cu"], st["used"], st["n"], st["total"], st["max_q"],
            st["max_k"], st["flags"], st["mask"], positions=st["pos"], sinks=st["sinks"], alibi_slopes=st["alibi"],
            out=st["out"])
    case, n, hk, g, mq, mk = st["case"], st["n"], st["hk"], st["hq"] // st["hk"], st["max_q"], st["max_k"]
    dev = st["q"].device
    cu, ctx, sq = st["cu"].long(), st["ctx"].long(), st["sq"].long()
    i, j = torch.arange(mq, device=dev), torch.arange(mk, device=dev)
    tok = (cu[:-1, None] + i).clamp(max=st["total"] - 1)
    q = st["q"][tok].float().unflatten(2, (hk, g)).permute(0, 2, 3, 1, 4)   # n, hk, g, mq, d
    x = torch.matmul(q.flatten(2, 3) * st["scale"], _rows_fp32(st, "k_cache").transpose(-1, -2)).unflatten(2, (g, mq))
    if case["softcap"]:
        x = case["softcap"] * torch.tanh(x / case["softcap"])
    c = j - ctx[:, None]                                          # n, mk: the key's node
    inside = (c >= 0) & (c < sq[:, None])
    pos = torch.where(inside, st["pos"].long()[(cu[:-1, None] + c).clamp(0, st["total"] - 1)], j)
    if case["alibi"]:
        x = x + st["alibi"].view(1, hk, g, 1, 1) * (pos - ctx[:, None]).view(n, 1, 1, 1, mk)
    node = c.clamp(0, 32 * st["mask"].shape[1] - 1)
    word = st["mask"].long()[tok].gather(2, (node // 32)[:, None].expand(n, mq, mk))
    see = (word >> (node % 32)[:, None] & 1).bool() & inside[:, None] | (c < 0)[:, None]
    see = see & (i < sq[:, None])[..., None]
    if case["window"]:
        see = see & (pos[:, None] > st["pos"].long()[tok][..., None] - case["window"])
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
    o = torch.matmul(p.flatten(2, 3), _rows_fp32(st, "v_cache")).unflatten(2, (g, mq)) / total.masked_fill(total == 0, 1.0)
    s, at = _token_place(st)
    return o.permute(0, 3, 1, 2, 4).flatten(2, 3)[s, at - ctx[s]].to(torch.bfloat16)


def _accept(st):
    outs = [st["k_cache"], st["v_cache"], st["path"], st["accepted"], st["used_out"]]
    if own:
        st["problem"].cache_accept(st["k_cache"], st["v_cache"], st["table"], st["cu"], st["used"], st["parents"],
                                   st["last"], st["n"], st["total"], st["max_q"], st["max_k"], st["path"],
                                   st["accepted"], st["used_out"])
        return outs
    dev = st["table"].device
    order = torch.arange(st["n"], device=dev)
    last = st["last"].long()
    on = _ancestors(st)[order, last.clamp(min=0)] & (last >= 0)[:, None]
    s, node = torch.nonzero(on, as_tuple=True)                      # ascending nodes of a sequence: its branch
    count = on.sum(1)
    t = torch.arange(len(s), device=dev) - _starts(count)[s]
    st["path"].fill_(-1)
    st["path"][s, t] = node.to(torch.int32)
    ctx = st["ctx"].long()[s]
    frm, to = ctx + node, ctx + t
    b = st["b"]
    for cache in outs[:2]:
        cache[st["table"][s, to // b].long(), to % b] = cache[st["table"][s, frm // b].long(), frm % b]
    st["accepted"].copy_(count)
    st["used_out"].copy_(st["ctx"] + count)
    return outs


# ------------------------------------------------------------------ 64 bits
def _e4m3_nearest(y):
    """The nearest e4m3 value (ties to even, at most 448) of float64 values."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3.0)
    return torch.sign(y) * torch.round(a / step) * step


def exact(case, seed):
    if case["kind"] == "plan":
        return None                      # whole numbers: held to the plain form
    st = prepare(case, seed)
    dev, b, hk, d = st["table"].device, st["b"], st["hk"], st["d"]
    sq, ctx = _lengths(case)
    if case["kind"] == "accept":
        outs = [st["k_cache"].double(), st["v_cache"].double()]
        for s, path in enumerate(_branches(case)):
            for t, r in enumerate(path):
                frm, to = ctx[s] + r, ctx[s] + t
                if r != t:
                    for cache, o in zip((st["k_cache"], st["v_cache"]), outs):
                        o[int(st["table"][s, to // b]), to % b] = cache[int(st["table"][s, frm // b]), frm % b].double()
        return outs + [None, None, None]
    if case["kind"] == "rope":
        rot = case["rot"]
        freq = torch.tensor(st["freq"], dtype=torch.float64, device=dev)
        outs = [torch.empty(st["total"], st["hq"], d, dtype=torch.float64, device=dev)]
        outs += [torch.zeros(st["blocks"] * b, hk, d, dtype=torch.float64, device=dev) for _ in range(2)]
        step = max(1, (1 << 25) // (st["hq"] * d))
        for t in range(0, st["total"], step):
            phase = torch.polar(torch.full((1,), st["magnitude"], dtype=torch.float64, device=dev),
                                st["pos"][t:t + step].double()[:, None] * freq)[:, None]
            for k, x in enumerate((st["q"], st["k_new"])):
                x = x[t:t + step].double()
                y = x.clone()
                if case["layout"] == "half":
                    z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * phase
                    y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
                else:
                    z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * phase
                    y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
                if k == 0:
                    outs[0][t:t + step] = y
                elif case["kv"] == "fp8":     # what is stored is the bf16 value in 8 bits
                    outs[1][st["slots"][t:t + step]] = _e4m3_nearest(y.to(torch.bfloat16).double() / case["kscale"])
                else:
                    outs[1][st["slots"][t:t + step]] = y
            v = st["v_new"][t:t + step].double()
            outs[2][st["slots"][t:t + step]] = _e4m3_nearest(v / case["kscale"]) if case["kv"] == "fp8" else v
        return outs
    out = torch.zeros(st["total"], st["hq"], d, dtype=torch.float64, device=dev)
    g, t0 = st["hq"] // hk, 0
    for s, parents in enumerate(_trees(case)):
        depth = _depths(parents)
        at = torch.tensor(list(range(ctx[s])) + [ctx[s] + x for x in depth], device=dev)     # positions of the keys
        see = torch.zeros(sq[s], ctx[s] + sq[s], dtype=torch.bool)
        see[:, :ctx[s]] = True
        for i, q in enumerate(parents):
            if q >= 0:
                see[i, ctx[s]:] = see[q, ctx[s]:]
            see[i, ctx[s] + i] = True
        see = see.to(dev)
        if case["window"]:
            see &= at[None] > at[ctx[s]:, None] - case["window"]
        j = torch.arange(ctx[s] + sq[s], device=dev)
        block, slot = st["table"][s, j // b].long(), j % b
        for h in range(hk):
            k, v = (st[x][block, slot, h].double() for x in ("k_cache", "v_cache"))
            for e in range(h * g, h * g + g):
                x = st["q"][t0:t0 + sq[s], e].double() @ k.T * st["scale"]
                if case["softcap"]:
                    x = case["softcap"] * torch.tanh(x / case["softcap"])
                if case["alibi"]:
                    x = x + st["alibi"][e].double() * (at - ctx[s])[None]
                x = x.masked_fill(~see, -math.inf)
                lse = torch.logsumexp(x, -1)
                if case["sinks"]:
                    lse = torch.logaddexp(lse, st["sinks"][e].double().expand_as(lse))
                out[t0:t0 + sq[s], e] = torch.exp(x - lse[:, None]) @ v
        t0 += sq[s]
    return out
