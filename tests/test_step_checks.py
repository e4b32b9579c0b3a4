"""What the calls of a speculative decoding step refuse before anything is launched,
the rotary frequencies, and the plain implementations against hand-made examples.
CPU only."""
import math

import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests import step_ref as S
from tests.test_binding_checks import elsewhere, reaches_the_library
from tests.test_problem_create import run  # noqa: F401

N, HQ, HK, D, B, WIDTH, BLOCKS, T = 3, 8, 2, 64, 16, 4, 20, 9


# ---------------------------------------------------------------- the library's refusals
def test_calls_that_the_library_refuses(run):
    run("""
CAUSAL = ua.UA_FLAG_CAUSAL
p = create(flags=CAUSAL | ua.UA_FLAG_SINKS | ua.UA_FLAG_ALIBI | ua.UA_FLAG_WINDOW | ua.UA_FLAG_QQ_BIAS, window=9)
A = 1 << 12                                   # an address that only the checks look at

def plan(p=p, table=A, held=A, pool=A, left=A, ctx=A, new=A, parents=A, pstride=8, n=2, cap=8, granted=A, cu=A, used=A,
         pos=A, slots=A, mask=A, words=1):
    return ua.ua_plan_step(p, table, held, pool, left, ctx, new, parents, pstride, n, cap, granted, cu, used, pos, slots,
                           mask, words, stream=0)

def rope(p=p, q=A, qs=1024, k=A, v=A, kvs=256, pos=A, slots=A, n=2, out=2 * A, outs=1024, kc=A, vc=A):
    return ua.ua_rope_store(p, q, qs, k, v, kvs, pos, slots, n, out, outs, kc, vc, stream=0)

def tree(p=p, q=A, k=A, v=A, table=A, cu=A, used=A, n=2, total=8, max_q=4, max_k=40, mask=A, words=1, pos=A,
         flags=CAUSAL | ua.UA_FLAG_SINKS | ua.UA_FLAG_ALIBI | ua.UA_FLAG_WINDOW, sinks=A, alibi=A, out=A):
    return ua.ua_forward_tree(p, q, k, v, table, cu, used, n, total, max_q, max_k, mask, words, pos, flags, sinks, alibi,
                              out, stream=0)

def accept(p=p, k=A, v=A, table=A, cu=A, used=A, parents=A, pstride=4, last=A, n=2, total=8, max_q=4, max_k=40, path=A,
           path_stride=4, accepted=A, used_out=A):
    return ua.ua_cache_accept(p, k, v, table, cu, used, parents, pstride, last, n, total, max_q, max_k, path, path_stride,
                              accepted, used_out, stream=0)

# Before ua_set_rope there is nothing to rotate by.
assert rope() == 1
for n, layout, magnitude, freq, want in ((8, 0, 1.0, 0.5, 0), (64, 1, 1.25, 1.0, 0), (0, 0, 1.0, 1.0, 1), (12, 0, 1.0, 1.0, 2),
                                         (72, 0, 1.0, 1.0, 2), (8, 2, 1.0, 1.0, 1), (8, 0, float("inf"), 1.0, 1),
                                         (8, 0, 1.0, -0.1, 1), (8, 0, 1.0, float("nan"), 1), (8, 0, 1.0, 6.5, 1), (8, 0, 1.0, 6.0, 0)):
    assert ua.ua_set_rope(p, [freq] * n, layout, magnitude) == want, (n, layout, magnitude, freq)
assert ua.ua_set_rope(None, [1.0] * 8) == 1

# A call that passes the checks ends in a CUDA error here.
for call in (plan, rope, tree, accept):
    assert call() == 3, (call.__name__, call())
    assert call(p=None) == 1
    names = call.__code__.co_varnames[1:call.__code__.co_argcount]
    pointers = [x for x, d in zip(names, call.__defaults__[1:]) if d in (A, 2 * A)]
    optional = {"plan": ("parents", "mask"), "tree": ("pos", "sinks", "alibi")}.get(call.__name__, ())
    for name in pointers:
        if name not in optional:
            assert call(**{name: None}) == 1, (call.__name__, name)
        wide = name in ("q", "k", "v", "kc", "vc", "out")
        for off in ((2, 8) if wide else (4,) if name == "slots" else (1, 2, 3)):
            assert call(**{name: A + off}) == 1, (call.__name__, name, off)

# ua_plan_step
for bad in (dict(n=-1), dict(n=5), dict(cap=-1), dict(cap=65), dict(pstride=0), dict(words=0)):
    assert plan(**bad) == 1, bad
assert plan(n=0, cap=0, table=None, held=None, pool=None, left=None, ctx=None, new=None, granted=None, cu=None,
            used=None) == 0
assert plan(cap=0, pos=None, slots=None) == 3
assert plan(parents=None, pstride=0, mask=None, words=0) == 3
many = create(max_num_seqs=20000)
assert plan(p=many, n=16385) == 2 and plan(p=many, n=16384) == 3

# ua_rope_store
for bad in (dict(n=-1), dict(n=65), dict(qs=1016), dict(qs=1028), dict(kvs=248), dict(kvs=260), dict(outs=1016),
            dict(outs=1025), dict(out=A, outs=1032)):
    assert rope(**bad) == 1, bad
assert rope(n=0, q=None) == 0
assert rope(out=A) == 3                       # in place

# ua_forward_tree
for bad in (dict(flags=ua.UA_FLAG_SINKS, alibi=None), dict(pos=None), dict(words=0), dict(max_q=40, max_k=40, total=40),
            dict(sinks=None), dict(flags=CAUSAL), dict(flags=CAUSAL | ua.UA_FLAG_SOFTCAP, sinks=None, alibi=None)):
    assert tree(**bad) == 1, bad
plain = dict(flags=CAUSAL, sinks=None, alibi=None)
assert tree(pos=None, **plain) == 3
assert tree(n=0, **plain) == 0 and tree(total=0, **plain) == 0
assert ua.ua_forward_tree(p, A, A, A, A, A, A, 2, 8, 4, 40, A, 1, A, CAUSAL | ua.UA_FLAG_QQ_BIAS, None, None, A, stream=0) == 1
for kind in (ua.UA_DTYPE_FP8_E4M3, ua.UA_DTYPE_FP4_E2M1):
    packed = create(kv_dtype=kind)
    assert tree(p=packed, mask=None, **plain) == 1 and tree(p=packed, n=0, **plain) == 0
    ua.ua_destroy(packed)
assert tree(p=create(path=ua.UA_PATH_SPLIT_KV), **plain) == 2
big = create(max_total_q=4096, max_blocks_per_seq=300)
assert tree(p=big, total=2000, max_q=1025, max_k=2000, words=33, **plain) == 2
assert tree(p=big, total=2000, max_q=1024, max_k=2000, words=32, **plain) == 3
assert tree(p=create(num_q_heads=256, num_kv_heads=1), **plain) == 2

# ua_cache_accept
for bad in (dict(n=-1), dict(n=5), dict(total=65), dict(max_q=41), dict(max_k=129), dict(pstride=3), dict(path_stride=0)):
    assert accept(**bad) == 1, bad
assert accept(n=0, k=None) == 0
assert accept(p=big, max_q=1025, max_k=2000, pstride=1025) == 2
""")


def test_a_tree_problem_has_room_for_every_share(run):
    run("""
def work(**kw):
    before = fake.fake_allocated()
    ua.ua_destroy(create(max_total_q=64, **kw))
    return fake.fake_allocated() - before
# 304 shares of two partials of 128 rows (152 at d = 256); not for key weights, whose size is documented.
assert work(num_q_heads=64, num_kv_heads=8) >= 608 * 128 * 130 * 4
assert work(num_q_heads=64, num_kv_heads=8, head_size=256) >= 304 * 128 * 258 * 4
assert work(num_q_heads=64, num_kv_heads=8, flags=ua.UA_FLAG_CAUSAL | ua.UA_FLAG_KEY_WEIGHTS) < work(num_q_heads=64, num_kv_heads=8)
""")


# ---------------------------------------------------------------- the binding's refusals
@pytest.fixture()
def p():
    x = ua.Problem.__new__(ua.Problem)
    x.handle = None
    x.flags, x.head_size, x.num_q_heads, x.num_kv_heads = ua.UA_FLAG_CAUSAL, D, HQ, HK
    x.block_size, x.max_blocks_per_seq, x.num_blocks = B, WIDTH, BLOCKS
    return x


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bad_vectors(n, kind=torch.int32):
    other = torch.int64 if kind is torch.int32 else torch.int32
    yield torch.zeros(n - 1, dtype=kind)
    yield torch.zeros(n, dtype=other)
    if n > 1:
        yield torch.zeros(2 * n, dtype=kind)[::2]
    yield elsewhere(torch.zeros(n, dtype=kind))


def check_calls(call, vectors, others):
    reaches_the_library(call)
    for name, (n, kind) in vectors.items():
        for bad in bad_vectors(n, kind):
            with pytest.raises(ValueError):
                call(**{name: bad})
    for name, bads in others.items():
        for bad in bads:
            with pytest.raises(ValueError):
                call(**{name: bad})


def test_plan_step_arguments(p):
    good = dict(block_table=i32(N, WIDTH), blocks_held=i32(N), free_blocks=i32(BLOCKS), free_count=i32(1), ctx_lens=i32(N),
                new_lens=i32(N), num_seqs=N, max_tokens=T, granted=i32(N), cu_seqlens_q=i32(N + 1), seqused_k=i32(N),
                positions=i32(T), slots=torch.zeros(T, dtype=torch.int64), parents=i32(N, 5), tree_mask=i32(T, 2), stream=0)

    def call(**over):
        p.plan_step(**{**good, **over})

    check_calls(call, {**{k: (N, torch.int32) for k in ("blocks_held", "ctx_lens", "new_lens", "granted", "seqused_k")},
                       "free_blocks": (BLOCKS, torch.int32), "free_count": (1, torch.int32),
                       "cu_seqlens_q": (N + 1, torch.int32), "positions": (T, torch.int32), "slots": (T, torch.int64)},
                dict(block_table=[i32(N, WIDTH + 1), i32(N - 1, WIDTH), i32(N, 2 * WIDTH)[:, ::2], i32(N * WIDTH),
                                  torch.zeros(N, WIDTH, dtype=torch.int64)],
                     parents=[i32(N - 1, 5), i32(5, N).T, i32(N), torch.zeros(N, 5), elsewhere(i32(N, 5)), i32(1, 5).expand(N, 5)],
                     tree_mask=[i32(T - 1, 2), i32(2, T).T, i32(T), i32(T, 4)[:, :2], torch.zeros(T, 2), elsewhere(i32(T, 2))]))
    reaches_the_library(call, parents=None, tree_mask=None)
    reaches_the_library(call, parents=i32(N + 2, 9)[:, :5])


def test_rope_store_arguments(p):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = bf(BLOCKS, B, HK, D)
    good = dict(q=bf(T, HQ, D), k_new=bf(T, HK, D), v_new=bf(T, HK, D), positions=i32(T),
                slots=torch.zeros(T, dtype=torch.int64), total_q=T, k_cache=cache, v_cache=cache.clone(),
                q_out=bf(T, HQ, D), stream=0)

    def call(**over):
        p.rope_store(**{**good, **over})

    rows = lambda h: [bf(T - 1, h, D), bf(T, h + 1, D), bf(T, h, D // 2), bf(T, D, h).transpose(1, 2), torch.zeros(T, h, D),  # noqa: E731
                      elsewhere(bf(T, h, D)), bf(T, 2 * h, D)[:, ::2]]
    check_calls(call, {"positions": (T, torch.int32), "slots": (T, torch.int64)},
                dict(q=rows(HQ), q_out=rows(HQ), k_new=rows(HK), v_new=rows(HK) + [bf(T, 2 * HK, D)[:, :HK]]))
    fused = bf(T, HQ + 2 * HK, D)
    q, k, v = fused.split([HQ, HK, HK], 1)
    reaches_the_library(call, q=q, k_new=k, v_new=v, q_out=q)
    reaches_the_library(call, q_out=None)


def test_forward_tree_arguments(p):
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = bf(BLOCKS, B, HK, D)

    def call(tree_mask=i32(T, 1), positions=i32(T)):
        p.forward_tree(bf(T, HQ, D), cache, cache, i32(N, WIDTH), i32(N + 1), i32(N), N, T, 5, 50, ua.UA_FLAG_CAUSAL, tree_mask,
                       positions=positions, stream=0)

    check_calls(call, {"positions": (T, torch.int32)},
                dict(tree_mask=[i32(T - 1, 1), i32(T), i32(T, 2)[:, :1], torch.zeros(T, 1), elsewhere(i32(T, 1))]))
    reaches_the_library(call, tree_mask=torch.zeros(T, 1, dtype=torch.uint32), positions=None)


def test_cache_accept_arguments(p):
    cache = torch.zeros(BLOCKS, B, HK, D, dtype=torch.bfloat16)
    good = dict(cu_seqlens_q=i32(N + 1), seqused_k=i32(N), parents=i32(N, 5), last=i32(N), path=i32(N, 5), accepted=i32(N),
                seqused_out=i32(N))

    def call(**over):
        x = {**good, **over}
        p.cache_accept(cache, cache, i32(N, WIDTH), x["cu_seqlens_q"], x["seqused_k"], x["parents"], x["last"], N, T, 5, 50,
                       x["path"], x["accepted"], x["seqused_out"], stream=0)

    check_calls(call, {**{k: (N, torch.int32) for k in ("seqused_k", "last", "accepted", "seqused_out")},
                       "cu_seqlens_q": (N + 1, torch.int32)},
                dict(parents=[i32(N, 4), i32(N - 1, 5), i32(5, N).T, torch.zeros(N, 5), elsewhere(i32(N, 5))],
                     path=[i32(N + 1, 5), i32(N), i32(N, 6)[:, :5], i32(N, 0), torch.zeros(N, 5), elsewhere(i32(N, 5))]))


def test_rows_and_tables_of_tree_calls(p):
    """q is packed (a view of a fused projection has other strides), tables have the
    problem's width."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    cache = bf(BLOCKS, B, HK, D)
    good = dict(q=bf(T, HQ, D), table=i32(N, WIDTH), cu=i32(N + 1), used=i32(N), out=bf(T, HQ, D))

    def tree(**over):
        x = {**good, **over}
        p.forward_tree(x["q"], cache, cache, x["table"], x["cu"], x["used"], N, T, 5, 50, ua.UA_FLAG_CAUSAL, i32(T, 1),
                       out=x["out"], stream=0)

    rows = [bf(T, HQ + 2, D)[:, :HQ], bf(T - 1, HQ, D), torch.zeros(T, HQ, D), elsewhere(bf(T, HQ, D))]
    tables = [i32(N, WIDTH + 1), i32(N - 1, WIDTH), i32(N, 2 * WIDTH)[:, ::2], torch.zeros(N, WIDTH, dtype=torch.int64)]
    check_calls(tree, {"cu": (N + 1, torch.int32), "used": (N, torch.int32)}, dict(q=rows, out=rows, table=tables))
    reaches_the_library(tree, out=None)

    def accept(table=i32(N, WIDTH)):
        p.cache_accept(cache, cache, table, i32(N + 1), i32(N), i32(N, 5), i32(N), N, T, 5, 50, i32(N, 5), i32(N), i32(N),
                       stream=0)

    check_calls(accept, {}, dict(table=tables))


# ---------------------------------------------------------------- frequencies
def test_rope_frequencies():
    plain, one = ua.rope_frequencies(64)
    assert one == 1.0 and len(plain) == 32 and plain[0] == 1.0 and plain[16] == 0.01
    assert ua.rope_frequencies(64, scaling="linear", factor=4.0)[0] == [f / 4 for f in plain]
    ntk, _ = ua.rope_frequencies(64, scaling="ntk", factor=8.0)
    assert ntk[0] == 1.0 and math.isclose(ntk[31], plain[31] / 8, rel_tol=1e-12)
    bands, _ = ua.rope_frequencies(64, scaling="bands", factor=8.0, trained=8192, low=1.0, high=4.0)
    for f, b in zip(plain, bands):
        turns = 8192 * f / (2 * math.pi)
        assert b == f if turns >= 4 else b == f / 8 if turns <= 1 else f / 8 < b < f
    yarn, m = ua.rope_frequencies(64, scaling="yarn", factor=16.0, trained=4096, low=1.0, high=32.0)
    assert math.isclose(m, 0.1 * math.log(16) + 1) and yarn[0] == 1.0 and math.isclose(yarn[31], plain[31] / 16)
    assert all(p / 16 <= y <= p for p, y in zip(plain, yarn)) and any(p / 16 < y < p for p, y in zip(plain, yarn))
    assert ua.rope_frequencies(64, scaling="yarn", factor=1.0, trained=4096)[1] == 1.0
    for bad in (dict(rotated=63), dict(rotated=0), dict(rotated=64, scaling="other"), dict(rotated=64, scaling="bands"),
                dict(rotated=64, scaling="yarn", trained=10, low=3.0, high=2.0), dict(rotated=64, factor=0.0),
                dict(rotated=2, scaling="ntk")):
        with pytest.raises(ValueError):
            ua.rope_frequencies(**bad)


# ---------------------------------------------------------------- the plain implementations
def test_reference_plan_by_hand():
    st = S.Step([[5, 6, -1], [7, -1, -1]], [2, 1], [1, 2, 3], 16, 10)
    out, err = st.plan([10, 16], [1, 17], 18, None, 0)        # the first needs one block and gives one back
    assert err == 0 and out["granted"] == [1, 17] and out["cu"] == [0, 1, 18] and out["used"] == [11, 33]
    assert st.held == [1, 3] and st.table[1] == [7, 6, 3] and st.pool == [1, 2]
    assert out["slots"][:2] == [5 * 16 + 10, 6 * 16] and out["slots"][-1] == 3 * 16 and out["pos"] == [10] + list(range(16, 33))


def test_reference_trees_by_hand():
    tree = [-1, 0, 0, 1, -1]
    assert S.branch(tree, 3) == [0, 1, 3] and S.branch(tree, -1) == [] and S.depths(tree) == [0, 1, 1, 2, 0]
    assert S.mask_of(tree, 1)[:, 0].tolist() == [1, 3, 5, 11, 16]


def test_reference_rotation_keeps_lengths_and_composes():
    g = np.random.default_rng(3)
    x = g.normal(size=(4, 2, 16))
    freq = [0.7, 0.01, 0.3]
    for pairs in (False, True):
        y = S.rotate(x, [5, 0, 123456, 9], freq, pairs)
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1)) and np.array_equal(y[1], x[1])
        assert np.allclose(S.rotate(S.rotate(x, [2] * 4, freq, pairs), [3] * 4, freq, pairs), S.rotate(x, [5] * 4, freq, pairs))
    # Far positions: the angle modulo a turn, against exact arithmetic of the same double.
    assert abs(S._fraction(2 ** 31 - 1, 1.0) - math.fmod(2 ** 31 - 1, 2 * math.pi)) < 1e-6


def test_reference_attention_of_a_chain_is_causal_attention():
    from tests import cache_ref as R
    g = np.random.default_rng(4)
    q, k, v = g.normal(size=(6, 4, 8)), g.normal(size=(20, 2, 8)), g.normal(size=(20, 2, 8))
    chain = np.tril(np.ones((6, 6), bool))
    kw = dict(softcap=3.0, window=7, sinks=np.array([0.1, 2.0, -np.inf, np.inf]), alibi=np.array([.5, .25, .1, 0.]))
    want = R.attention(q, k, v, 0.4, **kw)[0]
    assert np.allclose(S.tree_attention(q, k, v, 0.4, chain, pos=np.arange(14, 20), **kw)[0], want, atol=1e-12)
