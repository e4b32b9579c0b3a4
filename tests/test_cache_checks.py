"""What the calls of ``Problem`` refuse of caches, and the step calls of sinks and slopes, that
the kernels would read or write past.  CPU only: the problem has no handle, so that a call whose arguments
pass ends in the library's "invalid argument"."""
import math

import pytest
import torch

import paged_varlen_flash_gb300 as ua
from tests.test_binding_checks import _built, elsewhere, reaches_the_library  # noqa: F401

N, HQ, HK, D, B, WIDTH, BLOCKS, T = 3, 8, 2, 128, 16, 4, 20, 9
KINDS = {ua.UA_DTYPE_BF16: torch.bfloat16, ua.UA_DTYPE_FP8_E4M3: torch.uint8, ua.UA_DTYPE_FP4_E2M1: torch.uint8}


def problem(kind, known=True):
    """A problem of that cache type, with what __init__ notes beside the handle (or without)."""
    x = ua.Problem.__new__(ua.Problem)
    x.handle, x.kv_dtype = None, kind
    x.flags, x.head_size, x.num_q_heads, x.num_kv_heads = ua.UA_FLAG_CAUSAL, D, HQ, HK
    x.block_size, x.max_blocks_per_seq, x.num_blocks = B, WIDTH, BLOCKS
    if known:
        x._cache_shape = ua.cache_shape(BLOCKS, HK, D, B, kind)
        x._cache_bytes = math.prod(x._cache_shape) * KINDS[kind].itemsize
    return x


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def calls(p):
    rows = i32(N, WIDTH), i32(N + 1), i32(N)
    return [
        lambda k, v: p.rope_store(bf(T, HQ, D), bf(T, HK, D), bf(T, HK, D), i32(T), torch.zeros(T, dtype=torch.int64), T, k, v,
                                  q_out=bf(T, HQ, D), stream=0),
        lambda k, v: p.forward_tree(bf(T, HQ, D), k, v, *rows, N, T, 5, 50, ua.UA_FLAG_CAUSAL, i32(T, 1), stream=0),
        lambda k, v: p.cache_accept(k, v, *rows, i32(N, 5), i32(N), N, T, 5, 50, i32(N, 5), i32(N), i32(N), stream=0),
    ]


def bad_caches(kind):
    shape, dtype = ua.cache_shape(BLOCKS, HK, D, B, kind), KINDS[kind]
    make = lambda *s, t=dtype: torch.zeros(*s, dtype=t)  # noqa: E731
    yield make(shape[0] - 1, *shape[1:])                       # too few blocks
    yield make(*shape[:-1], shape[-1] // 2)
    yield make(shape[0] * shape[1], *shape[2:])                # another layout
    yield make(*shape[:-1], 2 * shape[-1])[..., ::2]
    yield make(*shape, t=torch.float32)
    yield make(*shape, t=torch.uint8 if dtype is torch.bfloat16 else torch.bfloat16)
    yield make(*shape, t=torch.float16)
    yield elsewhere(make(*shape))


@pytest.mark.parametrize("known", [True, False])
@pytest.mark.parametrize("kind", list(KINDS))
def test_caches_of_step_calls(kind, known):
    p = problem(kind, known)
    shape, dtype = ua.cache_shape(BLOCKS, HK, D, B, kind), KINDS[kind]
    good = torch.zeros(*shape, dtype=dtype)
    more = torch.zeros(shape[0] + 3, *shape[1:], dtype=dtype)
    for call in calls(p):
        for k, v in ((good, good.clone()), (more, more), (good, more), (more, good), (more[1:], more[3:])):
            reaches_the_library(lambda: call(k, v))
        if kind == ua.UA_DTYPE_FP8_E4M3:
            reaches_the_library(lambda: call(good.view(torch.float8_e4m3fn), good))
        for bad in bad_caches(kind):
            for k, v in ((bad, good), (good, bad), (bad, bad)):
                with pytest.raises(ValueError):
                    call(k, v)


def test_sinks_and_slopes_of_tree_calls():
    p = problem(ua.UA_DTYPE_BF16)
    cache = bf(BLOCKS, B, HK, D)

    def call(sinks=None, alibi_slopes=None):
        p.forward_tree(bf(T, HQ, D), cache, cache, i32(N, WIDTH), i32(N + 1), i32(N), N, T, 5, 50, ua.UA_FLAG_CAUSAL, i32(T, 1),
                       positions=i32(T), sinks=sinks, alibi_slopes=alibi_slopes, stream=0)

    for good in (None, torch.zeros(HQ), torch.zeros(HQ + 2)):
        reaches_the_library(call, sinks=good, alibi_slopes=good)
    for bad in (torch.zeros(HQ - 1), torch.zeros(HQ, dtype=torch.float64), bf(HQ), torch.zeros(2 * HQ)[::2],
                elsewhere(torch.zeros(HQ))):
        for name in ("sinks", "alibi_slopes"):
            with pytest.raises(ValueError):
                call(**{name: bad})


def other_calls(p):
    rows = i32(N, WIDTH), i32(N + 1), i32(N)
    w, pages = torch.zeros(N, HK, 50), bf(4, B, HK, D)
    return [
        lambda k, v: p.forward(bf(T, HQ, D), k, v, *rows, N, T, 5, 50, ua.UA_FLAG_CAUSAL, stream=0),
        lambda k, v: p.forward_topk(bf(T, HQ, D), k, v, *rows, N, T, 5, 50, i32(T, 8), i32(T), ua.UA_FLAG_CAUSAL, stream=0),
        lambda k, v: p.forward_weights(bf(T, HQ, D), k, v, *rows, N, T, 5, 50, ua.UA_FLAG_CAUSAL, None, w, stream=0),
        lambda k, v: p.cache_store(bf(T, HK, D), bf(T, HK, D), k, v, *rows, N, T, 5, 50, stream=0),
        lambda k, v: p.cache_expand(k, v, rows[0], rows[2], N, 50, pages, pages, rows[0], stream=0),
        lambda k, v: p.cache_evict(k, v, rows[0], rows[2], N, 50, w, w, 10, 2, i32(N, HK, 10), i32(N), stream=0),
    ]


@pytest.mark.parametrize("kind", list(KINDS))
def test_caches_of_the_other_calls(kind):
    """Whatever their shape, they are as long as the problem's."""
    p = problem(kind)
    shape, dtype = ua.cache_shape(BLOCKS, HK, D, B, kind), KINDS[kind]
    good = torch.zeros(*shape, dtype=dtype)
    for call in other_calls(p):
        for k, v in ((good, good), (good.flatten(), good.view(torch.uint8)), (torch.cat([good, good]), good)):
            reaches_the_library(lambda: call(k, v))
        for bad in (good[1:], good.flatten()[1:], torch.cat([good, good], -1)[..., ::2], torch.cat([good, good], 1)[:, ::2]):
            for k, v in ((bad, good), (good, bad)):
                with pytest.raises(ValueError):
                    call(k, v)
    # Addresses say nothing about what is behind them.
    a = 1 << 12
    reaches_the_library(lambda: p.forward(a, a, a, a, a, a, N, T, 5, 50, ua.UA_FLAG_CAUSAL, out=a, stream=0))


def test_what_a_problem_knows_of_its_caches(monkeypatch):
    monkeypatch.setattr(ua.binding, "ua_problem_create", lambda *a: None)
    for kind, bits in ((ua.UA_DTYPE_BF16, 16), (ua.UA_DTYPE_FP8_E4M3, 8), (ua.UA_DTYPE_FP4_E2M1, 4.5)):
        p = ua.Problem(HQ, HK, D, B, BLOCKS, N, WIDTH, T, ua.UA_FLAG_CAUSAL, 0.1, kv_dtype=kind)
        assert p.kv_dtype == kind and p._cache_shape == ua.cache_shape(BLOCKS, HK, D, B, kind)
        assert p._cache_bytes == BLOCKS * B * HK * D * bits / 8
