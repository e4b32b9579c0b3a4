"""What the cache methods of ``Problem`` refuse before the library is called: shapes,
strides and element types that the kernels would read or write past.  CPU only: the
problem has no handle, so that a call whose arguments pass ends in the library's
"invalid argument"."""
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from paged_varlen_flash_gb300 import build as ua_build

N, HQ, HK, D, B, WIDTH, BLOCKS, KEYS = 3, 8, 2, 64, 16, 4, 20, 50


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 3


def elsewhere(t):
    """A tensor that says it is on another device."""
    return t.as_subclass(Elsewhere)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ua_build.build()
    ua.load_library()


@pytest.fixture()
def p():
    x = ua.Problem.__new__(ua.Problem)
    x.handle = None
    x.flags, x.head_size, x.num_q_heads, x.num_kv_heads = ua.UA_FLAG_CAUSAL, D, HQ, HK
    x.block_size, x.max_blocks_per_seq = B, WIDTH
    return x


def reaches_the_library(call, **over):
    with pytest.raises(ua.UAError) as e:
        call(**over)
    assert e.value.status == 1


def base():
    cache = torch.zeros(BLOCKS, B, HK, D, dtype=torch.bfloat16)
    return dict(q=torch.zeros(N, HQ, D, dtype=torch.bfloat16), k=cache, v=cache.clone(),
                table=torch.zeros(N, WIDTH, dtype=torch.int32), cu=torch.zeros(N + 1, dtype=torch.int32),
                used=torch.zeros(N, dtype=torch.int32), w=torch.zeros(N, HK, KEYS + 5))


def weights_call(p, w_in, w_out, num_seqs=N, keys=KEYS):
    t = base()
    p.forward_weights(t["q"], t["k"], t["v"], t["table"], t["cu"], t["used"], num_seqs, N, 1, keys,
                      ua.UA_FLAG_CAUSAL, w_in, w_out, stream=0)


BAD_WEIGHTS = [
    torch.zeros(N, HK, KEYS - 1),                        # a key without a column
    torch.zeros(N, HK - 1, KEYS),                        # too few heads
    torch.zeros(N, HK + 1, KEYS),
    torch.zeros(N - 1, HK, KEYS),                        # too few sequences
    torch.zeros(N, HK, KEYS, dtype=torch.float64),
    torch.zeros(N, HK, KEYS, dtype=torch.bfloat16),
    elsewhere(torch.zeros(N, HK, KEYS)),             # not where q is
    torch.zeros(N, HK * KEYS),
]


@pytest.mark.parametrize("case", range(len(BAD_WEIGHTS)))
def test_key_weights_of_other_shapes_and_types(p, case):
    bad, good = BAD_WEIGHTS[case], torch.zeros(N, HK, KEYS)
    for w_in, w_out in ((None, bad), (bad, bad), (bad, good), (good, bad)):
        with pytest.raises(ValueError):
            weights_call(p, w_in, w_out)


def test_key_weights_that_fit(p):
    big = torch.zeros(N + 2, HK, KEYS + 9)
    for w in (torch.zeros(N, HK, KEYS), big, big[1:, :, :KEYS]):
        reaches_the_library(weights_call, p=p, w_in=None, w_out=w)
        reaches_the_library(weights_call, p=p, w_in=w, w_out=w)


def evict_call(p, w_in=None, w_out=None, budget=10, kept=None, used=None, dst=None, keys=KEYS):
    t = base()
    w_in = t["w"] if w_in is None else w_in
    w_out = t["w"] if w_out is None else w_out
    kept = torch.zeros(N, HK, budget, dtype=torch.int32) if kept is None else kept
    p.cache_evict(t["k"], t["v"], t["table"], t["used"], N, keys, w_in, w_out, budget, 2, kept,
                  t["used"] if used is None else used, dst_block_table=dst, stream=0)


@pytest.mark.parametrize("case", range(len(BAD_WEIGHTS)))
def test_evicted_weights_of_other_shapes_and_types(p, case):
    reaches_the_library(evict_call, p=p)
    for w in (dict(w_in=BAD_WEIGHTS[case]), dict(w_out=BAD_WEIGHTS[case]),
              dict(w_in=BAD_WEIGHTS[case], w_out=BAD_WEIGHTS[case])):
        with pytest.raises(ValueError):
            evict_call(p, **w)


@pytest.mark.parametrize("bad", [
    dict(kept=torch.zeros(N, HK, 10, dtype=torch.int16)), dict(kept=torch.zeros(N, HK, 10, dtype=torch.int64)),
    dict(kept=torch.zeros(N, HK, 10)), dict(kept=torch.zeros(N, HK, 9, dtype=torch.int32)),
    dict(kept=torch.zeros(N, HK, 20, dtype=torch.int32)[:, :, ::2]),
    dict(kept=elsewhere(torch.zeros(N, HK, 10, dtype=torch.int32))),
    dict(used=torch.zeros(N - 1, dtype=torch.int32)), dict(used=torch.zeros(N, dtype=torch.int16)),
    dict(used=torch.zeros(N, dtype=torch.int64)), dict(used=torch.zeros(2 * N, dtype=torch.int32)[::2]),
    dict(used=elsewhere(torch.zeros(N, dtype=torch.int32))),
])
def test_eviction_results_of_other_shapes_and_types(p, bad):
    with pytest.raises(ValueError):
        evict_call(p, **bad)
    reaches_the_library(evict_call, p=p, used=torch.zeros(N + 4, dtype=torch.int32))


INT = torch.int32


@pytest.mark.parametrize("bad", [
    torch.zeros(N, 1, dtype=INT),                            # compact: ceil(budget / b) ids a row
    torch.zeros(N, WIDTH + 1, dtype=INT),
    torch.zeros(N - 1, WIDTH, dtype=INT), torch.zeros(N * WIDTH, dtype=INT),
    torch.zeros(WIDTH, N, dtype=INT).T, torch.zeros(N, WIDTH, dtype=torch.int64),
    torch.zeros(N, WIDTH, dtype=torch.int16), elsewhere(torch.zeros(N, WIDTH, dtype=INT)),
])
def test_destination_tables_of_another_layout(p, bad):
    with pytest.raises(ValueError):
        evict_call(p, dst=bad)


def test_destination_tables_that_fit(p):
    full = torch.zeros(N + 1, WIDTH, dtype=INT)
    for dst in (full, full[1:], full[:, :1], full[:, 1:]):   # 10 kept keys are one block of 16
        reaches_the_library(evict_call, p=p, dst=dst)
    with pytest.raises(ValueError):
        evict_call(p, budget=17, dst=full[:, :1])            # two blocks
    reaches_the_library(evict_call, p=p, budget=17, keys=16, dst=full[:, :1])


def store_call(p, k_new, v_new, total_q=N):
    t = base()
    p.cache_store(k_new, v_new, t["k"], t["v"], t["table"], t["cu"], t["used"], N, total_q, 1, KEYS, stream=0)


BF = torch.bfloat16


@pytest.mark.parametrize("bad", [
    torch.zeros(N - 1, HK, D, dtype=BF), torch.zeros(N, HK - 1, D, dtype=BF), torch.zeros(N, HK + 1, D, dtype=BF),
    torch.zeros(N, HK, D // 2, dtype=BF), torch.zeros(N, HK, 2 * D, dtype=BF),
    torch.zeros(N, HK, D, dtype=torch.float16), torch.zeros(N, HK, D), torch.zeros(N, HK, D, dtype=torch.uint8),
    elsewhere(torch.zeros(N, HK, D, dtype=BF)),
])
def test_new_rows_of_other_shapes_and_types(p, bad):
    good = torch.zeros(N, HK, D, dtype=BF)
    for k_new, v_new in ((bad, bad), (good, bad), (bad, good)):
        with pytest.raises(ValueError):
            store_call(p, k_new, v_new)


def test_new_rows_that_fit(p):
    fused = torch.zeros(N + 3, 2 * HK + 1, D, dtype=BF)      # a padded batch of a fused projection
    reaches_the_library(store_call, p=p, k_new=fused[:, :HK], v_new=fused[:, HK:2 * HK])
    reaches_the_library(store_call, p=p, k_new=fused[:, :HK], v_new=fused[:, HK:2 * HK], total_q=N + 3)


def expand_call(p, k_out=None, v_out=None, table=None, begin=None):
    t = base()
    k_out = torch.zeros(6, B, HK, D, dtype=BF) if k_out is None else k_out
    v_out = torch.zeros(6, B, HK, D, dtype=BF) if v_out is None else v_out
    table = torch.zeros(N, 9, dtype=INT) if table is None else table
    p.cache_expand(t["k"], t["v"], t["table"], t["used"], N, KEYS, k_out, v_out, table, begin=begin, stream=0)


@pytest.mark.parametrize("bad", [
    dict(v_out=torch.zeros(5, B, HK, D, dtype=BF)),          # fewer blocks than k_out names
    dict(k_out=torch.zeros(5, B, HK, D, dtype=BF)),
    dict(k_out=torch.zeros(6, B, HK, D)), dict(v_out=torch.zeros(6, B, HK, D, dtype=torch.uint8)),
    dict(k_out=torch.zeros(6, B // 2, HK, D, dtype=BF), v_out=torch.zeros(6, B // 2, HK, D, dtype=BF)),
    dict(k_out=torch.zeros(6, B, 1, D, dtype=BF), v_out=torch.zeros(6, B, 1, D, dtype=BF)),
    dict(k_out=torch.zeros(6, B, HK, 2 * D, dtype=BF)[..., :D]), dict(v_out=torch.zeros(12, B, HK, D, dtype=BF)[::2]),
    dict(k_out=torch.zeros(6, B * HK * D, dtype=BF), v_out=torch.zeros(6, B * HK * D, dtype=BF)),
    dict(k_out=elsewhere(torch.zeros(6, B, HK, D, dtype=BF)),
         v_out=elsewhere(torch.zeros(6, B, HK, D, dtype=BF))),
    dict(table=torch.zeros(N - 1, 9, dtype=INT)), dict(table=torch.zeros(N, 9, dtype=torch.int64)),
    dict(table=torch.zeros(N, 9, dtype=torch.int16)), dict(table=torch.zeros(9, N, dtype=INT).T),
    dict(table=elsewhere(torch.zeros(N, 9, dtype=INT))),
    dict(begin=torch.zeros(N - 1, dtype=INT)), dict(begin=torch.zeros(N, dtype=torch.int64)),
    dict(begin=torch.zeros(N, dtype=torch.int16)),
])
def test_pages_and_tables_to_expand_into_of_other_shapes_and_types(p, bad):
    with pytest.raises(ValueError):
        expand_call(p, **bad)


def test_pages_and_tables_to_expand_into_that_fit(p):
    reaches_the_library(expand_call, p=p)
    reaches_the_library(expand_call, p=p, table=torch.zeros(N + 2, 12, dtype=INT)[1:, 3:],
                        begin=torch.zeros(N + 1, dtype=INT))


def test_current_stream_with_and_without_the_short_accessors():
    """The stream of whatever device is current at the call; the public API where torch
    lacks the accessors."""
    from types import SimpleNamespace as NS
    from paged_varlen_flash_gb300.binding import _stream_reader
    now = dict(device=0, streams={0: 11, 1: 22})
    cuda = NS(current_device=lambda: now["device"],
              current_stream=lambda: NS(cuda_stream=now["streams"][now["device"]]))
    raw = dict(_cuda_getDevice=lambda: now["device"], _cuda_getCurrentRawStream=lambda d: now["streams"][d])
    for c in (raw, {}, dict(_cuda_getDevice=raw["_cuda_getDevice"])):
        read = _stream_reader(NS(cuda=cuda, _C=NS(**c)))
        now.update(device=0, streams={0: 11, 1: 22})
        assert read() == 11
        now["device"] = 1
        assert read() == 22
        now["streams"][1] = 33
        assert read() == 33
