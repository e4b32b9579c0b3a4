"""Pins of the plain cache implementations the GPU tests compare with, and the
cache entry points' host checks that need no device.  CPU only."""
import ctypes

import numpy as np
import pytest
import torch

import paged_varlen_flash_gb300 as ua
from paged_varlen_flash_gb300 import build as ua_build
from tests import cache_ref as R


@pytest.fixture(scope="module")
def lib():
    ua_build.build()
    return ua.load_library()


def test_e4m3_tables_agree_with_torch():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().numpy().astype(np.float64)
    np.testing.assert_array_equal(R.e4m3_values(codes.numpy()), want)
    x = np.random.default_rng(0).normal(size=20000) * 100
    x = np.clip(x, -448, 448).astype(np.float32).astype(np.float64)
    got = R.e4m3_values(R.e4m3_codes(x))
    want = torch.tensor(x, dtype=torch.float32).to(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(got, want.astype(np.float64))


def test_fp4_rounds_midpoints_to_even_codes():
    # amax 6 makes the group scale 1, so the values are the ratios themselves.
    x = np.array([[6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0, 0.2, 0.3, 0, -0.0, 4.9, 5.1]])
    codes, s8 = R.quantise_fp4(x, 1.0)
    assert s8.tolist() == [[0x38]]
    assert codes[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 0, 14, 0, 1, 0, 0, 6, 7]


def test_fp4_special_groups():
    x = np.zeros((4, 16))
    x[1, 3] = np.inf
    x[1, 4] = -1e30
    x[2, 5] = np.nan
    x[3] = 1e-9
    codes, s8 = R.quantise_fp4(x, 1.0)
    assert s8[:, 0].tolist() == [0, 0x7e, 0x7f, 0]
    assert codes[1, 3] == 7 and codes[1, 4] == 15 and codes[1].sum() == 22
    assert not codes[0].any() and not codes[2].any() and not codes[3].any()


def test_attention_weights_sum_to_one_and_follow_the_masks():
    g = np.random.default_rng(1)
    q, k, v = g.normal(size=(3, 4, 64)), g.normal(size=(9, 2, 64)), g.normal(size=(9, 2, 64))
    o, a, w, _ = R.attention(q, k, v, 0.125, window=4)
    np.testing.assert_allclose(w.sum(-1), 1.0, atol=1e-14)
    assert np.all(w[:, 0, 7:] == 0) and np.all(w[:, 0, :3] == 0) and np.all(w[:, 2, 5:] > 0)
    np.testing.assert_allclose(o[0, 3], w[3, 0] @ v[:, 1], atol=1e-14)
    _, _, w, _ = R.attention(q, k, v, 0.125, sinks=np.array([np.inf, -np.inf, 0.0, 1.0]))
    assert np.all(w[0] == 0) and np.allclose(w[1].sum(-1), 1) and np.all(w[2].sum(-1) < 1)


def test_evict_choice_orders_and_ties():
    w = np.array([1.0, 5.0, 5.0, np.nan, 5.0, np.inf, 0.0, 9.0], np.float32)
    assert R.evict_choice(w, 8, 4, 1).tolist() == [1, 2, 5, 7]
    assert R.evict_choice(w, 8, 7, 0).tolist() == [0, 1, 2, 4, 5, 6, 7]
    assert R.evict_choice(w, 8, 3, 3).tolist() == [5, 6, 7]
    assert R.evict_choice(w, 3, 4, 1).tolist() == [0, 1, 2]


def test_new_constants():
    assert ua.UA_FLAG_KEY_WEIGHTS == 1 << 6 and ua.UA_DTYPE_FP4_E2M1 == 2
    assert ua.cache_shape(7, 2, 128, 16, ua.UA_DTYPE_FP4_E2M1) == (7, 2, 16 * 72)
    assert ua.cache_shape(7, 2, 128, 16) == (7, 16, 2, 128)


def _desc(**over):
    base = dict(num_q_heads=8, num_kv_heads=2, head_size=128, block_size=16, num_blocks=64,
                max_num_seqs=4, max_blocks_per_seq=8, max_total_q=64, dtype=0,
                flags=ua.UA_FLAG_CAUSAL, scale=0.125, softcap=0.0, window=0, path=0,
                kv_dtype=ua.UA_DTYPE_FP4_E2M1, k_scale=1.0, v_scale=1.0)
    base.update(over)
    return ua.binding.ProblemDesc(**base)


@pytest.mark.parametrize("over,status", [
    (dict(k_scale=0.0), 1), (dict(v_scale=float("nan")), 1), (dict(v_scale=float("inf")), 1),
    (dict(kv_dtype=3), 1), (dict(path=1), 2), (dict(path=2), 2), (dict(path=3), 2), (dict(path=4), 1),
    (dict(head_size=96), 2), (dict(block_size=8), 2),
])
def test_fp4_descriptions_are_checked_before_any_device_work(lib, over, status):
    h = ctypes.c_void_p()
    assert lib.ua_problem_create(ctypes.byref(_desc(**over)), ctypes.byref(h)) == status
    assert not h.value


def test_noalloc_refuses_a_4bit_cache(lib):
    st = ua.ua_forward_noalloc(_desc(), None, None, None, None, None, None, 1, 1, 1, 1,
                               ua.UA_FLAG_CAUSAL, None, None, None, stream=0)
    assert st == 2


def test_entry_points_check_their_handle_first(lib):
    assert ua.ua_cache_store(None, None, None, 0, None, None, None, None, None, 1, 1, 1, 1, stream=0) == 1
    assert ua.ua_cache_expand(None, None, None, None, None, None, 1, 1, None, None, None, 1, 1, stream=0) == 1
    assert ua.ua_cache_evict(None, None, None, None, None, None, 1, 1, None, None, 1, 1, 0, None, None,
                             stream=0) == 1
    assert ua.ua_forward_weights(None, None, None, None, None, None, None, 1, 1, 1, 1, 0, None, None, None,
                                 None, 1, 1.0, None, stream=0) == 1


def test_row_strides_are_read_from_the_dimensions_that_have_them():
    from paged_varlen_flash_gb300.binding import _token_stride, _weight_stride
    w = torch.zeros(4, 2, 12)
    assert _weight_stride(w, "w") == 12 and _weight_stride(w[1:, :, :9], "w") == 12
    assert _weight_stride(torch.zeros(3, 5, 12)[:, 1:2, :10], "w") == 60
    assert _weight_stride(torch.zeros(1, 1, 12)[:, :, :7], "w") == 7
    assert _weight_stride(torch.zeros(12).expand(4, 2, 12), "w") == 0    # the call refuses it
    for bad in (w[:, :1].expand(4, 2, 12), w.transpose(1, 2), w[::2], w[0]):
        with pytest.raises(ValueError):
            _weight_stride(bad, "w")
    x = torch.zeros(6, 4, 64)
    assert _token_stride(x, "x") == 256 and _token_stride(x[:, :2], "x") == 256
    assert _token_stride(x[:1, :2], "x") == 256 and _token_stride(x[:, 1:2, :32], "x") == 256
    for bad in (x[:, ::2], x.transpose(0, 2), x[0]):
        with pytest.raises(ValueError):
            _token_stride(bad, "x")
