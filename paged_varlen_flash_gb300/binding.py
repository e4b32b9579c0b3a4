"""ctypes binding of ``include/ua.h`` (argument marshalling only).

Every function here forwards to the C ABI of ``libua.so``; all arithmetic runs
in that library's CUDA kernels.  Tensors are torch tensors (device memory for
``ua_forward``, host memory for ``ua_forward_host``); streams are torch CUDA
streams or raw ``cudaStream_t`` integers.
"""
import ctypes
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "libua.so")

UA_OK = 0
UA_FLAG_CAUSAL = 1 << 0
UA_FLAG_SOFTCAP = 1 << 1
UA_FLAG_ALIBI = 1 << 2
UA_FLAG_WINDOW = 1 << 3
UA_FLAG_SINKS = 1 << 4
UA_FLAG_QQ_BIAS = 1 << 5
UA_FLAG_KEY_WEIGHTS = 1 << 6
UA_PARTIALS_F32 = 0
UA_PARTIALS_BF16 = 1

UA_DEVERR_CONTEXT = 1 << 0
UA_DEVERR_BLOCK_ID = 1 << 1
UA_DEVERR_CU_SEQLENS = 1 << 2
UA_DEVERR_BOUNDS = 1 << 3
UA_DEVERR_TIMEOUT = 1 << 4
UA_DEVERR_TREE = 1 << 5
UA_DEVERR_POOL = 1 << 6

UA_ROPE_HALF = 0
UA_ROPE_PAIRS = 1

UA_DTYPE_BF16 = 0
UA_DTYPE_FP8_E4M3 = 1
UA_DTYPE_FP4_E2M1 = 2

UA_PATH_AUTO = 0
UA_PATH_SPLIT_KV = 1
UA_PATH_TENSOR_CORE = 2
UA_PATH_DECODE_TC = 3

_lib = None


class UAError(RuntimeError):
    def __init__(self, status, what=""):
        msg = "%s: %s" % (what or "ua", ua_status_string(status))
        if status == 3 and _lib is not None:
            msg += " (%s)" % _lib.ua_last_cuda_error().decode()
        super().__init__(msg)
        self.status = status


class ProblemDesc(ctypes.Structure):
    _fields_ = [
        ("num_q_heads", ctypes.c_int32),
        ("num_kv_heads", ctypes.c_int32),
        ("head_size", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
        ("max_num_seqs", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("max_total_q", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("scale", ctypes.c_float),
        ("softcap", ctypes.c_float),
        ("window", ctypes.c_int32),
        ("path", ctypes.c_uint32),
        ("kv_dtype", ctypes.c_int32),
        ("k_scale", ctypes.c_float),
        ("v_scale", ctypes.c_float),
        ("split_partials", ctypes.c_int32),
    ]


def lib_path():
    return _LIB_PATH


def load_library():
    """Load ``libua.so``; raise if it has not been built (no fallback path)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(
            "libua.so is not built (%s); run `python -m paged_varlen_flash_gb300.build`"
            % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, u32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32
    lib.ua_problem_create.argtypes = [ctypes.POINTER(ProblemDesc), ctypes.POINTER(vp)]
    lib.ua_problem_create.restype = ctypes.c_int
    fwd = [vp, vp, vp, vp, vp, vp, vp, i32, i64, i32, i32, u32, vp, vp, vp, vp]
    lib.ua_forward.argtypes = fwd
    lib.ua_forward.restype = ctypes.c_int
    lib.ua_forward_host.argtypes = fwd
    lib.ua_forward_host.restype = ctypes.c_int
    lib.ua_check_device_error.argtypes = [vp, vp, ctypes.POINTER(i32)]
    lib.ua_check_device_error.restype = ctypes.c_int
    lib.ua_last_launch_count.argtypes = [vp]
    lib.ua_last_launch_count.restype = i32
    lib.ua_last_path.argtypes = [vp]
    lib.ua_last_path.restype = ctypes.c_char_p
    lib.ua_forward_topk.argtypes = [vp] * 7 + [i32, ctypes.c_int64, i32, i32, vp, vp, i32,
                                               ctypes.c_uint32, vp, vp, vp, vp]
    lib.ua_forward_topk.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.ua_forward_weights.argtypes = [vp] * 7 + [i32, i64, i32, i32, u32, vp, vp, vp, vp, i64, f32,
                                                  vp, vp]
    lib.ua_forward_weights.restype = ctypes.c_int
    lib.ua_cache_store.argtypes = [vp, vp, vp, i64, vp, vp, vp, vp, vp, i32, i64, i32, i32, vp]
    lib.ua_cache_store.restype = ctypes.c_int
    lib.ua_cache_expand.argtypes = [vp] * 6 + [i32, i32, vp, vp, vp, i32, i64, vp]
    lib.ua_cache_expand.restype = ctypes.c_int
    lib.ua_cache_evict.argtypes = [vp] * 6 + [i32, i32, vp, vp, i64, i32, i32, vp, vp, vp]
    lib.ua_cache_evict.restype = ctypes.c_int
    lib.ua_plan_step.argtypes = [vp] * 8 + [i64, i32, i64] + [vp] * 6 + [i32, vp]
    lib.ua_plan_step.restype = ctypes.c_int
    lib.ua_set_rope.argtypes = [vp, ctypes.POINTER(ctypes.c_double), i32, u32, f32]
    lib.ua_set_rope.restype = ctypes.c_int
    lib.ua_rope_store.argtypes = [vp, vp, i64, vp, vp, i64, vp, vp, i64, vp, i64, vp, vp, vp]
    lib.ua_rope_store.restype = ctypes.c_int
    lib.ua_forward_tree.argtypes = [vp] * 7 + [i32, i64, i32, i32, vp, i32, vp, u32, vp, vp, vp, vp]
    lib.ua_forward_tree.restype = ctypes.c_int
    lib.ua_cache_accept.argtypes = [vp] * 7 + [i64, vp, i32, i64, i32, i32, vp, i32, vp, vp, vp]
    lib.ua_cache_accept.restype = ctypes.c_int
    lib.ua_set_qq_bias.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int64]
    lib.ua_set_qq_bias.restype = ctypes.c_int
    lib.ua_debug_stall_data_waits.argtypes = [vp, i32, i64]
    lib.ua_debug_stall_data_waits.restype = ctypes.c_int
    lib.ua_set_profile_events.argtypes = [vp, vp, vp]
    lib.ua_set_profile_events.restype = ctypes.c_int
    lib.ua_destroy.argtypes = [vp]
    lib.ua_destroy.restype = None
    lib.ua_status_string.argtypes = [ctypes.c_int]
    lib.ua_status_string.restype = ctypes.c_char_p
    lib.ua_last_cuda_error.argtypes = []
    lib.ua_last_cuda_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def ua_status_string(status):
    return load_library().ua_status_string(int(status)).decode()


def _ptr(t):
    try:
        return t.data_ptr()
    except AttributeError:               # None or an address
        return t


def _stream_reader(torch):
    """A function that returns the current device's stream, without a Stream object
    (0.3 us against 2.9) where torch has the accessors that this takes."""
    torch.cuda.current_device()          # initialises CUDA
    device = getattr(torch._C, "_cuda_getDevice", None)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if device is None or raw is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(device())


_current_stream = None


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            import torch
            _current_stream = _stream_reader(torch)
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _empty_like(t, stream):
    """Memory like t's for a call on ``stream``.  The allocator hands out what its current
    stream has given back, which kernels of that stream may still use: another stream gets
    memory of its own, kept until what the current one has queued by then is done."""
    import torch
    if stream is None or not t.is_cuda:
        return torch.empty_like(t)
    raw, current = _stream(stream), torch.cuda.current_stream(t.device)
    if raw == current.cuda_stream:
        return torch.empty_like(t)
    own = torch.cuda.ExternalStream(raw, device=t.device) if raw else torch.cuda.default_stream(t.device)
    with torch.cuda.stream(own):
        out = torch.empty_like(t)
    out.record_stream(current)
    return out


def flags_of(causal=True, softcap=0.0, alibi=False, window=0, sinks=False, qq_bias=False):
    f = 0
    if causal:
        f |= UA_FLAG_CAUSAL
    if softcap:
        f |= UA_FLAG_SOFTCAP
    if alibi:
        f |= UA_FLAG_ALIBI
    if window:
        f |= UA_FLAG_WINDOW
    if sinks:
        f |= UA_FLAG_SINKS
    if qq_bias:
        f |= UA_FLAG_QQ_BIAS
    return f


def ua_problem_create(num_q_heads, num_kv_heads, head_size, block_size, num_blocks,
                      max_num_seqs, max_blocks_per_seq, max_total_q, flags, scale,
                      softcap=0.0, window=0, path=UA_PATH_AUTO, kv_dtype=UA_DTYPE_BF16,
                      k_scale=1.0, v_scale=1.0, split_partials=UA_PARTIALS_F32):
    """Returns an opaque problem handle (int); raises UAError on failure."""
    lib = load_library()
    d = ProblemDesc(num_q_heads, num_kv_heads, head_size, block_size, num_blocks,
                    max_num_seqs, max_blocks_per_seq, max_total_q, UA_DTYPE_BF16, flags,
                    scale, softcap, window, path, kv_dtype, k_scale, v_scale, split_partials)
    h = ctypes.c_void_p()
    st = lib.ua_problem_create(ctypes.byref(d), ctypes.byref(h))
    if st != UA_OK:
        raise UAError(st, "ua_problem_create")
    return h.value


def ua_forward(problem, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
               num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks, alibi_slopes,
               out, stream=None):
    """Enqueue a forward pass; all tensors are device tensors.  Returns the
    status code (0 = ok) without raising, so callers can test error paths."""
    return load_library().ua_forward(
        problem, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(cu_seqlens_q), _ptr(seqused_k), num_seqs, total_q, max_seqlen_q,
        max_seqlen_k, flags, _ptr(sinks), _ptr(alibi_slopes), _ptr(out), _stream(stream))


def ua_forward_topk(problem, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                    num_seqs, total_q, max_seqlen_q, max_seqlen_k, topk_idx, topk_len,
                    topk_stride, flags, sinks, alibi_slopes, out, stream=None):
    """Enqueue a sparse top-k forward (device tensors; topk_idx int32
    [total_q, topk_stride], topk_len int32 [total_q]).  Returns the status."""
    return load_library().ua_forward_topk(
        problem, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
        _ptr(cu_seqlens_q), _ptr(seqused_k), num_seqs, total_q, max_seqlen_q,
        max_seqlen_k, _ptr(topk_idx), _ptr(topk_len), topk_stride, flags, _ptr(sinks),
        _ptr(alibi_slopes), _ptr(out), _stream(stream))


def ua_forward_weights(problem, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                       num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks, alibi_slopes,
                       weights_in, weights_out, weight_stride, decay, out, stream=None):
    """Enqueue a forward pass that also accumulates every cached key's attention
    weight (fp32 [num_seqs, H_k, weight_stride]).  Returns the status."""
    return load_library().ua_forward_weights(
        problem, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(cu_seqlens_q),
        _ptr(seqused_k), num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, _ptr(sinks),
        _ptr(alibi_slopes), _ptr(weights_in), _ptr(weights_out), weight_stride, decay, _ptr(out),
        _stream(stream))


def ua_cache_store(problem, k_new, v_new, new_stride, k_cache, v_cache, block_table, cu_seqlens_q,
                   seqused_k, num_seqs, total_q, max_seqlen_q, max_seqlen_k, stream=None):
    """Enqueue the write of a chunk's K/V rows into the paged caches.  Returns
    the status."""
    return load_library().ua_cache_store(
        problem, _ptr(k_new), _ptr(v_new), new_stride, _ptr(k_cache), _ptr(v_cache),
        _ptr(block_table), _ptr(cu_seqlens_q), _ptr(seqused_k), num_seqs, total_q, max_seqlen_q,
        max_seqlen_k, _stream(stream))


def ua_cache_expand(problem, k_cache, v_cache, block_table, seqused_k, begin, num_seqs, max_keys,
                    k_out, v_out, out_block_table, out_table_stride, out_num_blocks, stream=None):
    """Enqueue the expansion of cached keys into bf16 pages.  Returns the status."""
    return load_library().ua_cache_expand(
        problem, _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(seqused_k), _ptr(begin),
        num_seqs, max_keys, _ptr(k_out), _ptr(v_out), _ptr(out_block_table), out_table_stride,
        out_num_blocks, _stream(stream))


def ua_cache_evict(problem, k_cache, v_cache, block_table, dst_block_table, seqused_k, num_seqs,
                   max_seqlen_k, weights_in, weights_out, weight_stride, budget, recent, kept,
                   seqused_out, stream=None):
    """Enqueue an eviction by key weights.  Returns the status."""
    return load_library().ua_cache_evict(
        problem, _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(dst_block_table),
        _ptr(seqused_k), num_seqs, max_seqlen_k, _ptr(weights_in), _ptr(weights_out),
        weight_stride, budget, recent, _ptr(kept), _ptr(seqused_out), _stream(stream))


def ua_plan_step(problem, block_table, blocks_held, free_blocks, free_count, ctx_lens, new_lens, parents,
                 parents_stride, num_seqs, max_tokens, granted, cu_seqlens_q, seqused_k, positions, slots,
                 tree_mask, mask_stride, stream=None):
    """Enqueue the hand-out of a step's blocks, slots, positions and ancestor masks.
    Returns the status."""
    return load_library().ua_plan_step(
        problem, _ptr(block_table), _ptr(blocks_held), _ptr(free_blocks), _ptr(free_count), _ptr(ctx_lens),
        _ptr(new_lens), _ptr(parents), parents_stride, num_seqs, max_tokens, _ptr(granted), _ptr(cu_seqlens_q),
        _ptr(seqused_k), _ptr(positions), _ptr(slots), _ptr(tree_mask), mask_stride, _stream(stream))


def ua_set_rope(problem, inv_freq, layout=UA_ROPE_HALF, magnitude=1.0):
    """Set the rotary frequencies (a sequence of floats, radians per position) of
    later ``ua_rope_store`` calls.  Returns the status."""
    values = (ctypes.c_double * len(inv_freq))(*inv_freq)
    return load_library().ua_set_rope(problem, values, len(inv_freq), layout, magnitude)


def ua_rope_store(problem, q, q_stride, k_new, v_new, kv_stride, positions, slots, total_q, q_out, out_stride,
                  k_cache, v_cache, stream=None):
    """Enqueue the rotation of q and k and the store of k and v.  Returns the status."""
    return load_library().ua_rope_store(
        problem, _ptr(q), q_stride, _ptr(k_new), _ptr(v_new), kv_stride, _ptr(positions), _ptr(slots), total_q,
        _ptr(q_out), out_stride, _ptr(k_cache), _ptr(v_cache), _stream(stream))


def ua_forward_tree(problem, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, num_seqs, total_q,
                    max_seqlen_q, max_seqlen_k, tree_mask, mask_stride, positions, flags, sinks, alibi_slopes, out,
                    stream=None):
    """Enqueue attention for trees of drafted tokens.  Returns the status."""
    return load_library().ua_forward_tree(
        problem, _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(cu_seqlens_q), _ptr(seqused_k),
        num_seqs, total_q, max_seqlen_q, max_seqlen_k, _ptr(tree_mask), mask_stride, _ptr(positions), flags,
        _ptr(sinks), _ptr(alibi_slopes), _ptr(out), _stream(stream))


def ua_cache_accept(problem, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, parents, parents_stride, last,
                    num_seqs, total_q, max_seqlen_q, max_seqlen_k, path, path_stride, accepted, seqused_out,
                    stream=None):
    """Enqueue the move of the accepted branches.  Returns the status."""
    return load_library().ua_cache_accept(
        problem, _ptr(k_cache), _ptr(v_cache), _ptr(block_table), _ptr(cu_seqlens_q), _ptr(seqused_k), _ptr(parents),
        parents_stride, _ptr(last), num_seqs, total_q, max_seqlen_q, max_seqlen_k, _ptr(path), path_stride,
        _ptr(accepted), _ptr(seqused_out), _stream(stream))


def rope_frequencies(rotated, base=10000.0, scaling=None, factor=1.0, trained=0, low=1.0, high=4.0):
    """Frequencies (radians per position) of ``rotated`` dims and the factor on cos
    and sin, for ``Problem.set_rope``: base^(-2i / rotated), and with ``scaling``

    * ``"linear"``  all divided by ``factor`` (positions interpolated);
    * ``"ntk"``     the base raised to base * factor^(rotated / (rotated - 2)), which
                    divides the lowest frequency by ``factor`` and keeps the highest;
    * ``"bands"``   divided by ``factor`` where fewer than ``low`` turns fit the
                    ``trained`` context, kept from ``high`` turns on, linear between;
    * ``"yarn"``    the same, linear in the pair's number between the (whole) ones that
                    make ``high`` and ``low`` turns (cut at 0 and ``rotated`` - 1, which
                    may lie behind the last pair), and cos and sin times
                    0.1 ln(factor) + 1.
    """
    n = rotated // 2
    if rotated < 2 or rotated % 2 or base <= 0 or factor <= 0:
        raise ValueError("rotated must be even and positive, base and factor positive")
    if scaling == "ntk":
        if rotated < 4:
            raise ValueError("ntk needs at least two pairs")
        base *= factor ** (rotated / (rotated - 2))
    freq = [base ** (-i / n) for i in range(n)]
    if scaling in (None, "ntk"):
        return freq, 1.0
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling not in ("bands", "yarn"):
        raise ValueError("scaling must be None, 'linear', 'ntk', 'bands' or 'yarn'")
    if trained <= 0 or not 0 < low < high:
        raise ValueError("%s needs the trained context and 0 < low < high" % scaling)
    turns = [trained * f / (2 * math.pi) for f in freq]
    if scaling == "bands":
        keep = [(t - low) / (high - low) for t in turns]
    else:
        # The (fractional) number of a pair that makes `turns` turns in the trained context.
        dim = lambda t: n * math.log(trained / (2 * math.pi * t)) / math.log(base)  # noqa: E731
        first, end = max(math.floor(dim(high)), 0), min(math.ceil(dim(low)), rotated - 1)
        keep = [1 - (i - first) / max(end - first, 1e-3) for i in range(n)]
    keep = [min(1.0, max(0.0, k)) for k in keep]
    return ([f * (k + (1 - k) / factor) for f, k in zip(freq, keep)],
            0.1 * math.log(factor) + 1.0 if scaling == "yarn" and factor > 1 else 1.0)


def cache_shape(num_blocks, num_kv_heads, head_size, block_size, kv_dtype=UA_DTYPE_BF16):
    """Shape of one K or V cache: bf16 or uint8 [num_blocks, b, H_k, d], or for
    the 4-bit format uint8 [num_blocks, H_k, bytes of a (block, KV head) page]."""
    if kv_dtype == UA_DTYPE_FP4_E2M1:
        return (num_blocks, num_kv_heads, block_size * (head_size // 2 + head_size // 16))
    return (num_blocks, block_size, num_kv_heads, head_size)


def _token_stride(t, name, total_q=0, num_kv_heads=None, head_size=None):
    """Elements between the tokens of a [total, H_k, d] tensor whose rows are contiguous
    (of at least total_q tokens, and those heads and dims)."""
    stride = t.stride()
    if len(stride) != 3:
        raise ValueError("%s must be [total_q, H_k, d]" % name)
    step, head, unit = stride
    n, heads, dims = t.shape
    if (unit != 1 or (heads > 1 and head != dims) or n < total_q or
            (num_kv_heads is not None and (heads != num_kv_heads or dims != head_size))):
        raise ValueError("%s must be [total_q, H_k, d] with contiguous heads" % name)
    return step if n > 1 else max(step, heads * dims)


def _weight_stride(t, name):
    """Elements between the rows of a [num_seqs, H_k, n] tensor; a dimension of
    one row has no stride of its own."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3 and stride[2] == 1:
        if shape[1] > 1:
            if shape[0] <= 1 or stride[0] == shape[1] * stride[1]:
                return stride[1]
        else:
            return stride[0] if shape[0] > 1 else shape[2]
    raise ValueError("%s must be [num_seqs, H_k, n] with evenly spaced rows" % name)


_type_names = {}


def _check(t, name, kind, device):
    """Refuse a tensor of another element type, or not on that device (as get_device counts)."""
    dtype = t.dtype
    if (_type_names.get(dtype) or _type_names.setdefault(dtype, str(dtype))) != kind or t.get_device() != device:
        raise ValueError("%s must be %s, on the device of the other tensors" % (name, kind))


def _refuse_vector(t, name, n, kind, device):
    if t.numel() < n or not t.is_contiguous():
        raise ValueError("%s must be contiguous, with at least %d elements" % (name, n))
    raise ValueError("%s must be %s, on the device of the other tensors" % (name, kind))


_int_types = _row_types = _cache_types = None


def _ints():
    """torch.int32 and torch.int64 (torch is not imported with this module)."""
    global _int_types
    if _int_types is None:
        import torch
        _int_types = torch.int32, torch.int64
    return _int_types


def _rows():
    """torch.bfloat16 and torch.float32."""
    global _row_types
    if _row_types is None:
        import torch
        _row_types = torch.bfloat16, torch.float32
    return _row_types


def _types_of(kv_dtype):
    """The element types of a cache of that kv_dtype."""
    global _cache_types
    if _cache_types is None:
        import torch
        codes = torch.uint8, torch.float8_e4m3fn
        _cache_types = {UA_DTYPE_BF16: (torch.bfloat16,), UA_DTYPE_FP8_E4M3: codes, UA_DTYPE_FP4_E2M1: codes[:1]}
    return _cache_types[kv_dtype]


def _head_terms(t, name, num_q_heads, device):
    """The address of sinks or slopes, a contiguous fp32 [H_q]."""
    if (t.dtype is not _rows()[1] or t.numel() < num_q_heads or not t.is_contiguous() or
            t.get_device() != device):
        _refuse_vector(t, name, num_q_heads, "float32", device)
    return t.data_ptr()


def _check_table(table, num_seqs, width, device):
    """Refuse a block table that is not a contiguous int32 [num_seqs, width]."""
    shape = table.shape
    if (table.dtype is not _ints()[0] or not table.is_contiguous() or len(shape) != 2 or shape[1] != width or
            shape[0] < num_seqs or table.get_device() != device):
        raise ValueError("block_table must be a contiguous int32 [num_seqs, max_blocks_per_seq]")


def _tree_rows(parents, num_seqs, device):
    """Elements between the rows of the trees' parents [num_seqs, n], and n."""
    shape, stride = parents.shape, parents.stride()
    if len(shape) != 2 or shape[0] < num_seqs or shape[1] < 1 or (shape[1] > 1 and stride[1] != 1) or (
            shape[0] > 1 and stride[0] < shape[1]):
        raise ValueError("parents must be [num_seqs, nodes] with unit inner stride")
    if parents.dtype is not _ints()[0] or parents.get_device() != device:
        raise ValueError("parents must be int32, on the device of the other tensors")
    return stride[0] if shape[0] > 1 else shape[1], shape[1]


def _mask_stride(mask, tokens, device):
    """Words between the rows of a tree mask [tokens, words]."""
    shape = mask.shape
    if len(shape) != 2 or shape[0] < tokens or shape[1] < 1 or not mask.is_contiguous():
        raise ValueError("tree_mask must be a contiguous [tokens, words]")
    if (mask.dtype is not _ints()[0] and str(mask.dtype) != "torch.uint32") or mask.get_device() != device:
        raise ValueError("tree_mask must be int32 or uint32, on the device of the other tensors")
    return shape[1]


def _weight_rows(t, name, num_seqs, num_kv_heads, n, like):
    """Row stride of key weights that hold at least n keys of num_seqs sequences."""
    stride = _weight_stride(t, name)
    shape = t.shape
    if shape[0] < num_seqs or shape[1] != num_kv_heads or shape[2] < n:
        raise ValueError("%s must be [num_seqs, H_k, n] with a column per key" % name)
    _check(t, name, "torch.float32", like.get_device())
    return stride


def ua_forward_host(problem, q_host, k_cache, v_cache, block_table_host, cu_seqlens_q_host,
                    seqused_k_host, num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags,
                    sinks_host, alibi_host, out_host, stream=None):
    """Forward with host-resident per-step inputs and output (caches on device)."""
    return load_library().ua_forward_host(
        problem, _ptr(q_host), _ptr(k_cache), _ptr(v_cache), _ptr(block_table_host),
        _ptr(cu_seqlens_q_host), _ptr(seqused_k_host), num_seqs, total_q, max_seqlen_q,
        max_seqlen_k, flags, _ptr(sinks_host), _ptr(alibi_host), _ptr(out_host),
        _stream(stream))


def ua_forward_noalloc(desc, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                       num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags, sinks,
                       alibi_slopes, out, device_error=None, stream=None):
    """The allocation-free forward (``ProblemDesc`` instead of a problem
    handle; partials in the library's static device scratch).  Returns the
    status code without raising."""
    lib = load_library()
    fn = lib.ua_forward_noalloc
    vp = ctypes.c_void_p
    fn.argtypes = [ctypes.POINTER(ProblemDesc), vp, vp, vp, vp, vp, vp, ctypes.c_int32,
                   ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_uint32, vp, vp,
                   vp, vp, vp]
    fn.restype = ctypes.c_int
    return fn(ctypes.byref(desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table),
              _ptr(cu_seqlens_q), _ptr(seqused_k), num_seqs, total_q, max_seqlen_q,
              max_seqlen_k, flags, _ptr(sinks), _ptr(alibi_slopes), _ptr(out),
              _ptr(device_error), _stream(stream))


def ua_set_qq_bias(problem, bias, n, row_stride):
    """Bind the query-query bias matrix (device fp32, element (a, c) at
    a * row_stride + c) to a problem; ``bias=None`` clears it.  Returns the
    status code without raising."""
    return load_library().ua_set_qq_bias(problem, _ptr(bias), n, row_stride)


def ua_debug_stall_data_waits(problem, enable, limit_ns=2_000_000):
    """Testing hook: make the next forward calls' first K/V data wait run out
    after ``limit_ns`` (see include/ua.h).  Returns the status code."""
    return load_library().ua_debug_stall_data_waits(problem, int(enable), int(limit_ns))


def ua_check_device_error(problem, stream=None):
    """Synchronise the stream and return (and clear) the device error word."""
    code = ctypes.c_int32(0)
    st = load_library().ua_check_device_error(problem, _stream(stream), ctypes.byref(code))
    if st not in (UA_OK, 5):
        raise UAError(st, "ua_check_device_error")
    return code.value


def ua_destroy(problem):
    if problem:
        load_library().ua_destroy(problem)


class Problem:
    """Owning wrapper around a ``ua_problem`` handle."""

    def __init__(self, num_q_heads, num_kv_heads, head_size, block_size, num_blocks,
                 max_num_seqs, max_blocks_per_seq, max_total_q, flags, scale, softcap=0.0,
                 window=0, path=UA_PATH_AUTO, kv_dtype=UA_DTYPE_BF16, k_scale=1.0, v_scale=1.0,
                 split_partials=UA_PARTIALS_F32):
        self.handle = ua_problem_create(num_q_heads, num_kv_heads, head_size, block_size,
                                        num_blocks, max_num_seqs, max_blocks_per_seq,
                                        max_total_q, flags, scale, softcap, window, path,
                                        kv_dtype, k_scale, v_scale, split_partials)
        self.flags = flags
        self.kv_dtype = kv_dtype
        self._cache_shape = cache_shape(num_blocks, num_kv_heads, head_size, block_size, kv_dtype)
        self._cache_bytes = math.prod(self._cache_shape) * (2 if kv_dtype == UA_DTYPE_BF16 else 1)
        self.head_size = head_size
        self.block_size = block_size
        self.num_blocks = num_blocks
        self.max_blocks_per_seq = max_blocks_per_seq
        self.num_q_heads = num_q_heads
        self.num_kv_heads = num_kv_heads

    kv_dtype, _cache_shape = UA_DTYPE_BF16, None

    def _check_caches(self, k_cache, v_cache, device):
        """Refuse caches that are not the problem's: kernels would read or write past them."""
        shape, types = self._cache_shape, _types_of(self.kv_dtype)
        kind = types[0]
        if (k_cache.shape == shape and v_cache.shape == shape and k_cache.dtype is kind and v_cache.dtype is kind and
                k_cache.is_contiguous() and v_cache.is_contiguous() and k_cache.get_device() == v_cache.get_device() == device):
            return                       # (the usual case, in as few calls as it takes)
        shape = cache_shape(self.num_blocks, self.num_kv_heads, self.head_size, self.block_size, self.kv_dtype)
        for t in (k_cache, v_cache):
            if (t.dtype not in types or t.shape[1:] != shape[1:] or t.shape[0] < shape[0] or not t.is_contiguous() or
                    t.get_device() != device):
                raise ValueError("k_cache and v_cache must be contiguous %s of %s, on the device of the other tensors" % (
                    list(shape), " or ".join(map(str, types))))

    _cache_bytes = 0

    def _check_room(self, k_cache, v_cache):
        """Refuse tensors that are shorter than the problem's caches, or not contiguous: kernels
        would read or write past them.  (Addresses are taken as they are.)"""
        n = self._cache_bytes
        try:
            if k_cache.nbytes >= n and v_cache.nbytes >= n and k_cache.is_contiguous() and v_cache.is_contiguous():
                return
        except AttributeError:
            pass
        for t in (k_cache, v_cache):
            if hasattr(t, "nbytes") and (t.nbytes < n or not t.is_contiguous()):
                raise ValueError("k_cache and v_cache must be contiguous, with %d bytes at least" % n)

    @classmethod
    def for_workload(cls, w, max_total_q=None, max_num_seqs=None, extra_flags=0,
                     path=UA_PATH_AUTO, split_partials=UA_PARTIALS_F32):
        flags = flags_of(w.causal, w.softcap, w.alibi_slopes is not None, w.window,
                         w.sinks is not None, getattr(w, "qq_bias", None) is not None) | extra_flags
        fp8 = getattr(w, "kv_fp8", False)
        return cls(w.hq, w.hk, w.d, w.b, w.num_blocks, max_num_seqs or max(1, w.num_seqs),
                   w.max_blocks_per_seq, max_total_q or max(1, w.total_q), flags, w.scale,
                   w.softcap, w.window, path, UA_DTYPE_FP8_E4M3 if fp8 else UA_DTYPE_BF16,
                   getattr(w, "k_scale", 1.0), getattr(w, "v_scale", 1.0), split_partials)

    def forward(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, num_seqs,
                total_q, max_seqlen_q, max_seqlen_k, flags, sinks=None, alibi_slopes=None,
                out=None, stream=None):
        self._check_room(k_cache, v_cache)
        if out is None:
            out = _empty_like(q, stream)
        st = ua_forward(self.handle, q, k_cache, v_cache, block_table, cu_seqlens_q,
                        seqused_k, num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags,
                        sinks, alibi_slopes, out, stream)
        if st != UA_OK:
            raise UAError(st, "ua_forward")
        return out

    def forward_topk(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                     num_seqs, total_q, max_seqlen_q, max_seqlen_k, topk_idx, topk_len, flags,
                     sinks=None, alibi_slopes=None, out=None, stream=None):
        self._check_room(k_cache, v_cache)
        if out is None:
            out = _empty_like(q, stream)
        if topk_idx.dim() != 2 or topk_idx.stride(1) != 1:
            raise ValueError("topk_idx must be [total_q, K] with unit inner stride")
        st = ua_forward_topk(self.handle, q, k_cache, v_cache, block_table, cu_seqlens_q,
                             seqused_k, num_seqs, total_q, max_seqlen_q, max_seqlen_k, topk_idx,
                             topk_len, topk_idx.stride(0), flags, sinks, alibi_slopes, out,
                             stream)
        if st != UA_OK:
            raise UAError(st, "ua_forward_topk")
        return out

    def forward_weights(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, num_seqs,
                        total_q, max_seqlen_q, max_seqlen_k, flags, weights_in, weights_out,
                        decay=1.0, sinks=None, alibi_slopes=None, out=None, stream=None):
        """``forward`` that also writes decay * weights_in plus this call's
        attention weights to ``weights_out`` (fp32 [num_seqs, H_k, n >= max_seqlen_k];
        ``weights_in`` may be the same tensor, or None for zeros)."""
        self._check_room(k_cache, v_cache)
        rows = num_seqs, self.num_kv_heads, max_seqlen_k, q
        stride = _weight_rows(weights_out, "weights_out", *rows)
        if weights_in is not None and _weight_rows(weights_in, "weights_in", *rows) != stride:
            raise ValueError("weights_in and weights_out must share a row stride")
        if out is None:
            out = _empty_like(q, stream)
        st = ua_forward_weights(self.handle, q, k_cache, v_cache, block_table, cu_seqlens_q,
                                seqused_k, num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags,
                                sinks, alibi_slopes, weights_in, weights_out, stride, decay, out,
                                stream)
        if st != UA_OK:
            raise UAError(st, "ua_forward_weights")
        return out

    def cache_store(self, k_new, v_new, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                    num_seqs, total_q, max_seqlen_q, max_seqlen_k, stream=None):
        """Write a chunk's rows (bf16 [total_q, H_k, d]; tokens may be strided)
        to the positions ``forward`` expects them at."""
        self._check_room(k_cache, v_cache)
        stride = _token_stride(k_new, "k_new", total_q, self.num_kv_heads, self.head_size)
        device = k_cache.get_device()
        _check(k_new, "k_new", "torch.bfloat16", device)
        _check(v_new, "v_new", "torch.bfloat16", device)
        if _token_stride(v_new, "v_new", total_q, self.num_kv_heads, self.head_size) != stride:
            raise ValueError("k_new and v_new must share a token stride")
        # A decode step's store waits for the host: no call more than it takes.
        st = load_library().ua_cache_store(
            self.handle, k_new.data_ptr(), v_new.data_ptr(), stride, k_cache.data_ptr(),
            v_cache.data_ptr(), block_table.data_ptr(), cu_seqlens_q.data_ptr(),
            seqused_k.data_ptr(), num_seqs, total_q, max_seqlen_q, max_seqlen_k, _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_cache_store")

    def cache_expand(self, k_cache, v_cache, block_table, seqused_k, num_seqs, max_keys, k_out,
                     v_out, out_block_table, begin=None, stream=None):
        """Expand the keys from ``begin`` (or 0) on into the bf16 pages
        ``k_out`` / ``v_out`` [blocks, b, H_k, d]."""
        self._check_room(k_cache, v_cache)
        step, device = out_block_table.stride(), k_cache.get_device()
        if len(step) != 2 or step[1] != 1 or out_block_table.shape[0] < num_seqs:
            raise ValueError("out_block_table must be [num_seqs, n] with unit inner stride")
        shape = k_out.shape
        if (len(shape) != 4 or shape[1] != self.block_size or shape[2] != self.num_kv_heads or
                shape[3] != self.head_size or v_out.shape != shape or not k_out.is_contiguous() or
                not v_out.is_contiguous()):
            raise ValueError("k_out and v_out must be contiguous [blocks, b, H_k, d]")
        _check(k_out, "k_out", "torch.bfloat16", device)
        _check(v_out, "v_out", "torch.bfloat16", device)
        _check(out_block_table, "out_block_table", "torch.int32", device)
        if begin is not None:
            if begin.numel() < num_seqs or not begin.is_contiguous():
                raise ValueError("begin must be a contiguous [num_seqs]")
            _check(begin, "begin", "torch.int32", device)
        st = load_library().ua_cache_expand(
            self.handle, k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
            seqused_k.data_ptr(), _ptr(begin), num_seqs, max_keys, k_out.data_ptr(),
            v_out.data_ptr(), out_block_table.data_ptr(), step[0], shape[0], _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_cache_expand")

    def cache_evict(self, k_cache, v_cache, block_table, seqused_k, num_seqs, max_seqlen_k,
                    weights_in, weights_out, budget, recent, kept, seqused_out,
                    dst_block_table=None, stream=None):
        """Keep ``budget`` keys of every (sequence, KV head) by weight, in place
        or into ``dst_block_table`` (rows as far apart as block_table's); ``kept``
        int32 [num_seqs, H_k, budget]."""
        self._check_room(k_cache, v_cache)
        rows = num_seqs, self.num_kv_heads, max_seqlen_k, block_table
        stride = _weight_rows(weights_in, "weights_in", *rows)
        if _weight_rows(weights_out, "weights_out", *rows) != stride:
            raise ValueError("weights_in and weights_out must share a row stride")
        if tuple(kept.shape) != (num_seqs, self.num_kv_heads, budget) or not kept.is_contiguous():
            raise ValueError("kept must be a contiguous [num_seqs, H_k, budget]")
        _check(kept, "kept", "torch.int32", block_table.get_device())
        if seqused_out.numel() < num_seqs or not seqused_out.is_contiguous():
            raise ValueError("seqused_out must be a contiguous [num_seqs]")
        _check(seqused_out, "seqused_out", "torch.int32", block_table.get_device())
        if dst_block_table is not None:
            # Read with block_table's row stride, one id per block of kept keys.
            shape, step = dst_block_table.shape, dst_block_table.stride()
            blocks = -(-min(budget, max_seqlen_k) // self.block_size)
            if (len(shape) != 2 or shape[0] < num_seqs or shape[1] < blocks or (shape[1] > 1 and step[1] != 1) or
                    (num_seqs > 1 and step[0] != self.max_blocks_per_seq)):
                raise ValueError("dst_block_table must be laid out like block_table")
            _check(dst_block_table, "dst_block_table", "torch.int32", block_table.get_device())
        st = ua_cache_evict(self.handle, k_cache, v_cache, block_table, dst_block_table, seqused_k,
                            num_seqs, max_seqlen_k, weights_in, weights_out, stride, budget,
                            recent, kept, seqused_out, stream)
        if st != UA_OK:
            raise UAError(st, "ua_cache_evict")

    def plan_step(self, block_table, blocks_held, free_blocks, free_count, ctx_lens, new_lens, num_seqs, max_tokens,
                  granted, cu_seqlens_q, seqused_k, positions, slots, parents=None, tree_mask=None, stream=None):
        """Give the sequences of a step their blocks and tokens: ``new_lens`` tokens
        behind ``ctx_lens`` keys, drafted as chains or as trees (``parents`` int32
        [num_seqs, nodes], -1 for a node without parent).  In and out: ``block_table``,
        ``blocks_held``, ``free_blocks`` (a stack of ``free_count`` ids); out:
        ``granted``, ``cu_seqlens_q``, ``seqused_k``, and per packed token ``positions``,
        ``slots`` (int64) and ``tree_mask`` (int32 or uint32 [max_tokens, words])."""
        # A step waits for the host: checks without a call more than they take.
        i32, i64 = _ints()
        device, width = block_table.get_device(), self.max_blocks_per_seq
        _check_table(block_table, num_seqs, width, device)
        for t, n, name in ((blocks_held, num_seqs, "blocks_held"), (free_blocks, self.num_blocks, "free_blocks"),
                           (free_count, 1, "free_count"), (ctx_lens, num_seqs, "ctx_lens"),
                           (new_lens, num_seqs, "new_lens"), (granted, num_seqs, "granted"),
                           (cu_seqlens_q, num_seqs + 1, "cu_seqlens_q"), (seqused_k, num_seqs, "seqused_k"),
                           (positions, max_tokens, "positions")):
            if t.dtype is not i32 or t.numel() < n or not t.is_contiguous() or t.get_device() != device:
                _refuse_vector(t, name, n, "int32", device)
        if slots.dtype is not i64 or slots.numel() < max_tokens or not slots.is_contiguous() or slots.get_device() != device:
            _refuse_vector(slots, "slots", max_tokens, "int64", device)
        tree = mask = None
        stride = words = 0
        if parents is not None:
            tree, stride = parents.data_ptr(), _tree_rows(parents, num_seqs, device)[0]
        if tree_mask is not None:
            mask, words = tree_mask.data_ptr(), _mask_stride(tree_mask, max_tokens, device)
        st = load_library().ua_plan_step(
            self.handle, block_table.data_ptr(), blocks_held.data_ptr(), free_blocks.data_ptr(), free_count.data_ptr(),
            ctx_lens.data_ptr(), new_lens.data_ptr(), tree, stride, num_seqs, max_tokens, granted.data_ptr(),
            cu_seqlens_q.data_ptr(), seqused_k.data_ptr(), positions.data_ptr(), slots.data_ptr(), mask, words,
            _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_plan_step")

    def set_rope(self, inv_freq, layout=UA_ROPE_HALF, magnitude=1.0):
        """Set the rotary frequencies of later ``rope_store`` calls: radians per
        position of every pair (``rope_frequencies`` computes them), which dims form
        a pair, and the factor on cos and sin."""
        st = ua_set_rope(self.handle, inv_freq, layout, magnitude)
        if st != UA_OK:
            raise UAError(st, "ua_set_rope")

    def rope_store(self, q, k_new, v_new, positions, slots, total_q, k_cache, v_cache, q_out=None, stream=None):
        """Rotate q and k (bf16 [total_q, heads, d]; tokens may be strided) by
        ``positions`` and write k and v to ``slots`` (int64; negative: not stored).
        Returns the rotated q (``q_out``, which may be q)."""
        i32, i64 = _ints()
        bf16 = _rows()[0]
        device, heads, kv_heads, d = k_cache.get_device(), self.num_q_heads, self.num_kv_heads, self.head_size
        self._check_caches(k_cache, v_cache, device)
        if q_out is None:
            q_out = _empty_like(q, stream)
        q_stride = _token_stride(q, "q", total_q, heads, d)
        stride = _token_stride(k_new, "k_new", total_q, kv_heads, d)
        out_stride = _token_stride(q_out, "q_out", total_q, heads, d)
        if _token_stride(v_new, "v_new", total_q, kv_heads, d) != stride:
            raise ValueError("k_new and v_new must share a token stride")
        if not (q.dtype is bf16 and k_new.dtype is bf16 and v_new.dtype is bf16 and q_out.dtype is bf16 and
                q.get_device() == k_new.get_device() == v_new.get_device() == q_out.get_device() == device):
            raise ValueError("q, k_new, v_new and q_out must be torch.bfloat16, on the device of the caches")
        if positions.dtype is not i32 or positions.numel() < total_q or not positions.is_contiguous() or (
                positions.get_device() != device):
            _refuse_vector(positions, "positions", total_q, "int32", device)
        if slots.dtype is not i64 or slots.numel() < total_q or not slots.is_contiguous() or slots.get_device() != device:
            _refuse_vector(slots, "slots", total_q, "int64", device)
        st = load_library().ua_rope_store(
            self.handle, q.data_ptr(), q_stride, k_new.data_ptr(), v_new.data_ptr(), stride, positions.data_ptr(),
            slots.data_ptr(), total_q, q_out.data_ptr(), out_stride, k_cache.data_ptr(), v_cache.data_ptr(),
            _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_rope_store")
        return q_out

    def forward_tree(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, num_seqs, total_q, max_seqlen_q,
                     max_seqlen_k, flags, tree_mask, positions=None, sinks=None, alibi_slopes=None, out=None,
                     stream=None):
        """``forward`` for trees of drafted tokens: of its chunk's own keys a row sees
        those whose bits its row of ``tree_mask`` (int32 or uint32 [total_q, words])
        has.  ``positions`` (int32 [total_q]) are needed with a window or ALiBi.  q and
        ``out`` are contiguous."""
        device, row = q.get_device(), self.num_q_heads * self.head_size
        words = _mask_stride(tree_mask, total_q, device)
        places = None
        _check_table(block_table, num_seqs, self.max_blocks_per_seq, device)
        if not q.is_contiguous() or q.numel() < total_q * row:
            raise ValueError("q must be a contiguous [total_q, H_q, d]")
        _check(q, "q", "torch.bfloat16", device)
        self._check_caches(k_cache, v_cache, device)
        sink = slope = None
        if sinks is not None:
            sink = _head_terms(sinks, "sinks", self.num_q_heads, device)
        if alibi_slopes is not None:
            slope = _head_terms(alibi_slopes, "alibi_slopes", self.num_q_heads, device)
        i32 = _ints()[0]
        for t, n, name in ((cu_seqlens_q, num_seqs + 1, "cu_seqlens_q"), (seqused_k, num_seqs, "seqused_k")):
            if t.dtype is not i32 or t.numel() < n or not t.is_contiguous() or t.get_device() != device:
                _refuse_vector(t, name, n, "int32", device)
        if positions is not None:
            if positions.dtype is not i32 or positions.numel() < total_q or not positions.is_contiguous() or (
                    positions.get_device() != device):
                _refuse_vector(positions, "positions", total_q, "int32", device)
            places = positions.data_ptr()
        if out is None:
            out = _empty_like(q, stream)
        else:
            if not out.is_contiguous() or out.numel() < total_q * row:
                raise ValueError("out must be a contiguous [total_q, H_q, d]")
            _check(out, "out", "torch.bfloat16", device)
        st = load_library().ua_forward_tree(
            self.handle, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(),
            cu_seqlens_q.data_ptr(), seqused_k.data_ptr(), num_seqs, total_q, max_seqlen_q, max_seqlen_k,
            tree_mask.data_ptr(), words, places, flags, sink, slope, out.data_ptr(), _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_forward_tree")
        return out

    def cache_accept(self, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k, parents, last, num_seqs, total_q,
                     max_seqlen_q, max_seqlen_k, path, accepted, seqused_out, stream=None):
        """Keep the branch that ends at node ``last`` of every tree: its rows move
        right behind the context.  Out: ``path`` (int32 [num_seqs, n], -1 behind the
        branch), ``accepted`` (its length) and ``seqused_out``."""
        device = k_cache.get_device()
        self._check_caches(k_cache, v_cache, device)
        stride, nodes = _tree_rows(parents, num_seqs, device)
        if nodes < max_seqlen_q:
            raise ValueError("parents must have a column per node")
        _check_table(block_table, num_seqs, self.max_blocks_per_seq, device)
        wide = path.shape
        if len(wide) != 2 or wide[0] != num_seqs or wide[1] < 1:
            raise ValueError("path must be [num_seqs, n]")
        i32 = _ints()[0]
        for t, n, name in ((path, 1, "path"), (cu_seqlens_q, num_seqs + 1, "cu_seqlens_q"),
                           (seqused_k, num_seqs, "seqused_k"), (last, num_seqs, "last"),
                           (accepted, num_seqs, "accepted"), (seqused_out, num_seqs, "seqused_out")):
            if t.dtype is not i32 or t.numel() < n or not t.is_contiguous() or t.get_device() != device:
                _refuse_vector(t, name, n, "int32", device)
        st = load_library().ua_cache_accept(
            self.handle, k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), cu_seqlens_q.data_ptr(),
            seqused_k.data_ptr(), parents.data_ptr(), stride, last.data_ptr(), num_seqs, total_q, max_seqlen_q,
            max_seqlen_k, path.data_ptr(), wide[1], accepted.data_ptr(), seqused_out.data_ptr(), _stream(stream))
        if st != UA_OK:
            raise UAError(st, "ua_cache_accept")

    def forward_workload(self, w, out=None, stream=None):
        """Forward on a device-resident ``workloads.Workload`` (through
        ``ua_forward_topk`` when it carries top-k lists)."""
        qq = getattr(w, "qq_bias", None)
        flags = flags_of(w.causal, w.softcap, w.alibi_slopes is not None, w.window,
                         w.sinks is not None, qq is not None)
        if qq is not None:
            self.set_qq_bias(qq)
        if getattr(w, "topk_idx", None) is not None:
            return self.forward_topk(w.q, w.k_cache, w.v_cache, w.block_table, w.cu_seqlens_q,
                                     w.seqused_k, w.num_seqs, w.total_q, w.max_seqlen_q,
                                     w.max_seqlen_k, w.topk_idx, w.topk_len, flags, w.sinks,
                                     w.alibi_slopes, out, stream)
        return self.forward(w.q, w.k_cache, w.v_cache, w.block_table, w.cu_seqlens_q,
                            w.seqused_k, w.num_seqs, w.total_q, w.max_seqlen_q,
                            w.max_seqlen_k, flags, w.sinks, w.alibi_slopes, out, stream)

    def set_qq_bias(self, bias):
        """Bind a device fp32 matrix [n, >= n] (unit inner stride) as the
        query-query bias of later calls with UA_FLAG_QQ_BIAS; None clears it.
        The problem keeps a reference so the memory outlives its use."""
        if bias is None:
            st = ua_set_qq_bias(self.handle, None, 0, 0)
        else:
            if bias.dim() != 2 or bias.stride(1) != 1 or bias.shape[1] < bias.shape[0]:
                raise ValueError("qq bias must be [n, >= n] with unit inner stride")
            st = ua_set_qq_bias(self.handle, bias, bias.shape[0], bias.stride(0))
        if st != UA_OK:
            raise UAError(st, "ua_set_qq_bias")
        self._qq_bias = bias

    def check_device_error(self, stream=None):
        return ua_check_device_error(self.handle, stream)

    def last_launch_count(self):
        return load_library().ua_last_launch_count(self.handle)

    def set_profile_events(self, ev_begin=None, ev_end=None):
        """Record torch.cuda.Event pairs around the dominant kernel of later
        forward calls (None, None switches the hook off)."""
        b = ev_begin.cuda_event if ev_begin is not None else None
        e = ev_end.cuda_event if ev_end is not None else None
        st = load_library().ua_set_profile_events(self.handle, b, e)
        if st != UA_OK:
            raise UAError(st, "ua_set_profile_events")

    def last_path(self):
        return load_library().ua_last_path(self.handle).decode()

    def close(self):
        if self.handle:
            ua_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
