"""ctypes binding of ``include/ua.h`` (argument marshalling only).

Every function here forwards to the C ABI of ``libua.so``; all arithmetic runs
in that library's CUDA kernels.  Tensors are torch tensors (device memory for
``ua_forward``, host memory for ``ua_forward_host``); streams are torch CUDA
streams or raw ``cudaStream_t`` integers.
"""
import ctypes
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
    n, heads, dims = t.shape
    if (stride[2] != 1 or (heads > 1 and stride[1] != dims) or n < total_q or
            (num_kv_heads is not None and (heads != num_kv_heads or dims != head_size))):
        raise ValueError("%s must be [total_q, H_k, d] with contiguous heads" % name)
    return stride[0] if n > 1 else max(stride[0], heads * dims)


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
        self.head_size = head_size
        self.block_size = block_size
        self.max_blocks_per_seq = max_blocks_per_seq
        self.num_q_heads = num_q_heads
        self.num_kv_heads = num_kv_heads

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
        if out is None:
            import torch
            out = torch.empty_like(q)
        st = ua_forward(self.handle, q, k_cache, v_cache, block_table, cu_seqlens_q,
                        seqused_k, num_seqs, total_q, max_seqlen_q, max_seqlen_k, flags,
                        sinks, alibi_slopes, out, stream)
        if st != UA_OK:
            raise UAError(st, "ua_forward")
        return out

    def forward_topk(self, q, k_cache, v_cache, block_table, cu_seqlens_q, seqused_k,
                     num_seqs, total_q, max_seqlen_q, max_seqlen_k, topk_idx, topk_len, flags,
                     sinks=None, alibi_slopes=None, out=None, stream=None):
        if out is None:
            import torch
            out = torch.empty_like(q)
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
        rows = num_seqs, self.num_kv_heads, max_seqlen_k, q
        stride = _weight_rows(weights_out, "weights_out", *rows)
        if weights_in is not None and _weight_rows(weights_in, "weights_in", *rows) != stride:
            raise ValueError("weights_in and weights_out must share a row stride")
        if out is None:
            import torch
            out = torch.empty_like(q)
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
