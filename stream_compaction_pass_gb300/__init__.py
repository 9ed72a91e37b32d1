"""Device-wide prefix sums and order-preserving stream compaction on one
NVIDIA GB300 (sm_103a): a thin ctypes binding of libstreamscan.so.

The functions carry the C ABI's names (include/streamscan.h) and only
marshal arguments: device pointers, element counts and the CUDA stream.
Every step of the computation runs in the library's CUDA kernels; there is
no CPU fallback.  If libstreamscan.so has not been built, every call raises
LibraryMissing (build it with ``python -m stream_compaction_pass_gb300.build``).

Arguments that are arrays may be torch tensors (CUDA tensors for device
pointers, CPU tensors or numpy arrays for host pointers) or raw integer
addresses.  For tensors, `n` defaults to the element count and `stream` to
torch's current stream on the tensor's device.
"""

from __future__ import annotations

import ctypes
import os
import re
import struct

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libstreamscan.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "streamscan.h")

SS_OK = 0
SS_ERR_INVALID_ARG = 1
SS_ERR_CUDA = 2
SS_ERR_LOOKBACK_TIMEOUT = 3
SS_ERR_NO_MEMORY = 4
SS_ERR_UNSUPPORTED = 5

SS_I32, SS_U32, SS_F32 = 0, 1, 2

SS_ALGO_LOOKBACK = 0
SS_ALGO_REDUCE_THEN_SCAN = 1
SS_ALGO_RTS_BLELLOCH = 2
SS_ALGO_RTS_BLELLOCH_PAD32 = 3
SS_ALGO_RTS_BLELLOCH_PAD2 = 4

SS_WIDE_U32_U64, SS_WIDE_I32_I64, SS_WIDE_I64, SS_WIDE_F64 = 0, 1, 2, 3

SS_BF16, SS_F16, SS_E4M3, SS_E2M1, SS_ELEM_F32 = 0, 1, 2, 3, 4


class LibraryMissing(ImportError):
    pass


class StreamScanError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status
        self.detail = detail


class _KvPages(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("weight", ctypes.c_void_p), ("k_block", ctypes.c_void_p), ("v_block", ctypes.c_void_p)]


class _KvTable(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("row_stride", ctypes.c_int64), ("max_pages", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("lens", ctypes.c_void_p), ("max_len", ctypes.c_int32)]


class _KvAttention(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int), ("q_heads", ctypes.c_int32), ("q", ctypes.c_void_p),
                ("q_seq_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("out_seq_stride", ctypes.c_int64), ("out_head_stride", ctypes.c_int64), ("scale", ctypes.c_float),
                ("window", ctypes.c_int32), ("sinks", ctypes.c_int32), ("lse", ctypes.c_void_p),
                ("weight_in", ctypes.c_void_p), ("weight_out", ctypes.c_void_p)]


class _KvFree(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("capacity", ctypes.c_int64), ("state", ctypes.c_void_p)]


_lib = None


def _declare(lib):
    P, SZ, I, U64, I64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64, ctypes.c_int64
    sigs = {
        "scan_inclusive_i32": [P, P, SZ, P],
        "scan_exclusive_i32": [P, P, SZ, P],
        "scan_inclusive_u32": [P, P, SZ, P],
        "scan_exclusive_u32": [P, P, SZ, P],
        "scan_inclusive_f32": [P, P, SZ, P],
        "scan_exclusive_f32": [P, P, SZ, P],
        "compact_u32": [P, P, P, P, SZ, P],
        "compact_positive_f32": [P, P, P, SZ, P],
        "ss_compact_positive": [I, P, P, P, SZ, P],
        "ss_compact_u32_unordered": [P, P, P, P, SZ, P],
        "ss_compact_positive_unordered": [I, P, P, P, SZ, P],
        "ss_moe_counts_offsets": [P, SZ, ctypes.c_int32, ctypes.c_uint32, P, P, P],
        "scan_inclusive_u32_u64": [P, P, SZ, P],
        "scan_exclusive_u32_u64": [P, P, SZ, P],
        "scan_inclusive_i64": [P, P, SZ, P],
        "scan_exclusive_i64": [P, P, SZ, P],
        "scan_inclusive_f64": [P, P, SZ, P],
        "scan_exclusive_f64": [P, P, SZ, P],
        "ss_scan_wide": [I, I, P, P, SZ, P],
        "ss_scan_rows": [I, I, P, P, SZ, SZ, P],
        "ss_scan_segments": [I, I, P, P, SZ, P, SZ, P],
        "ss_set_host_mode": [I],
        "ss_scan": [I, I, I, P, P, SZ, P],
        "ss_scan_seeded": [I, I, P, P, SZ, P, P, P],
        "ss_reduce_sum": [I, P, P, SZ, P],
        "ss_scan_host": [I, I, P, P, SZ, P],
        "ss_copy_u32": [P, P, SZ, P],
        "ss_scan_trace": [I, P, P, SZ, P, P],
        "ss_stream_status": [P, ctypes.POINTER(I64)],
        "ss_set_scan_config": [I],
        "ss_set_compact_config": [I],
        "ss_set_segments_config": [I],
        "ss_debug_set_lookback_fault": [I64, U64],
        "ss_scan_noalloc": [I, I, P, P, SZ, P],
        "ss_debug_set_noalloc_calls": [U64],
        "ss_scan_temp_bytes": [SZ, ctypes.POINTER(SZ)],
        "ss_scan_ws": [I, I, P, P, SZ, P, SZ, P],
        "ss_temp_status": [P, P, ctypes.POINTER(I64)],
        "ss_kv_append": [P, P, I, P, P, I64, I64, P, SZ, P],
        "ss_kv_attend": [P, P, P, P],
        "ss_kv_evict": [P, P, P, P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P, P],
        "ss_kv_assign": [P, P, ctypes.c_int32, I64, P, P, P, P, P, P, P, SZ, P],
        "ss_qk_norm_rope": [P, P, P, P],
        "ss_qk_norm_rope_backward": [P, P, P, P, P, P, P, P],
        "ss_kv_append_rope": [P, P, P, P, P, P],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = I
    lib.ss_status_string.argtypes = [I]
    lib.ss_status_string.restype = ctypes.c_char_p
    lib.ss_last_error_detail.argtypes = []
    lib.ss_last_error_detail.restype = ctypes.c_char_p
    lib.ss_scan_tile_elems.argtypes = []
    lib.ss_scan_tile_elems.restype = SZ
    lib.ss_scan_config_count.argtypes = []
    lib.ss_scan_config_count.restype = I
    lib.ss_shutdown.argtypes = []
    lib.ss_shutdown.restype = None
    lib.ss_debug_noalloc_clear_period.argtypes = []
    lib.ss_debug_noalloc_clear_period.restype = U64
    return lib


def lib():
    """The loaded libstreamscan.so (raises LibraryMissing if not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise LibraryMissing(
                f"{LIB_PATH} is not built; run `python -m stream_compaction_pass_gb300.build` "
                "(needs nvcc); there is no CPU fallback")
        _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def header_functions() -> list[str]:
    """Names of the functions include/streamscan.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\*?\s*([A-Za-z_][A-Za-z0-9_]*)\s*\(",
                                 text, flags=re.M)))


def _addr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    if hasattr(x, "ctypes"):
        return x.ctypes.data
    raise TypeError(f"cannot take the address of {type(x)!r}")


def _numel(x) -> int:
    if hasattr(x, "numel"):
        return int(x.numel())
    return int(x.size)


def _stream(stream, *tensors) -> int:
    if stream is not None:
        if isinstance(stream, int):
            return stream
        return int(stream.cuda_stream)
    for t in tensors:
        if hasattr(t, "is_cuda") and t.is_cuda:
            return _current_stream(t.get_device())
    return 0


_raw_stream = None  # torch's current stream of a device, by the cheapest call it offers


def _current_stream(device: int) -> int:
    global _raw_stream
    if _raw_stream is None:
        import torch
        # the Stream object that current_stream builds costs 2 us, a third of a small call
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda d: int(torch.cuda.current_stream(d).cuda_stream))
    return _raw_stream(device)


def _check(st: int, where: str) -> None:
    if st != SS_OK:
        detail = lib().ss_last_error_detail().decode() or lib().ss_status_string(st).decode()
        raise StreamScanError(st, where, detail)


def _scan_named(name: str, inp, out, n, stream) -> None:
    if n is None:
        n = _numel(inp)
    _check(getattr(lib(), name)(_addr(inp), _addr(out), n, _stream(stream, inp, out)), name)


def scan_inclusive_i32(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_i32", inp, out, n, stream)


def scan_exclusive_i32(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_i32", inp, out, n, stream)


def scan_inclusive_u32(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_u32", inp, out, n, stream)


def scan_exclusive_u32(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_u32", inp, out, n, stream)


def scan_inclusive_f32(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_f32", inp, out, n, stream)


def scan_exclusive_f32(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_f32", inp, out, n, stream)


def compact_u32(keys, flags, out, d_count, n=None, stream=None):
    if n is None:
        n = _numel(keys)
    _check(lib().compact_u32(_addr(keys), _addr(flags), _addr(out), _addr(d_count), n,
                             _stream(stream, keys, flags, out)), "compact_u32")


def compact_positive_f32(inp, out, d_count, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().compact_positive_f32(_addr(inp), _addr(out), _addr(d_count), n, _stream(stream, inp, out)),
           "compact_positive_f32")


def ss_compact_positive(dtype: int, inp, out, d_count, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_compact_positive(dtype, _addr(inp), _addr(out), _addr(d_count), n, _stream(stream, inp, out)),
           "ss_compact_positive")


def ss_compact_u32_unordered(keys, flags, out, d_count, n=None, stream=None):
    if n is None:
        n = _numel(keys)
    _check(lib().ss_compact_u32_unordered(_addr(keys), _addr(flags), _addr(out), _addr(d_count), n,
                                          _stream(stream, keys, flags, out)), "ss_compact_u32_unordered")


def ss_compact_positive_unordered(dtype: int, inp, out, d_count, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_compact_positive_unordered(dtype, _addr(inp), _addr(out), _addr(d_count), n,
                                               _stream(stream, inp, out)), "ss_compact_positive_unordered")


def scan_inclusive_u32_u64(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_u32_u64", inp, out, n, stream)


def scan_exclusive_u32_u64(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_u32_u64", inp, out, n, stream)


def scan_inclusive_i64(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_i64", inp, out, n, stream)


def scan_exclusive_i64(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_i64", inp, out, n, stream)


def scan_inclusive_f64(inp, out, n=None, stream=None):
    _scan_named("scan_inclusive_f64", inp, out, n, stream)


def scan_exclusive_f64(inp, out, n=None, stream=None):
    _scan_named("scan_exclusive_f64", inp, out, n, stream)


def ss_scan_wide(wide_type: int, inclusive: bool, inp, out, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_scan_wide(wide_type, int(bool(inclusive)), _addr(inp), _addr(out), n,
                              _stream(stream, inp, out)), "ss_scan_wide")


def ss_scan_rows(dtype: int, inclusive: bool, inp, out, rows: int, cols: int, stream=None):
    _check(lib().ss_scan_rows(dtype, int(bool(inclusive)), _addr(inp), _addr(out), rows, cols,
                              _stream(stream, inp, out)), "ss_scan_rows")


def ss_scan_segments(dtype: int, inclusive: bool, inp, out, offsets, num_segments=None, n=None, stream=None):
    """offsets: device uint64/int64 tensor of num_segments + 1 entries."""
    if n is None:
        n = _numel(inp)
    if num_segments is None:
        num_segments = _numel(offsets) - 1
    _check(lib().ss_scan_segments(dtype, int(bool(inclusive)), _addr(inp), _addr(out), n, _addr(offsets),
                                  num_segments, _stream(stream, inp, out)), "ss_scan_segments")


def ss_moe_counts_offsets(topk_ids, num_experts: int, align: int, counts, offsets, m=None, stream=None):
    if m is None:
        m = _numel(topk_ids)
    _check(lib().ss_moe_counts_offsets(_addr(topk_ids), m, num_experts, align, _addr(counts), _addr(offsets),
                                       _stream(stream, topk_ids, counts, offsets)), "ss_moe_counts_offsets")


def ss_scan(dtype: int, inclusive: bool, algo: int, inp, out, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_scan(dtype, int(bool(inclusive)), algo, _addr(inp), _addr(out), n,
                         _stream(stream, inp, out)), "ss_scan")


def ss_scan_seeded(dtype: int, inclusive: bool, inp, out, carry_in=None, carry_out=None, n=None,
                   stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_scan_seeded(dtype, int(bool(inclusive)), _addr(inp), _addr(out), n,
                                _addr(carry_in), _addr(carry_out), _stream(stream, inp, out)),
           "ss_scan_seeded")


def ss_reduce_sum(dtype: int, inp, d_total, n=None, stream=None):
    """Sum of `inp` (device) into d_total (device, one element)."""
    if n is None:
        n = _numel(inp)
    _check(lib().ss_reduce_sum(dtype, _addr(inp), _addr(d_total), n, _stream(stream, inp, d_total)),
           "ss_reduce_sum")


def ss_scan_host(dtype: int, inclusive: bool, h_in, h_out, n=None, stream=None):
    if n is None:
        n = _numel(h_in)
    _check(lib().ss_scan_host(dtype, int(bool(inclusive)), _addr(h_in), _addr(h_out), n,
                              _stream(stream)), "ss_scan_host")


def ss_copy_u32(inp, out, n=None, stream=None):
    if n is None:
        n = _numel(inp)
    _check(lib().ss_copy_u32(_addr(inp), _addr(out), n, _stream(stream, inp, out)), "ss_copy_u32")


def ss_scan_trace(config: int, inp, out, trace, n=None, stream=None):
    """Exclusive uint32 scan recording 8 uint64 per tile of look-back timing."""
    if n is None:
        n = _numel(inp)
    _check(lib().ss_scan_trace(config, _addr(inp), _addr(out), n, _addr(trace),
                               _stream(stream, inp, out)), "ss_scan_trace")


def ss_stream_status(stream=None):
    """Waits for the stream; returns (status, failing_tile) and clears it."""
    tile = ctypes.c_int64(-1)
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    st = lib().ss_stream_status(_stream(stream), ctypes.byref(tile))
    return st, tile.value


def ss_status_string(status: int) -> str:
    return lib().ss_status_string(status).decode()


def ss_last_error_detail() -> str:
    return lib().ss_last_error_detail().decode()


def ss_scan_tile_elems() -> int:
    return int(lib().ss_scan_tile_elems())


def ss_scan_config_count() -> int:
    return int(lib().ss_scan_config_count())


def ss_set_scan_config(config: int) -> None:
    _check(lib().ss_set_scan_config(config), "ss_set_scan_config")


def ss_set_host_mode(mode: int) -> None:
    _check(lib().ss_set_host_mode(mode), "ss_set_host_mode")


def ss_set_compact_config(config: int) -> None:
    _check(lib().ss_set_compact_config(config), "ss_set_compact_config")


def ss_set_segments_config(config: int) -> None:
    _check(lib().ss_set_segments_config(config), "ss_set_segments_config")


def ss_shutdown() -> None:
    lib().ss_shutdown()


def ss_debug_set_lookback_fault(tile: int, timeout_ns: int = 0) -> None:
    _check(lib().ss_debug_set_lookback_fault(tile, timeout_ns), "ss_debug_set_lookback_fault")


def ss_debug_set_noalloc_calls(calls: int) -> None:
    _check(lib().ss_debug_set_noalloc_calls(calls), "ss_debug_set_noalloc_calls")


def ss_debug_noalloc_clear_period() -> int:
    return int(lib().ss_debug_noalloc_clear_period())


def ss_scan_noalloc(dtype: int, inclusive: bool, inp, out, n=None, stream=None):
    """Single-pass scan whose scratch is a fixed device array: allocates
    nothing (n <= 2^30; the first call on a device sets that device up)."""
    if n is None:
        n = _numel(inp)
    st = lib().ss_scan_noalloc(dtype, int(bool(inclusive)), _addr(inp), _addr(out), n,
                               _stream(stream, inp, out))
    if st != SS_OK:
        raise StreamScanError(st, "ss_scan_noalloc", ss_status_string(st))


def ss_scan_temp_bytes(n: int) -> int:
    """Device scratch bytes that ss_scan_ws needs for n elements."""
    b = ctypes.c_size_t(0)
    _check(lib().ss_scan_temp_bytes(n, ctypes.byref(b)), "ss_scan_temp_bytes")
    return int(b.value)


def ss_scan_ws(dtype: int, inclusive: bool, inp, out, temp, n=None, temp_bytes=None, stream=None):
    """The library's scan with caller-provided scratch `temp` (device,
    256-byte aligned, at least ss_scan_temp_bytes(n) bytes)."""
    if n is None:
        n = _numel(inp)
    if temp_bytes is None:
        temp_bytes = temp.numel() * temp.element_size()
    st = lib().ss_scan_ws(dtype, int(bool(inclusive)), _addr(inp), _addr(out), n, _addr(temp), temp_bytes,
                          _stream(stream, inp, out))
    if st != SS_OK:
        raise StreamScanError(st, "ss_scan_ws", ss_status_string(st))


def ss_temp_status(temp, stream=None):
    """Waits for the stream; returns (status, failing_tile) held in `temp`
    and clears it."""
    tile = ctypes.c_int64(-1)
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    st = lib().ss_temp_status(_addr(temp), _stream(stream), ctypes.byref(tile))
    return st, tile.value


_elems = {}   # torch dtype -> the library's element type
_dtypes = {}  # name -> torch dtype


def _load_dtypes() -> None:
    import torch
    _elems.update({torch.bfloat16: SS_BF16, torch.float16: SS_F16, torch.float8_e4m3fn: SS_E4M3})
    _dtypes.update({"float32": torch.float32, "int32": torch.int32, "int64": torch.int64})


def _elem(t) -> int:
    """The library's element type of a torch tensor."""
    if not _elems:
        _load_dtypes()
    kind = _elems.get(t.dtype)
    if kind is None:
        raise TypeError(f"{t.dtype} is not a type of the key-value cache calls (bfloat16, float16, float8_e4m3fn)")
    return kind


def _like(name: str, t, shape, dtype: str, device: int) -> int:
    """The address of an optional contiguous tensor argument (0 for None), its
    shape, type and device checked; the C ABI sees only addresses."""
    if t is None:
        return 0
    if not _dtypes:
        _load_dtypes()
    if t.shape != shape or t.dtype is not _dtypes[dtype] or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                         f"{str(t.dtype)[6:]} {tuple(t.shape)}")
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    return t.data_ptr()


def _elsewhere(name: str, t, device: int) -> ValueError:
    return ValueError(f"{name} is on {t.device}, where {'the CPU' if device < 0 else f'cuda:{device}'} was expected")


def _refuse(device: int, **args) -> None:
    """Raises for the argument (a tensor, KVPages or KVTable) that is not on the cache's GPU."""
    if device < 0:
        raise ValueError("the cache is not on a GPU")
    for name, x in args.items():
        t = x if hasattr(x, "get_device") else x.k if isinstance(x, KVPages) else x.pages
        if t.get_device() != device:
            raise _elsewhere(name, t, device)


def _int32(**values) -> None:
    """Checks integers that the C ABI takes in 32 bits, where ctypes would keep the low ones."""
    for name, x in values.items():
        if not -1 << 31 <= x < 1 << 31:
            raise ValueError(f"{name} = {x} is not a 32-bit integer")


class KVPages:
    """The pool of a paged key-value cache (ss_kv_pages).

    k, v    CUDA tensors of shape (num_pages, kv_heads, page_size, head_dim),
            bfloat16, float16 or float8_e4m3fn, with the same strides (any
            order of the first three dimensions; the last one contiguous).
            Of 4-bit caches uint8 (..., head_dim / 2): two codes to a byte, the
            lower index in the low half.
    weight  float32 (num_pages, kv_heads, page_size), contiguous, or None.
    k_scale, v_scale  float32 (kv_heads,), for a float8 or 4-bit cache, or None (1).
    k_block, v_block  of a 4-bit cache: float8_e4m3fn (num_pages, kv_heads,
            page_size, head_dim / 16), contiguous: a scale for every 16 elements.
    The tensors are kept alive and may be updated in place.
    """

    def __init__(self, k, v, weight=None, k_scale=None, v_scale=None, k_block=None, v_block=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must be 4-dimensional, of one shape and type")
        if k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must have the same strides and a contiguous last dimension")
        pages, heads, page, dim = k.shape
        strides = k.stride()[:3]
        self.device = k.get_device()  # -1: the CPU, where no call works
        if (k_block is None) != (v_block is None):
            raise ValueError("a 4-bit cache has both k_block and v_block")
        blocks = [0, 0]
        if k_block is not None:
            if str(k.dtype) != "torch.uint8":
                raise TypeError(f"a cache with k_block and v_block holds uint8 pairs of codes, not {k.dtype}")
            dim, strides, kind = dim * 2, [2 * x for x in strides], SS_E2M1
            for i, (name, x) in enumerate((("k_block", k_block), ("v_block", v_block))):
                if x.shape != (pages, heads, page, dim // 16) or str(x.dtype) != "torch.float8_e4m3fn" or not x.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous float8_e4m3fn tensor of shape {(pages, heads, page, dim // 16)}, got "
                                     f"{str(x.dtype)[6:]} {tuple(x.shape)}")
                if x.get_device() != self.device:
                    raise _elsewhere(name, x, self.device)
                blocks[i] = x.data_ptr()
        else:
            kind = _elem(k)
        if v.get_device() != self.device:
            raise _elsewhere("v", v, self.device)
        d_weight = _like("weight", weight, (pages, heads, page), "float32", self.device)
        d_scales = [_like(name, x, (heads,), "float32", self.device) for name, x in (("k_scale", k_scale), ("v_scale", v_scale))]
        self.k, self.v, self.weight, self.k_scale, self.v_scale = k, v, weight, k_scale, v_scale
        self.k_block, self.v_block = k_block, v_block
        self.kv_heads, self.head_dim, self.weight_shape = heads, dim, k.shape[:3]
        self._c = _KvPages(kind, heads, dim, page, pages, _addr(k), _addr(v), *strides, *d_scales, d_weight, *blocks)
        self._ref = ctypes.addressof(self._c)


class KVTable:
    """The sequences of a paged key-value cache (ss_kv_table).

    pages    int32 (batch, max_pages): page numbers, rows may be strided.
    lens     int32 (batch,): lengths, read by every call at the time it runs.
    max_len  an upper bound on the lengths (default: max_pages * page_size);
             set it to the longest length in use to size launches by it.
    """

    def __init__(self, pages, lens, max_len=None):
        if pages.dim() != 2 or str(pages.dtype) != "torch.int32" or (pages.shape[1] > 1 and pages.stride(1) != 1):
            raise ValueError("pages must be a 2-dimensional int32 tensor with contiguous rows")
        self.device = pages.get_device()
        _like("lens", lens, (pages.shape[0],), "int32", self.device)
        _int32(max_len=max_len or 0)
        self.pages, self.lens, self.batch = pages, lens, pages.shape[0]
        self._c = _KvTable(_addr(pages), pages.stride(0), pages.shape[1], pages.shape[0], _addr(lens),
                           0 if max_len is None else max_len)
        self._ref = ctypes.addressof(self._c)

    @property
    def max_len(self):
        return self._c.max_len

    @max_len.setter
    def max_len(self, n):
        _int32(max_len=n)
        self._c.max_len = n


def ss_kv_append(cache: KVPages, seqs: KVTable, k_new, v_new, offsets=None, stream=None) -> None:
    """Writes new tokens' rows, (tokens, kv_heads, head_dim) tensors of one
    type and strides, to the last positions of their sequences; offsets is
    int32 (batch + 1,), or None for one token per sequence."""
    if k_new.dim() != 3 or k_new.shape != v_new.shape or k_new.dtype != v_new.dtype or k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must be 3-dimensional, of one shape, type and strides")
    tokens, heads, dim = k_new.shape
    token_stride, head_stride, unit = k_new.stride()
    if heads != cache.kv_heads or dim != cache.head_dim or unit != 1:
        raise ValueError(f"k_new must be (tokens, {cache.kv_heads}, {cache.head_dim}) with a contiguous last dimension")
    device = cache.device
    if device < 0 or seqs.device != device or k_new.get_device() != device or v_new.get_device() != device:
        _refuse(device, seqs=seqs, k_new=k_new, v_new=v_new)
    d_offsets = _like("offsets", offsets, (seqs.batch + 1,), "int32", device)
    _check(lib().ss_kv_append(cache._ref, seqs._ref, _elem(k_new), k_new.data_ptr(), v_new.data_ptr(), token_stride,
                              head_stride, d_offsets, tokens, _current_stream(device) if stream is None else _stream(stream)), "ss_kv_append")


def ss_kv_attend(cache: KVPages, seqs: KVTable, q, out, scale=None, window: int = 0, sinks: int = 0, lse=None,
                 weight_in=None, weight_out=None, stream=None) -> None:
    """Attention of q, (batch, q_heads, head_dim), over the cached positions
    into out; scale defaults to head_dim ** -0.5.  lse: float32 (batch,
    q_heads).  weight_out, weight_in: float32 tensors of the pool's weight
    shape (weight_out = weight_in = cache.weight accumulates in place);
    sequences may share pages only without them."""
    if q.dim() != 3 or q.shape != out.shape or q.dtype != out.dtype:
        raise ValueError("q and out must be 3-dimensional, of one shape and type")
    batch, heads, dim = q.shape
    q_seq, q_head, q_unit = q.stride()
    out_seq, out_head, out_unit = out.stride()
    if batch != seqs.batch or dim != cache.head_dim or q_unit != 1 or out_unit != 1:
        raise ValueError(f"q and out must be ({seqs.batch}, q_heads, {cache.head_dim}) with a contiguous last dimension")
    if window >> 31 or sinks >> 31:  # also the negative ones
        _int32(window=window, sinks=sinks)
    device = cache.device
    if device < 0 or seqs.device != device or q.get_device() != device or out.get_device() != device:
        _refuse(device, seqs=seqs, q=q, out=out)
    d_lse = _like("lse", lse, (batch, heads), "float32", device)
    d_in, d_out = (_like("weight_in", weight_in, cache.weight_shape, "float32", device),
                   _like("weight_out", weight_out, cache.weight_shape, "float32", device))
    a = _KvAttention(_elem(q), heads, q.data_ptr(), q_seq, q_head, out.data_ptr(), out_seq, out_head,
                     dim ** -0.5 if scale is None else scale, window, sinks, d_lse, d_in, d_out)
    _check(lib().ss_kv_attend(cache._ref, seqs._ref, ctypes.addressof(a),
                              _current_stream(device) if stream is None else _stream(stream)), "ss_kv_attend")


def ss_kv_evict(src: KVPages, src_seqs: KVTable, dst: KVPages, dst_seqs: KVTable, keep: int, sinks: int = 0,
                recent: int = 0, kept=None, stream=None) -> None:
    """Moves the kept rows of every sequence and head into dst's pages and
    their number into dst_seqs.lens; kept: int32 (batch, kv_heads, keep)."""
    if keep >> 31 or sinks >> 31 or recent >> 31:
        _int32(keep=keep, sinks=sinks, recent=recent)
    device = src.device
    if device < 0 or src_seqs.device != device or dst.device != device or dst_seqs.device != device:
        _refuse(device, src_seqs=src_seqs, dst=dst, dst_seqs=dst_seqs)
    d_kept = _like("kept", kept, (src_seqs.batch, src.kv_heads, keep), "int32", device)
    _check(lib().ss_kv_evict(src._ref, src_seqs._ref, dst._ref, dst_seqs._ref, keep, sinks, recent, d_kept,
                             _current_stream(device) if stream is None else _stream(stream)), "ss_kv_evict")


class KVFree:
    """The free pages of a pool, a ring (ss_kv_free).

    pages      int32 (capacity,), contiguous: page numbers; capacity is at least
               the number of pages that are handed out this way.
    state      int32 (2,): the place of the first free page, and how many there
               are from it on (going around the end).
    num_pages  of the pool (default: capacity).
    """

    def __init__(self, pages, state, num_pages=None):
        self.device = pages.get_device()
        _like("pages", pages, (pages.numel(),), "int32", self.device)
        _like("state", state, (2,), "int32", self.device)
        self.pages, self.state, self.num_pages = pages, state, pages.numel() if num_pages is None else num_pages
        _int32(num_pages=self.num_pages)
        self._c = _KvFree(pages.data_ptr(), pages.numel(), state.data_ptr())
        self._ref = ctypes.addressof(self._c)

    def get_device(self):
        return self.device


def ss_kv_assign(seqs: KVTable, free: KVFree, page_size: int, counts=None, restart=None, into: KVTable = None, left=None, offsets=None,
                 positions=None, slots=None, stream=None) -> None:
    """Pages for counts more tokens of every sequence (int32 (batch,); None: one
    each), from the front of the ring of free pages; those of sequences with
    restart set (bool (batch,)) go to its end.  into receives table and lengths,
    left (int32 (2,)) the ring's state; by default both are updated in place.
    offsets: int32 (batch + 1,); positions int32 and slots int64, (tokens,) each."""
    device = seqs.device
    to = seqs if into is None else into
    if device < 0 or free.device != device or to.device != device:
        _refuse(device, free=free, into=to)
    if page_size >> 31:
        _int32(page_size=page_size)
    batch = (seqs.batch,)
    tokens = (positions if slots is None else slots).numel() if positions is not None or slots is not None else 0
    if restart is not None and (restart.shape != batch or str(restart.dtype) not in ("torch.bool", "torch.uint8") or not restart.is_contiguous()):
        raise ValueError(f"restart must be a contiguous bool tensor of shape {batch}")
    if restart is not None and restart.get_device() != device:
        raise _elsewhere("restart", restart, device)
    d = (_like("counts", counts, batch, "int32", device), 0 if restart is None else restart.data_ptr(), _like("left", left, (2,), "int32", device),
         _like("offsets", offsets, (seqs.batch + 1,), "int32", device), _like("positions", positions, (tokens,), "int32", device),
         _like("slots", slots, (tokens,), "int64", device))
    _check(lib().ss_kv_assign(seqs._ref, to._ref, page_size, free.num_pages, d[0], d[1], free._ref, d[2], d[3], d[4], d[5], tokens,
                              _current_stream(device) if stream is None else _stream(stream)), "ss_kv_assign")


class Rope:
    """The rotation's frequencies (ss_rope).

    inv_freq     the angles of one position in radians, (rotary_dim / 2,), on the
                 GPU; best float64, as far positions multiply its error.  What is
                 derived from it is made on the current stream.
    interleaved  pairs are adjacent elements (else rotary_dim / 2 apart).
    """

    def __init__(self, inv_freq, interleaved: bool = False):
        import math

        import torch
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must have one dimension")
        x = inv_freq.detach().to(torch.float64) / (2 * math.pi)
        x = x - torch.floor(x + 0.5)
        self.device = x.get_device()
        self.turns = (x * 2.0 ** 64).to(torch.int64)  # modulo one turn; exact
        self.rotary_dim, self.interleaved = 2 * x.numel(), bool(interleaved)
        self._c = self.turns.data_ptr(), self.rotary_dim, int(self.interleaved)


# ss_qk and ss_rows as bytes, which cost less to make than ctypes structures
_QK = struct.Struct("@iiiiifqPqqPqqPPPPii")
_ROWS = struct.Struct("@Pqq")
_NO_ROWS = (0, 0, 0)
_row_kinds = {}  # torch dtype -> element type, of rows and weights


def _row_kind(name: str, dtype) -> int:
    if not _row_kinds:
        import torch
        _row_kinds.update({torch.bfloat16: SS_BF16, torch.float16: SS_F16, torch.float32: SS_ELEM_F32})
    kind = _row_kinds.get(dtype)
    if kind is None:
        raise TypeError(f"{name} is {dtype}: bfloat16, float16 and float32 are taken")
    return kind


def _place(name: str, t):
    """Address and strides of a (tokens, heads, head_dim) tensor."""
    token, head, unit = t.stride()
    if unit != 1:
        raise ValueError(f"{name} must have a contiguous last dimension")
    return t.data_ptr(), token, head


def _rows(name: str, t, shape, dtype, device: int):
    """The place of rows whose shape, type and device are checked; shape None: no heads."""
    if t is None or shape is None:
        if (t is None) != (shape is None):
            raise ValueError(f"{name} is missing" if t is None else f"{name} has no input")
        return _NO_ROWS
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {str(dtype)[6:]} of shape {tuple(shape)}, got {str(t.dtype)[6:]} {tuple(t.shape)}")
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    return _place(name, t)


def _weight(name: str, t, dim, dtype, device: int) -> int:
    if t.dtype is not dtype or t.shape != dim or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {dim}, and of the other weight's type")
    if t.get_device() != device:
        raise _elsewhere(name, t, device)
    return t.data_ptr()


def _qk(q, k, q_weight, k_weight, rope, positions, eps: float):
    """The description of q and k (either may be None), their shapes, type and device."""
    one = k if q is None else q
    if one is None:
        raise ValueError("q and k are both None")
    shape, dtype, device = one.shape, one.dtype, one.get_device()
    q_shape, k_shape = None if q is None else shape, None if k is None else k.shape
    if len(shape) != 3 or (k is not None and len(k_shape) != 3):
        raise ValueError("q and k must be (tokens, heads, head_dim)")
    tokens, heads, dim = shape
    kv_heads = 0
    if k is not None:
        of, kv_heads, wide = k_shape
        if of != tokens or wide != dim or k.dtype is not dtype:
            raise ValueError(f"q and k must be of the same tokens, head_dim and type, got {str(dtype)[6:]} {tuple(shape)} and {str(k.dtype)[6:]} {tuple(k_shape)}")
        if k.get_device() != device:
            raise _elsewhere("k", k, device)
    if device < 0:
        raise ValueError("q and k are not on a GPU")
    if rope.device != device:
        raise _elsewhere("rope", rope.turns, device)
    kind, weight, d_q, d_k = _row_kind("q" if q is not None else "k", dtype), SS_ELEM_F32, 0, 0
    if q_weight is not None or k_weight is not None:
        weight_type = (k_weight if q_weight is None else q_weight).dtype
        weight = kind if weight_type is dtype else _row_kind("q_weight", weight_type)
        if q_weight is not None:
            d_q = _weight("q_weight", q_weight, (dim,), weight_type, device)
        if k_weight is not None:
            d_k = _weight("k_weight", k_weight, (dim,), weight_type, device)
    c = _QK.pack(kind, weight, dim, 0 if q is None else heads, kv_heads, eps, tokens, *(_NO_ROWS if q is None else _place("q", q)),
                 *(_NO_ROWS if k is None else _place("k", k)), d_q, d_k, _like("positions", positions, (tokens,), "int32", device), *rope._c)
    return c, q_shape, k_shape, dtype, device


def ss_qk_norm_rope(q, k, q_weight, k_weight, rope: Rope, positions, q_out, k_out, eps: float = 1e-6, stream=None) -> None:
    """Root-mean-square norms of the heads' rows of q and k, (tokens, heads,
    head_dim), times their weights (head_dim,) or None, rotated by positions, int32
    (tokens,), into q_out and k_out (which may be q and k).  Either of q and k may
    be None."""
    c, qs, ks, dtype, device = _qk(q, k, q_weight, k_weight, rope, positions, eps)
    _check(lib().ss_qk_norm_rope(c, _ROWS.pack(*_rows("q_out", q_out, qs, dtype, device)), _ROWS.pack(*_rows("k_out", k_out, ks, dtype, device)),
                                 _current_stream(device) if stream is None else _stream(stream)), "ss_qk_norm_rope")


def ss_qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, rope: Rope, positions, dq, dk, dq_weight=None, dk_weight=None,
                             eps: float = 1e-6, stream=None) -> None:
    """The gradients of ss_qk_norm_rope from those of its outputs: dq and dk (which
    may be dq_out and dk_out), and float32 dq_weight and dk_weight (head_dim,)."""
    c, qs, ks, dtype, device = _qk(q, k, q_weight, k_weight, rope, positions, eps)
    dim = (ks if qs is None else qs)[2:]
    _check(lib().ss_qk_norm_rope_backward(c, _ROWS.pack(*_rows("dq_out", dq_out, qs, dtype, device)), _ROWS.pack(*_rows("dk_out", dk_out, ks, dtype, device)),
                                          _ROWS.pack(*_rows("dq", dq, qs, dtype, device)), _ROWS.pack(*_rows("dk", dk, ks, dtype, device)),
                                          _like("dq_weight", dq_weight, dim, "float32", device), _like("dk_weight", dk_weight, dim, "float32", device),
                                          _current_stream(device) if stream is None else _stream(stream)), "ss_qk_norm_rope_backward")


def ss_kv_append_rope(cache: KVPages, slots, q, k, v, q_weight, k_weight, rope: Rope, positions, q_out, eps: float = 1e-6, stream=None) -> None:
    """ss_qk_norm_rope whose k rows go to the cache, with v's as they are, at slots,
    int64 (tokens,), as ss_kv_assign gives them (-1: nowhere).  q may be None."""
    if k is None:
        raise ValueError("k is missing")
    c, qs, ks, dtype, device = _qk(q, k, q_weight, k_weight, rope, positions, eps)
    if cache.device != device:
        raise _elsewhere("cache.k", cache.k, device)
    _check(lib().ss_kv_append_rope(cache._ref, _like("slots", slots, ks[:1], "int64", device), c, _ROWS.pack(*_rows("v", v, ks, dtype, device)),
                                   _ROWS.pack(*_rows("q_out", q_out, qs, dtype, device)),
                                   _current_stream(device) if stream is None else _stream(stream)), "ss_kv_append_rope")
