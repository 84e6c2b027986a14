"""Python binding of libexl3.so, the sm_103a trellis-quantized linear layer.

The functions here carry the C ABI's names (include/exl3.h) and only marshal
arguments: tensors become device pointers, the stream defaults to torch's
current stream, and a non-zero status raises ``Exl3Error``. Every step of
the computation runs in the library's CUDA kernels; there is no fallback. If
``libexl3.so`` has not been built, loading it raises immediately.

With ``EXL3_BOUNDS_CHECKED=1`` in the environment the package builds and
loads ``libexl3_bounds.so`` instead: the same kernels with every access
checked against its launch's extents (a failed check records
EXL3_ERR_OUT_OF_BOUNDS in the device error word).
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

__all__ = [
    "Exl3Error", "build", "load", "EXL3_F16", "EXL3_F32", "EXL3_LAYOUT_KN", "EXL3_LAYOUT_NK",
    "EXL3_RECONSTRUCT_CHUNK_COLS", "EXL3_NOALLOC_SCRATCH_BYTES", "exl3_init", "exl3_status_string", "exl3_supported_bits",
    "exl3_aligned_logits_width", "exl3_decode_plan", "exl3_prefill_path", "exl3_linear_workspace_bytes_for",
    "exl3_linear_workspace_bytes", "exl3_workspace_init", "exl3_hadamard128", "exl3_reconstruct",
    "exl3_linear", "exl3_logits_masked", "exl3_get_device_status", "exl3_selftest_wait_timeout",
    "exl3_linear_decode_noalloc", "exl3_silu_mul", "exl3_reconstruct_rotated",
    "exl3_weight_rotated_workspace_bytes", "exl3_linear_weight_rotated", "exl3_bounds_checked",
    "exl3_selftest_bounds", "EXL3_KV8_BLOCK", "Exl3Kv8Cache", "Exl3Kv8Batch", "exl3_kv8_append",
    "exl3_kv8_attention_workspace_bytes", "exl3_kv8_attention", "exl3_kv8_weigh", "exl3_kv8_evict",
    "exl3_logits_adjust", "exl3_selftest_bounds_serving", "HEADER_SYMBOLS", "BOUNDS_CHECKED",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
BOUNDS_CHECKED = os.environ.get("EXL3_BOUNDS_CHECKED", "0") == "1"
LIB_PATH = os.path.join(_PKG, "libexl3_bounds.so" if BOUNDS_CHECKED else "libexl3.so")

EXL3_F16 = 0
EXL3_F32 = 1
EXL3_LAYOUT_KN = 0
EXL3_LAYOUT_NK = 1
EXL3_RECONSTRUCT_CHUNK_COLS = 32768
EXL3_NOALLOC_SCRATCH_BYTES = 24 << 20
EXL3_KV8_BLOCK = 64

STATUS_NAMES = {
    0: "EXL3_OK", 1: "EXL3_ERR_INVALID_ARG", 2: "EXL3_ERR_ALIGNMENT", 3: "EXL3_ERR_UNSUPPORTED_BITS",
    4: "EXL3_ERR_WORKSPACE_TOO_SMALL", 5: "EXL3_ERR_NOT_INITIALIZED", 6: "EXL3_ERR_CUDA",
    7: "EXL3_ERR_DEVICE_TIMEOUT", 8: "EXL3_ERR_NOALLOC_TOO_LARGE", 9: "EXL3_ERR_OUT_OF_BOUNDS",
    10: "EXL3_ERR_DEVICE_INDEX",
}

# Every function include/exl3.h declares.
HEADER_SYMBOLS = (
    "exl3_init", "exl3_status_string", "exl3_supported_bits", "exl3_aligned_logits_width",
    "exl3_decode_plan", "exl3_prefill_path", "exl3_linear_workspace_bytes_for", "exl3_linear_workspace_bytes",
    "exl3_workspace_init", "exl3_hadamard128", "exl3_reconstruct", "exl3_linear",
    "exl3_logits_masked", "exl3_get_device_status", "exl3_selftest_wait_timeout",
    "exl3_linear_decode_noalloc", "exl3_silu_mul", "exl3_reconstruct_rotated",
    "exl3_weight_rotated_workspace_bytes", "exl3_linear_weight_rotated", "exl3_bounds_checked",
    "exl3_selftest_bounds", "exl3_kv8_append", "exl3_kv8_attention_workspace_bytes", "exl3_kv8_attention",
    "exl3_kv8_weigh", "exl3_kv8_evict", "exl3_logits_adjust", "exl3_selftest_bounds_serving",
)


class Exl3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = int(status)
        self.name = STATUS_NAMES.get(self.status, f"status {status}")
        super().__init__(f"{where}: {self.name} ({_status_text(self.status)})")


_lib = None
_lock = threading.Lock()
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_vp = ctypes.c_void_p


class Exl3Kv8Cache(ctypes.Structure):
    """exl3_kv8_cache over the caller's tensors (kept alive by this object):
    k, v n_pages x n_kv_heads x 64 x head_dim (torch.float8_e4m3fn or uint8),
    k_scale, v_scale n_pages x n_kv_heads fp32, weight n_pages x n_kv_heads x
    64 fp32 or None; all contiguous."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("weight", _vp), ("n_pages", _i64),
                ("n_kv_heads", _i32), ("head_dim", _i32)]

    def __init__(self, k, v, k_scale, v_scale, weight=None):
        if k.dim() != 4 or k.shape[2] != EXL3_KV8_BLOCK or v.shape != k.shape or k.element_size() != 1 or v.element_size() != 1:
            raise ValueError("Exl3Kv8Cache: k and v are n_pages x n_kv_heads x 64 x head_dim, one byte an element")
        if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2] or (weight is not None and weight.shape != k.shape[:3]):
            raise ValueError("Exl3Kv8Cache: scales are n_pages x n_kv_heads, weight n_pages x n_kv_heads x 64")
        _require_f32_contiguous("Exl3Kv8Cache", k_scale, v_scale, weight)
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("Exl3Kv8Cache: k and v are contiguous")
        super().__init__(_ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale), _ptr(weight), k.shape[0], k.shape[1], k.shape[3])
        self._keep = (k, v, k_scale, v_scale, weight)
        self._ref = ctypes.byref(self)


class Exl3Kv8Batch(ctypes.Structure):
    """exl3_kv8_batch over the caller's int32 tensors (kept alive by this
    object): page_table n_seqs x max_pages, kv_len n_seqs, q_start n_seqs + 1;
    their contents may change between calls. rows and max_rows bound this
    call's rows, in total and for one sequence."""
    _fields_ = [("page_table", _vp), ("kv_len", _vp), ("q_start", _vp), ("n_seqs", _i32), ("max_pages", _i32),
                ("rows", _i32), ("max_rows", _i32)]

    def __init__(self, page_table, kv_len, q_start=None, rows=0, max_rows=0):
        n = page_table.shape[0]
        if page_table.dim() != 2 or kv_len.numel() != n or (q_start is not None and q_start.numel() != n + 1):
            raise ValueError("Exl3Kv8Batch: page_table is n_seqs x max_pages, kv_len n_seqs, q_start n_seqs + 1")
        for t in (page_table, kv_len, q_start):
            if t is not None and (t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous()):
                raise ValueError("Exl3Kv8Batch: tensors are contiguous int32")
        super().__init__(_ptr(page_table), _ptr(kv_len), _ptr(q_start), n, page_table.shape[1], rows, max_rows)
        self._keep = (page_table, kv_len, q_start)
        self._ref = ctypes.byref(self)


class _LogitsRules(ctypes.Structure):
    _fields_ = [("history", _vp), ("history_start", _vp), ("generated_from", _vp), ("repetition", _vp),
                ("presence", _vp), ("frequency", _vp), ("bias_id", _vp), ("bias_value", _vp), ("bias_start", _vp),
                ("allowed", _vp), ("history_size", _i32), ("bias_size", _i32)]


_PACK_RULES = struct.Struct("@10P2i").pack  # a _LogitsRules' bytes, in a quarter of the time


def _require_f32_contiguous(where, *tensors):
    for t in tensors:
        if t is not None and (t.element_size() != 4 or not t.is_floating_point() or not t.is_contiguous()):
            raise ValueError(f"{where}: expected contiguous fp32 tensors")


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library this process loads (libexl3.so, or libexl3_bounds.so
    under EXL3_BOUNDS_CHECKED=1) for sm_103a with nvcc (in-tree)."""
    if _lib is not None and not force:
        return LIB_PATH  # this process has loaded it
    from . import _build
    return _build.build(force=force, verbose=verbose, bounds_checked=BOUNDS_CHECKED)


def load():
    """Loads the library (LIB_PATH); raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with trellis_quantized_linear_gb300.build()")
        lib = ctypes.CDLL(LIB_PATH)
        sig = {
            "exl3_init": (ctypes.c_int, [ctypes.c_int]),
            "exl3_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "exl3_supported_bits": (ctypes.c_int, [ctypes.c_int]),
            "exl3_aligned_logits_width": (_i64, [_i64, _i64]),
            "exl3_decode_plan": (ctypes.c_int, [_i64, _i64, ctypes.c_int, ctypes.POINTER(ctypes.c_int),
                                                ctypes.POINTER(ctypes.c_int)]),
            "exl3_prefill_path": (ctypes.c_int, [_i64, _i64, ctypes.c_int]),
            "exl3_linear_workspace_bytes_for": (ctypes.c_size_t, [_i64, _i64, _i64, ctypes.c_int, _i64, ctypes.c_int]),
            "exl3_linear_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, _i64, ctypes.c_int, _i64]),
            "exl3_workspace_init": (ctypes.c_int, [_vp, ctypes.c_size_t, _vp]),
            "exl3_hadamard128": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _vp]),
            "exl3_reconstruct": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, ctypes.c_int, _vp]),
            "exl3_linear": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_int, _i64, _i64, _vp, _vp, _vp,
                                           ctypes.c_int, _i64, _vp, ctypes.c_size_t, _vp]),
            "exl3_logits_masked": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_int, _i64, _i64, _i64, _vp, _vp,
                                                  _vp, _vp, _i64, _vp, ctypes.c_size_t, _vp]),
            "exl3_get_device_status": (ctypes.c_int, [_vp]),
            "exl3_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, _vp]),
            "exl3_silu_mul": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp]),
            "exl3_linear_decode_noalloc": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_int, _i64, _i64, _vp, _vp,
                                                          _vp, ctypes.c_int, _vp]),
            "exl3_reconstruct_rotated": (ctypes.c_int, [_vp, ctypes.c_int, _i64, _i64, _i64, _i64, _vp, _vp, _vp,
                                                        ctypes.c_int, _vp]),
            "exl3_weight_rotated_workspace_bytes": (ctypes.c_size_t, [_i64, _i64]),
            "exl3_linear_weight_rotated": (ctypes.c_int, [_vp, _i64, _i64, _vp, ctypes.c_int, _i64, _i64, _vp, _vp,
                                                          _vp, ctypes.c_int, _vp, ctypes.c_size_t, _vp]),
            "exl3_bounds_checked": (ctypes.c_int, []),
            "exl3_selftest_bounds": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int), _vp]),
            "exl3_kv8_append": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _i64, _vp]),
            "exl3_kv8_attention_workspace_bytes": (ctypes.c_size_t, [_vp, _vp, _i32]),
            "exl3_kv8_attention": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, ctypes.c_float, ctypes.c_float,
                                                  ctypes.c_int, _vp, _i64, _vp, _vp, ctypes.c_size_t, _vp]),
            "exl3_kv8_weigh": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i32, ctypes.c_float, ctypes.c_float, ctypes.c_int,
                                              _vp, _vp]),
            "exl3_kv8_evict": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _vp, _vp, _vp]),
            "exl3_logits_adjust": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _vp]),
            "exl3_selftest_bounds_serving": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int),
                                                            ctypes.POINTER(ctypes.c_int), _vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _status_text(status: int) -> str:
    try:
        return load().exl3_status_string(int(status)).decode()
    except Exception:  # the library may be the thing that failed to load
        return STATUS_NAMES.get(int(status), "unknown")


def _check(status: int, where: str) -> None:
    if status != 0:
        raise Exl3Error(status, where)


def _ptr(t):
    """Device pointer of a tensor (or an int address, or None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_raw_stream = _raw_device = None  # (device) -> handle of torch's current stream, and () -> device


def _stream(stream):
    if stream is None:
        global _raw_stream, _raw_device
        if _raw_device is None:
            import torch
            # the raw handle of torch's current stream: torch.cuda.current_stream() builds an object
            # for it at every call, which takes longer than a launch
            get, device = getattr(torch._C, "_cuda_getCurrentRawStream", None), getattr(torch._C, "_cuda_getDevice", None)
            if get is None or device is None:
                get, device = (lambda _: torch.cuda.current_stream().cuda_stream), (lambda: None)
            _raw_stream, _raw_device = get, device  # the device last: another thread may be here
        return _raw_stream(_raw_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def exl3_init(device: int = 0) -> None:
    _check(load().exl3_init(int(device)), "exl3_init")


def exl3_status_string(status: int) -> str:
    return load().exl3_status_string(int(status)).decode()


def exl3_supported_bits(bits: int) -> bool:
    return bool(load().exl3_supported_bits(int(bits)))


def exl3_aligned_logits_width(n_decodable: int, n_stored: int) -> int:
    return int(load().exl3_aligned_logits_width(int(n_decodable), int(n_stored)))


def exl3_decode_plan(K: int, n_gemm: int, num_sms: int):
    s, g = ctypes.c_int(), ctypes.c_int()
    rc = load().exl3_decode_plan(int(K), int(n_gemm), int(num_sms), ctypes.byref(s), ctypes.byref(g))
    if rc != 0:
        raise ValueError("exl3_decode_plan: invalid geometry")
    return s.value, g.value


def exl3_prefill_path(M: int, n_gemm: int, num_sms: int) -> int:
    """1: a prefill-shaped call of M rows on an n_gemm-wide layer takes the
    fused prefill kernel; 0: reconstruct + GEMM; -1: invalid input."""
    return int(load().exl3_prefill_path(int(M), int(n_gemm), int(num_sms)))


def exl3_linear_workspace_bytes_for(M_max, K, n_gemm, bits, m_threshold, num_sms) -> int:
    return int(load().exl3_linear_workspace_bytes_for(int(M_max), int(K), int(n_gemm), int(bits),
                                                      int(m_threshold), int(num_sms)))


def exl3_linear_workspace_bytes(M_max, K, n_gemm, bits, m_threshold) -> int:
    return int(load().exl3_linear_workspace_bytes(int(M_max), int(K), int(n_gemm), int(bits), int(m_threshold)))


def exl3_workspace_init(workspace, workspace_bytes: int | None = None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().exl3_workspace_init(_ptr(workspace), int(nbytes), _stream(stream)), "exl3_workspace_init")


def exl3_hadamard128(x, y, pre_scale=None, rows: int | None = None, cols: int | None = None, stream=None) -> None:
    rows = x.shape[0] if rows is None else rows
    cols = x.shape[1] if cols is None else cols
    _check(load().exl3_hadamard128(_ptr(x), _ptr(y), _ptr(pre_scale), int(rows), int(cols), _stream(stream)),
           "exl3_hadamard128")


def exl3_reconstruct(trellis, bits: int, K: int, n_stored: int, n0: int, n_cols: int, w,
                     layout: int = EXL3_LAYOUT_KN, stream=None) -> None:
    _check(load().exl3_reconstruct(_ptr(trellis), int(bits), int(K), int(n_stored), int(n0), int(n_cols),
                                   _ptr(w), int(layout), _stream(stream)), "exl3_reconstruct")


def exl3_reconstruct_rotated(trellis, bits: int, K: int, n_stored: int, n0: int, n_cols: int, su, sv, w,
                             layout: int = EXL3_LAYOUT_KN, stream=None) -> None:
    _check(load().exl3_reconstruct_rotated(_ptr(trellis), int(bits), int(K), int(n_stored), int(n0), int(n_cols),
                                           _ptr(su), _ptr(sv), _ptr(w), int(layout), _stream(stream)),
           "exl3_reconstruct_rotated")


def exl3_weight_rotated_workspace_bytes(K: int, n_gemm: int) -> int:
    return int(load().exl3_weight_rotated_workspace_bytes(int(K), int(n_gemm)))


def exl3_linear_weight_rotated(x, M: int, K: int, trellis, bits: int, n_stored: int, n_gemm: int, su, sv, y,
                               y_dtype: int, workspace, workspace_bytes: int | None = None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().exl3_linear_weight_rotated(_ptr(x), int(M), int(K), _ptr(trellis), int(bits), int(n_stored),
                                             int(n_gemm), _ptr(su), _ptr(sv), _ptr(y), int(y_dtype),
                                             _ptr(workspace), int(nbytes), _stream(stream)),
           "exl3_linear_weight_rotated")


def exl3_linear(x, M: int, K: int, trellis, bits: int, n_stored: int, n_gemm: int, su, sv, y, y_dtype: int,
                m_threshold: int, workspace, workspace_bytes: int | None = None, stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().exl3_linear(_ptr(x), int(M), int(K), _ptr(trellis), int(bits), int(n_stored), int(n_gemm),
                              _ptr(su), _ptr(sv), _ptr(y), int(y_dtype), int(m_threshold), _ptr(workspace),
                              int(nbytes), _stream(stream)), "exl3_linear")


def exl3_logits_masked(x, M: int, K: int, trellis, bits: int, n_stored: int, n_gemm: int, n_decodable: int,
                       su, sv, logits, argmax, m_threshold: int, workspace, workspace_bytes: int | None = None,
                       stream=None) -> None:
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(load().exl3_logits_masked(_ptr(x), int(M), int(K), _ptr(trellis), int(bits), int(n_stored),
                                     int(n_gemm), int(n_decodable), _ptr(su), _ptr(sv), _ptr(logits),
                                     _ptr(argmax), int(m_threshold), _ptr(workspace), int(nbytes),
                                     _stream(stream)), "exl3_logits_masked")


def exl3_get_device_status(stream=None) -> int:
    """Synchronises the stream, reads and clears the device error word."""
    return int(load().exl3_get_device_status(_stream(stream)))


def exl3_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """Launches the bounded-wait self-test kernel (see include/exl3.h)."""
    _check(load().exl3_selftest_wait_timeout(int(limit_us), _stream(stream)), "exl3_selftest_wait_timeout")


def exl3_bounds_checked() -> bool:
    """True when the loaded library is the bounds-checked build."""
    return load().exl3_bounds_checked() == 1


def exl3_selftest_bounds(stream=None) -> tuple[int, int]:
    """Runs the bounds-check reporting self-test (see include/exl3.h); returns
    (units that reported, units probed): (6, 6) in the bounds-checked build,
    (0, 0) in libexl3.so."""
    rep, tot = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().exl3_selftest_bounds(ctypes.byref(rep), ctypes.byref(tot), _stream(stream)), "exl3_selftest_bounds")
    return rep.value, tot.value


def exl3_linear_decode_noalloc(x, M: int, K: int, trellis, bits: int, n_stored: int, n_gemm: int, su, sv, y,
                               y_dtype: int, stream=None) -> None:
    """Decode-shaped linear layer that allocates nothing: its scratch is a
    fixed buffer of EXL3_NOALLOC_SCRATCH_BYTES (24 MiB) inside the library.
    Rows run in groups of 16 through the 16-row decode kernel."""
    _check(load().exl3_linear_decode_noalloc(_ptr(x), int(M), int(K), _ptr(trellis), int(bits), int(n_stored),
                                             int(n_gemm), _ptr(su), _ptr(sv), _ptr(y), int(y_dtype),
                                             _stream(stream)), "exl3_linear_decode_noalloc")


def exl3_silu_mul(gate, up, out, n: int | None = None, stream=None) -> None:
    """out = fp16(silu(gate) * up), the dense-MLP glue between projections."""
    n = gate.numel() if n is None else n
    _check(load().exl3_silu_mul(_ptr(gate), _ptr(up), _ptr(out), int(n), _stream(stream)), "exl3_silu_mul")


# The tensors of the serving operators' calls, checked in as few steps as a call of a few
# microseconds allows: types, sizes and strides, as the kernels will read them.
_F16 = _F32 = _I32 = None


def _need_dtypes():
    global _F16, _F32, _I32
    import torch
    _F32, _I32, _F16 = torch.float32, torch.int32, torch.float16  # the one that is asked for last
    return _F16


def _rows(what, t, dtype, rows, cols):
    """Row stride of t, `rows` rows of at least `cols` elements (any row stride, each row contiguous)."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not dtype or len(shape) < 2 or shape[0] < rows or stride[-1] != 1 or shape[1] < cols and (
            len(shape) == 2 or rows > 0 and (not t[0].is_contiguous() or t[0].numel() < cols)):
        raise ValueError(f"{what}: expected {dtype}, {rows} x {cols} with contiguous rows, got {t.dtype} {tuple(shape)} with strides {stride}")
    return stride[0] if shape[0] > 1 else -(-cols // 8) * 8  # a single row's stride says nothing


def _array(what, t, dtype, n):
    """Pointer of t, contiguous and of at least n elements (an int address as it is; 0 for None)."""
    try:
        if t.dtype is dtype and t.numel() >= n and (n == 1 or t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        if t is None or isinstance(t, int):
            return t or 0
        raise
    if dtype is _I32 and t.element_size() == 4 and not t.is_floating_point() and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()  # other 32-bit integers
    raise ValueError(f"{what}: expected at least {n} contiguous {dtype}, got {t.dtype} {tuple(t.shape)} with strides {t.stride()}")


def exl3_kv8_append(cache: Exl3Kv8Cache, batch: Exl3Kv8Batch, k, v, stream=None) -> None:
    """Quantizes rows of keys and values (fp16, rows x n_kv_heads * head_dim,
    any row stride) into the 8-bit cache."""
    lib = _lib or load()
    rows, cols, f16 = batch.rows, cache.n_kv_heads * cache.head_dim, _F16 or _need_dtypes()
    ldk, ldv = _rows("exl3_kv8_append: k", k, f16, rows, cols), _rows("exl3_kv8_append: v", v, f16, rows, cols)
    status = lib.exl3_kv8_append(cache._ref, batch._ref, k.data_ptr(), ldk, v.data_ptr(), ldv, _stream(stream))
    if status:
        raise Exl3Error(status, "exl3_kv8_append")


def exl3_kv8_attention_workspace_bytes(cache: Exl3Kv8Cache, batch: Exl3Kv8Batch, n_heads: int) -> int:
    return int(load().exl3_kv8_attention_workspace_bytes(cache._ref, batch._ref, int(n_heads)))


def exl3_kv8_attention(cache: Exl3Kv8Cache, batch: Exl3Kv8Batch, q, n_heads: int, scale: float, out, workspace,
                       softcap: float = 0.0, causal: bool = True, lse=None, workspace_bytes: int | None = None,
                       stream=None) -> None:
    """Attention of q (fp16, rows x n_heads * head_dim, any row stride) over the
    8-bit cache into out (fp16, same shape); lse: rows x n_heads fp32 or None."""
    lib = _lib or load()
    rows, cols, f16 = batch.rows, n_heads * cache.head_dim, _F16 or _need_dtypes()
    ldq, ldo = _rows("exl3_kv8_attention: q", q, f16, rows, cols), _rows("exl3_kv8_attention: out", out, f16, rows, cols)
    lse = _array("exl3_kv8_attention: lse", lse, _F32, rows * n_heads)
    nbytes = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    status = lib.exl3_kv8_attention(cache._ref, batch._ref, q.data_ptr(), ldq, n_heads, scale, softcap, causal,
                                    out.data_ptr(), ldo, lse, _ptr(workspace), nbytes, _stream(stream))
    if status:
        raise Exl3Error(status, "exl3_kv8_attention")


def exl3_kv8_weigh(cache: Exl3Kv8Cache, batch: Exl3Kv8Batch, q, n_heads: int, scale: float, lse, softcap: float = 0.0,
                   causal: bool = True, stream=None) -> None:
    """Adds the attention that q's rows give each cached token to cache.weight;
    lse as exl3_kv8_attention returned it."""
    lib = _lib or load()
    rows, f16 = batch.rows, _F16 or _need_dtypes()
    ldq = _rows("exl3_kv8_weigh: q", q, f16, rows, n_heads * cache.head_dim)
    lse = _array("exl3_kv8_weigh: lse", lse, _F32, rows * n_heads)
    status = lib.exl3_kv8_weigh(cache._ref, batch._ref, q.data_ptr(), ldq, n_heads, scale, softcap, causal, lse,
                                _stream(stream))
    if status:
        raise Exl3Error(status, "exl3_kv8_weigh")


def exl3_kv8_evict(cache: Exl3Kv8Cache, batch: Exl3Kv8Batch, dst_pages, budget: int, recent: int, kept, new_len,
                   stream=None) -> None:
    """Moves each sequence's last `recent` and heaviest other tokens, `budget` in
    all, to dst_pages (int32, n_seqs x ceil(budget / 64)); kept (int32, n_seqs x
    n_kv_heads x budget) and new_len (int32, n_seqs) receive what was kept."""
    lib = _lib or load()
    if _F16 is None:
        _need_dtypes()
    n = batch.n_seqs
    dst_pages = _array("exl3_kv8_evict: dst_pages", dst_pages, _I32, n * -(-budget // EXL3_KV8_BLOCK))
    kept = _array("exl3_kv8_evict: kept", kept, _I32, n * cache.n_kv_heads * budget)
    new_len = _array("exl3_kv8_evict: new_len", new_len, _I32, n)
    status = lib.exl3_kv8_evict(cache._ref, batch._ref, dst_pages, budget, recent, kept, new_len, _stream(stream))
    if status:
        raise Exl3Error(status, "exl3_kv8_evict")


def exl3_logits_adjust(logits, n: int, out, argmax, history=None, history_start=None, generated_from=None,
                       repetition=None, presence=None, frequency=None, bias_id=None, bias_value=None, bias_start=None,
                       allowed=None, stream=None) -> None:
    """Penalties, biases and a grammar mask on the first n columns of logits
    (fp32, M x ld) into out (may be logits), and the greedy choice (int32, M).
    Token ids, starts and generated_from are int32, the penalties and
    bias_value fp32, allowed M x ceil(n / 32) words of 32 bits."""
    lib = _lib or load()
    if _F16 is None:
        _need_dtypes()
    i32, f32, M = _I32, _F32, logits.shape[0]
    ldl, ldo = _rows("exl3_logits_adjust: logits", logits, f32, M, n), _rows("exl3_logits_adjust: out", out, f32, M, n)
    n_history, n_bias = 0 if history is None else history.numel(), 0 if bias_id is None else bias_id.numel()
    # an empty tensor has no address: what belongs to an empty list is left out with it
    if n_history == 0 and history is not None:
        history_start = generated_from = None
    if n_bias == 0 and bias_id is not None:
        bias_value = bias_start = None
    rules = _PACK_RULES(
        _array("exl3_logits_adjust: history", history, i32, 0),
        _array("exl3_logits_adjust: history_start", history_start, i32, M + 1),
        _array("exl3_logits_adjust: generated_from", generated_from, i32, M),
        _array("exl3_logits_adjust: repetition", repetition, f32, M),
        _array("exl3_logits_adjust: presence", presence, f32, M),
        _array("exl3_logits_adjust: frequency", frequency, f32, M),
        _array("exl3_logits_adjust: bias_id", bias_id, i32, 0),
        _array("exl3_logits_adjust: bias_value", bias_value, f32, n_bias),
        _array("exl3_logits_adjust: bias_start", bias_start, i32, M + 1),
        _array("exl3_logits_adjust: allowed", allowed, i32, M * -(-n // 32)), n_history, n_bias)
    argmax = _array("exl3_logits_adjust: argmax", argmax, i32, M)
    status = lib.exl3_logits_adjust(logits.data_ptr(), ldl, M, n, rules, out.data_ptr(), ldo, argmax, _stream(stream))
    if status:
        raise Exl3Error(status, "exl3_logits_adjust")


def exl3_selftest_bounds_serving(stream=None) -> tuple[int, int]:
    """exl3_selftest_bounds for the serving operators' translation units."""
    rep, tot = ctypes.c_int(0), ctypes.c_int(0)
    _check(load().exl3_selftest_bounds_serving(ctypes.byref(rep), ctypes.byref(tot), _stream(stream)),
           "exl3_selftest_bounds_serving")
    return rep.value, tot.value
