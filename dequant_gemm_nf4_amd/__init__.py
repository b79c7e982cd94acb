"""Python binding of libbnbx, the MI355X (gfx950) NF4 4-bit weight library.

Argument marshalling only: every function here has the name of a C entry
point declared in ``include/bnbx.h`` and forwards to it through ctypes.  All
computation happens in the library's HIP kernels.  Device buffers may be
passed as integers (device addresses) or as objects with ``data_ptr()``
(torch tensors); ``stream`` is a hipStream_t handle (int), a torch stream, or
None for the caller's current torch stream when torch has a GPU, else the
null stream.

If the shared library is missing, importing works but every call raises
``BnbxLibraryMissing``: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import os

__all__ = [
    "BNBX_OK", "BNBX_E_INVAL", "BNBX_E_ALIGN", "BNBX_E_UNSUPPORTED", "BNBX_E_WORKSPACE",
    "BNBX_E_HIP", "BNBX_E_INTERNAL", "BnbxError", "BnbxLibraryMissing", "Nf4State", "library_path", "lib",
    "bnbx_status_str", "bnbx_nf4_codebook", "bnbx_fp4_codebook", "bnbx_dynamic_map",
    "bnbx_quantize_nf4_workspace_bytes",
    "bnbx_quantize_nf4", "bnbx_quantize_nf4_noalloc", "BNBX_NOALLOC_MAX_WEIGHTS",
    "bnbx_quantize_nf4_grouped_workspace_bytes", "bnbx_quantize_nf4_grouped", "QuantizeItem",
    "BNBX_QUANTIZE_MAX_ITEMS",
    "bnbx_dequantize_nf4", "bnbx_gemv_nf4", "bnbx_gemv_nf4_grouped", "GemvItem",
    "BNBX_GEMV_MAX_ITEMS",
    "bnbx_gemm_nf4_workspace_bytes", "bnbx_gemm_nf4", "bnbx_gemm_nf4_dx", "bnbx_gemm_nf4_lora",
    "bnbx_lora_down", "bnbx_probe_stream_read", "BNBX_PROBE_SINK_WORDS", "EXPORTED_SYMBOLS", "BNBX_QUANT_NF4", "BNBX_QUANT_FP4",
    "BNBX_DTYPE_BF16", "BNBX_DTYPE_F16", "BNBX_DQ_NONE", "BNBX_DQ_LINEAR", "BNBX_DQ_DYNAMIC",
    "rows_library_path", "rows_lib", "ROWS_EXPORTED_SYMBOLS", "BNBX_ROWS_MAX_GROUPS",
    "RowGroupsDesc", "bnbx_group_rows_workspace_bytes", "bnbx_group_rows",
    "bnbx_gemm_nf4_experts", "bnbx_gemm_nf4_experts_dx", "AdaptersDesc",
    "bnbx_gemm_nf4_adapters_workspace_bytes", "bnbx_gemm_nf4_adapters",
    "int8_library_path", "int8_lib", "INT8_EXPORTED_SYMBOLS", "BNBX_DTYPE_F32",
    "BNBX_INT8_MAX_COLS", "Int8RowsDesc", "bnbx_quantize_rows_int8", "bnbx_dequantize_rows_int8",
    "bnbx_gemm_int8_workspace_bytes", "bnbx_gemm_int8", "bnbx_linear_int8_workspace_bytes",
    "bnbx_linear_int8", "bnbx_gemm_int8_dx_workspace_bytes", "bnbx_gemm_int8_dx",
    "bnbx_gemm_int8_dw_workspace_bytes", "bnbx_gemm_int8_dw",
]

BNBX_OK = 0
BNBX_E_INVAL = -1
BNBX_E_ALIGN = -2
BNBX_E_UNSUPPORTED = -3
BNBX_E_WORKSPACE = -4
BNBX_E_HIP = -5
BNBX_E_INTERNAL = -6

BNBX_QUANT_NF4 = 0
BNBX_QUANT_FP4 = 1
BNBX_DTYPE_BF16 = 0
BNBX_DTYPE_F16 = 1
BNBX_DQ_NONE = 0
BNBX_DQ_LINEAR = 1
BNBX_DQ_DYNAMIC = 2

BNBX_NOALLOC_MAX_WEIGHTS = 1 << 28
BNBX_GEMV_MAX_ITEMS = 4
BNBX_QUANTIZE_MAX_ITEMS = 8

EXPORTED_SYMBOLS = (
    "bnbx_status_str", "bnbx_nf4_codebook", "bnbx_fp4_codebook", "bnbx_dynamic_map",
    "bnbx_quantize_nf4_workspace_bytes",
    "bnbx_quantize_nf4", "bnbx_quantize_nf4_noalloc", "bnbx_quantize_nf4_grouped_workspace_bytes",
    "bnbx_quantize_nf4_grouped", "bnbx_dequantize_nf4", "bnbx_gemv_nf4",
    "bnbx_gemv_nf4_grouped",
    "bnbx_gemm_nf4_workspace_bytes", "bnbx_gemm_nf4", "bnbx_gemm_nf4_dx", "bnbx_gemm_nf4_lora",
    "bnbx_lora_down",
    "bnbx_probe_stream_read",          # include/bnbx_probe.h (measurement aid)
)
BNBX_PROBE_SINK_WORDS = 1024

# libbnbx_rows.so (include/bnbx_rows.h)
BNBX_ROWS_MAX_GROUPS = 1024
ROWS_EXPORTED_SYMBOLS = (
    "bnbx_group_rows_workspace_bytes", "bnbx_group_rows", "bnbx_gemm_nf4_experts",
    "bnbx_gemm_nf4_experts_dx", "bnbx_gemm_nf4_adapters_workspace_bytes",
    "bnbx_gemm_nf4_adapters",
)

# libbnbx_int8.so (include/bnbx_int8.h)
BNBX_DTYPE_F32 = 2
BNBX_INT8_MAX_COLS = 131071
INT8_EXPORTED_SYMBOLS = (
    "bnbx_quantize_rows_int8", "bnbx_dequantize_rows_int8", "bnbx_gemm_int8_workspace_bytes",
    "bnbx_gemm_int8", "bnbx_linear_int8_workspace_bytes", "bnbx_linear_int8",
    "bnbx_gemm_int8_dx_workspace_bytes", "bnbx_gemm_int8_dx",
    "bnbx_gemm_int8_dw_workspace_bytes", "bnbx_gemm_int8_dw",
)

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "libbnbx.so")


class BnbxLibraryMissing(RuntimeError):
    pass


class BnbxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {bnbx_status_str(status)} ({status})")


class Nf4State(ctypes.Structure):
    """bnbx_nf4_state: host descriptor holding device pointers."""

    _fields_ = [
        ("n", ctypes.c_int64),
        ("blocksize", ctypes.c_int32),
        ("double_quant", ctypes.c_int32),
        ("quant_type", ctypes.c_int32),
        ("compute_dtype", ctypes.c_int32),
        ("absmax", ctypes.c_void_p),
        ("absmax2", ctypes.c_void_p),
        ("absmax_mean", ctypes.c_void_p),
    ]


class QuantizeItem(ctypes.Structure):
    """bnbx_quantize_item: one tensor of a grouped quantize (device pointers;
    the state pointer is a host address)."""

    _fields_ = [
        ("w", ctypes.c_void_p),
        ("packed", ctypes.c_void_p),
        ("st", ctypes.POINTER(Nf4State)),
    ]


class GemvItem(ctypes.Structure):
    """bnbx_gemv_item: one weight of a grouped GEMV (device pointers; the
    state pointer is a host address)."""

    _fields_ = [
        ("packed", ctypes.c_void_p),
        ("st", ctypes.POINTER(Nf4State)),
        ("N", ctypes.c_int32),
        ("y", ctypes.c_void_p),
        ("ldy", ctypes.c_int64),
    ]


class RowGroupsDesc(ctypes.Structure):
    """bnbx_row_groups: a plan of grouped rows (device pointers)."""

    _fields_ = [
        ("offsets", ctypes.c_void_p),
        ("order", ctypes.c_void_p),
        ("groups", ctypes.c_int32),
        ("rows", ctypes.c_int32),
    ]


class AdaptersDesc(ctypes.Structure):
    """bnbx_adapters: the low-rank adapters of a call (device pointers)."""

    _fields_ = [
        ("lora_a", ctypes.c_void_p),
        ("lora_b", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("lda", ctypes.c_int64),
        ("stride_a", ctypes.c_int64),
        ("ldb", ctypes.c_int64),
        ("stride_b", ctypes.c_int64),
        ("r", ctypes.c_int32),
    ]


class Int8RowsDesc(ctypes.Structure):
    """bnbx_int8_rows: rows of 8-bit codes (device pointers)."""

    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("ld", ctypes.c_int64),
        ("rows", ctypes.c_int32),
        ("cols", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libbnbx.so (built in-tree by dequant_gemm_nf4_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise BnbxLibraryMissing(
            f"{path} is not built; run `python -m dequant_gemm_nf4_amd.build` (no fallback exists)")
    # Loaded before torch had initialized HIP, the library's launches on
    # torch's memory failed (most likely two HIP runtime instances: torch
    # bundles its own).  Importing torch first avoided it in every run.
    try:
        import torch  # noqa: F401
    except ImportError:  # pragma: no cover
        pass
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sp = ctypes.POINTER(Nf4State)
    L.bnbx_status_str.argtypes = [i32]
    L.bnbx_status_str.restype = ctypes.c_char_p
    L.bnbx_nf4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.bnbx_nf4_codebook.restype = i32
    L.bnbx_fp4_codebook.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.bnbx_fp4_codebook.restype = i32
    L.bnbx_dynamic_map.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.bnbx_dynamic_map.restype = i32
    L.bnbx_quantize_nf4_workspace_bytes.argtypes = [i64, i32, i32]
    L.bnbx_quantize_nf4_workspace_bytes.restype = sz
    L.bnbx_quantize_nf4.argtypes = [vp, vp, sp, vp, sz, vp]
    L.bnbx_quantize_nf4.restype = i32
    L.bnbx_quantize_nf4_noalloc.argtypes = [vp, vp, sp, vp]
    L.bnbx_quantize_nf4_noalloc.restype = i32
    L.bnbx_quantize_nf4_grouped_workspace_bytes.argtypes = [ctypes.POINTER(i64), i32, i32, i32]
    L.bnbx_quantize_nf4_grouped_workspace_bytes.restype = sz
    L.bnbx_quantize_nf4_grouped.argtypes = [ctypes.POINTER(QuantizeItem), i32, vp, sz, vp]
    L.bnbx_quantize_nf4_grouped.restype = i32
    L.bnbx_dequantize_nf4.argtypes = [vp, sp, vp, vp]
    L.bnbx_dequantize_nf4.restype = i32
    L.bnbx_gemv_nf4.argtypes = [vp, i64, vp, sp, i32, i32, i32, vp, i64, vp]
    L.bnbx_gemv_nf4.restype = i32
    L.bnbx_gemv_nf4_grouped.argtypes = [vp, i64, ctypes.POINTER(GemvItem), i32, i32, i32, vp]
    L.bnbx_gemv_nf4_grouped.restype = i32
    L.bnbx_gemm_nf4_workspace_bytes.argtypes = [i32, i32, i32]
    L.bnbx_gemm_nf4_workspace_bytes.restype = sz
    L.bnbx_gemm_nf4.argtypes = [vp, i64, vp, sp, i32, i32, i32, vp, i64, vp, sz, vp]
    L.bnbx_gemm_nf4.restype = i32
    L.bnbx_gemm_nf4_lora.argtypes = [vp, i64, vp, sp, i32, i32, i32, vp, i64, vp, i64, i32, vp,
                                     i64, vp]
    L.bnbx_gemm_nf4_lora.restype = i32
    L.bnbx_gemm_nf4_dx.argtypes = [vp, i64, vp, sp, i32, i32, i32, vp, i64, vp]
    L.bnbx_gemm_nf4_dx.restype = i32
    L.bnbx_lora_down.argtypes = [vp, i64, vp, i64, i32, i32, i32, ctypes.c_float, i32, vp, i64, vp]
    L.bnbx_lora_down.restype = i32
    L.bnbx_probe_stream_read.argtypes = [vp, sz, vp, sz, vp, vp]
    L.bnbx_probe_stream_read.restype = i32
    _lib = L
    return L


_rows_lib = None


def rows_library_path() -> str:
    return os.path.join(_HERE, "libbnbx_rows.so")


def rows_lib() -> ctypes.CDLL:
    """Load libbnbx_rows.so, the row-grouped operators (built in-tree by
    dequant_gemm_nf4_amd.build)."""
    global _rows_lib
    if _rows_lib is not None:
        return _rows_lib
    path = rows_library_path()
    if not os.path.exists(path):
        raise BnbxLibraryMissing(
            f"{path} is not built; run `python -m dequant_gemm_nf4_amd.build` (no fallback exists)")
    try:
        import torch  # noqa: F401  (before the library, as in lib())
    except ImportError:  # pragma: no cover
        pass
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    sp, gp = ctypes.POINTER(Nf4State), ctypes.POINTER(RowGroupsDesc)
    L.bnbx_group_rows_workspace_bytes.argtypes = [i32, i32]
    L.bnbx_group_rows_workspace_bytes.restype = sz
    L.bnbx_group_rows.argtypes = [vp, i32, i32, vp, vp, vp, sz, vp]
    L.bnbx_group_rows.restype = i32
    L.bnbx_gemm_nf4_experts.argtypes = [vp, i64, i32, vp, sp, gp, i32, i32, i32, i32, vp, i64,
                                        i32, vp]
    L.bnbx_gemm_nf4_experts.restype = i32
    L.bnbx_gemm_nf4_experts_dx.argtypes = L.bnbx_gemm_nf4_experts.argtypes
    L.bnbx_gemm_nf4_experts_dx.restype = i32
    L.bnbx_gemm_nf4_adapters_workspace_bytes.argtypes = [i32, i32]
    L.bnbx_gemm_nf4_adapters_workspace_bytes.restype = sz
    L.bnbx_gemm_nf4_adapters.argtypes = [vp, i64, vp, sp, gp, i32, i32,
                                         ctypes.POINTER(AdaptersDesc), vp, i64, vp, sz, vp]
    L.bnbx_gemm_nf4_adapters.restype = i32
    _rows_lib = L
    return L


_int8_lib = None


def int8_library_path() -> str:
    return os.path.join(_HERE, "libbnbx_int8.so")


def int8_lib() -> ctypes.CDLL:
    """Load libbnbx_int8.so, the 8-bit operators (built in-tree by
    dequant_gemm_nf4_amd.build)."""
    global _int8_lib
    if _int8_lib is not None:
        return _int8_lib
    path = int8_library_path()
    if not os.path.exists(path):
        raise BnbxLibraryMissing(
            f"{path} is not built; run `python -m dequant_gemm_nf4_amd.build` (no fallback exists)")
    try:
        import torch  # noqa: F401  (before the library, as in lib())
    except ImportError:  # pragma: no cover
        pass
    L = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    qp = ctypes.POINTER(Int8RowsDesc)
    L.bnbx_quantize_rows_int8.argtypes = [vp, i64, qp, vp]
    L.bnbx_dequantize_rows_int8.argtypes = [qp, vp, i64, vp]
    L.bnbx_gemm_int8_workspace_bytes.argtypes = [i32, i32, i32]
    L.bnbx_gemm_int8.argtypes = [qp, qp, vp, i64, vp, sz, vp]
    L.bnbx_linear_int8_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.bnbx_linear_int8.argtypes = [vp, i64, i32, qp, qp, vp, i64, vp, sz, vp]
    L.bnbx_gemm_int8_dx_workspace_bytes.argtypes = [i32, i32, i32]
    L.bnbx_gemm_int8_dx.argtypes = [vp, i64, i32, qp, vp, i64, vp, sz, vp]
    L.bnbx_gemm_int8_dw_workspace_bytes.argtypes = [i32, i32, i32]
    L.bnbx_gemm_int8_dw.argtypes = [vp, i64, i32, qp, vp, i64, i32, vp, sz, vp]
    for name in INT8_EXPORTED_SYMBOLS:
        getattr(L, name).restype = sz if name.endswith("_bytes") else i32
    _int8_lib = L
    return L


def _ptr(a) -> int | None:
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return int(a.data_ptr())


_raw_stream = None


def current_stream(device: int | None = None) -> int | None:
    """Handle of the caller's current torch stream on a device (the current
    one by default); None (the null stream) without torch or a GPU.  The raw
    lookup takes a tenth of a microsecond; torch.cuda.current_stream(), which
    builds a stream object, three."""
    global _raw_stream
    if _raw_stream is None:
        try:
            import torch
        except ImportError:  # pragma: no cover
            return None
        if not torch.cuda.is_available():
            return None
        torch.cuda.init()
        _raw_stream = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
    return _raw_stream[0](_raw_stream[1]() if device is None else device)


def _stream(stream) -> int | None:
    if stream is None:
        return current_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != BNBX_OK:
        raise BnbxError(status, where)


def bnbx_status_str(status: int) -> str:
    return lib().bnbx_status_str(int(status)).decode()


def bnbx_nf4_codebook() -> list[float]:
    buf = (ctypes.c_float * 16)()
    _check(lib().bnbx_nf4_codebook(buf), "bnbx_nf4_codebook")
    return list(buf)


def bnbx_fp4_codebook() -> list[float]:
    buf = (ctypes.c_float * 16)()
    _check(lib().bnbx_fp4_codebook(buf), "bnbx_fp4_codebook")
    return list(buf)


def bnbx_dynamic_map() -> list[float]:
    buf = (ctypes.c_float * 256)()
    _check(lib().bnbx_dynamic_map(buf), "bnbx_dynamic_map")
    return list(buf)


def bnbx_quantize_nf4_workspace_bytes(n: int, blocksize: int = 64, double_quant: int = 1) -> int:
    return int(lib().bnbx_quantize_nf4_workspace_bytes(int(n), int(blocksize), int(double_quant)))


def bnbx_quantize_nf4(w, packed, state: Nf4State, workspace=None, workspace_bytes: int = 0,
                      stream=None) -> None:
    _check(lib().bnbx_quantize_nf4(_ptr(w), _ptr(packed), ctypes.byref(state), _ptr(workspace),
                                   int(workspace_bytes), _stream(stream)), "bnbx_quantize_nf4")


def bnbx_quantize_nf4_noalloc(w, packed, state: Nf4State, stream=None) -> None:
    _check(lib().bnbx_quantize_nf4_noalloc(_ptr(w), _ptr(packed), ctypes.byref(state),
                                           _stream(stream)), "bnbx_quantize_nf4_noalloc")


def bnbx_quantize_nf4_grouped_workspace_bytes(ns, blocksize: int = 64,
                                              double_quant: int = 1) -> int:
    arr = (ctypes.c_int64 * max(len(ns), 1))(*[int(n) for n in ns])
    return int(lib().bnbx_quantize_nf4_grouped_workspace_bytes(arr, len(ns), int(blocksize),
                                                               int(double_quant)))


def bnbx_quantize_nf4_grouped(items, workspace=None, workspace_bytes: int = 0,
                              stream=None) -> None:
    """items: sequence of (w, packed, state)."""
    n = len(items)
    arr = (QuantizeItem * max(n, 1))()
    states = [st for _, _, st in items]    # kept alive for the call
    for i, (w, packed, st) in enumerate(items):
        arr[i] = QuantizeItem(_ptr(w), _ptr(packed), ctypes.pointer(st))
    _check(lib().bnbx_quantize_nf4_grouped(arr, n, _ptr(workspace), int(workspace_bytes),
                                           _stream(stream)), "bnbx_quantize_nf4_grouped")
    del states


def bnbx_dequantize_nf4(packed, state: Nf4State, out, stream=None) -> None:
    _check(lib().bnbx_dequantize_nf4(_ptr(packed), ctypes.byref(state), _ptr(out),
                                     _stream(stream)), "bnbx_dequantize_nf4")


def bnbx_gemv_nf4(x, ldx: int, packed, state: Nf4State, M: int, N: int, K: int, y, ldy: int,
                  stream=None) -> None:
    _check(lib().bnbx_gemv_nf4(_ptr(x), int(ldx), _ptr(packed), ctypes.byref(state), int(M),
                               int(N), int(K), _ptr(y), int(ldy), _stream(stream)),
           "bnbx_gemv_nf4")


def bnbx_gemv_nf4_grouped(x, ldx: int, items, M: int, K: int, stream=None) -> None:
    """items: sequence of (packed, state, N, y, ldy)."""
    n = len(items)
    arr = (GemvItem * max(n, 1))()
    states = [st for _, st, _, _, _ in items]    # kept alive for the call
    for i, (packed, st, N, y, ldy) in enumerate(items):
        arr[i] = GemvItem(_ptr(packed), ctypes.pointer(st), int(N), _ptr(y), int(ldy))
    _check(lib().bnbx_gemv_nf4_grouped(_ptr(x), int(ldx), arr, n, int(M), int(K),
                                       _stream(stream)), "bnbx_gemv_nf4_grouped")
    del states


def bnbx_gemm_nf4_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().bnbx_gemm_nf4_workspace_bytes(int(M), int(N), int(K)))


def bnbx_gemm_nf4(x, ldx: int, packed, state: Nf4State, M: int, N: int, K: int, y, ldy: int,
                  workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(lib().bnbx_gemm_nf4(_ptr(x), int(ldx), _ptr(packed), ctypes.byref(state), int(M),
                               int(N), int(K), _ptr(y), int(ldy), _ptr(workspace),
                               int(workspace_bytes), _stream(stream)), "bnbx_gemm_nf4")


def bnbx_gemm_nf4_lora(x, ldx: int, packed, state: Nf4State, M: int, N: int, K: int, xa,
                       ldxa: int, lora_b, ldb: int, r: int, y, ldy: int, stream=None) -> None:
    _check(lib().bnbx_gemm_nf4_lora(_ptr(x), int(ldx), _ptr(packed), ctypes.byref(state), int(M),
                                    int(N), int(K), _ptr(xa), int(ldxa), _ptr(lora_b), int(ldb),
                                    int(r), _ptr(y), int(ldy), _stream(stream)),
           "bnbx_gemm_nf4_lora")


def bnbx_gemm_nf4_dx(dy, lddy: int, packed, state: Nf4State, M: int, N: int, K: int, dx,
                     lddx: int, stream=None) -> None:
    _check(lib().bnbx_gemm_nf4_dx(_ptr(dy), int(lddy), _ptr(packed), ctypes.byref(state), int(M),
                                  int(N), int(K), _ptr(dx), int(lddx), _stream(stream)),
           "bnbx_gemm_nf4_dx")


def bnbx_lora_down(x, ldx: int, lora_a, lda: int, M: int, K: int, r: int, scale: float,
                   compute_dtype: int, xa, ldxa: int, stream=None) -> None:
    _check(lib().bnbx_lora_down(_ptr(x), int(ldx), _ptr(lora_a), int(lda), int(M), int(K), int(r),
                                float(scale), int(compute_dtype), _ptr(xa), int(ldxa),
                                _stream(stream)), "bnbx_lora_down")


def _nbytes(t) -> int | None:
    return None if t is None or isinstance(t, int) else int(t.numel() * t.element_size())


def bnbx_probe_stream_read(a, a_bytes: int, b, b_bytes: int, sink, stream=None) -> None:
    # The library cannot see buffer sizes: for tensors, a byte count past the
    # end is rejected here rather than read.
    for t, n in ((a, a_bytes), (b, b_bytes), (sink, 4 * BNBX_PROBE_SINK_WORDS)):
        size = _nbytes(t)
        if size is not None and n > size:
            raise BnbxError(BNBX_E_INVAL, "bnbx_probe_stream_read: byte count past the buffer")
    _check(lib().bnbx_probe_stream_read(_ptr(a), int(a_bytes), _ptr(b), int(b_bytes), _ptr(sink),
                                        _stream(stream)), "bnbx_probe_stream_read")


def bnbx_group_rows_workspace_bytes(rows: int, groups: int) -> int:
    return rows_lib().bnbx_group_rows_workspace_bytes(rows, groups)


def bnbx_group_rows(ids, rows: int, groups: int, offsets, order, workspace=None,
                    workspace_bytes: int = 0, stream=None) -> None:
    _check(rows_lib().bnbx_group_rows(_ptr(ids), rows, groups, _ptr(offsets), _ptr(order),
                                      _ptr(workspace), workspace_bytes, _stream(stream)),
           "bnbx_group_rows")


def bnbx_gemm_nf4_experts(x, ldx: int, x_rows: int, packed, state: Nf4State, plan: RowGroupsDesc,
                          N: int, K: int, gather: int, scatter: int, y, ldy: int, y_rows: int,
                          stream=None) -> None:
    _check(rows_lib().bnbx_gemm_nf4_experts(_ptr(x), ldx, x_rows, _ptr(packed), state, plan, N, K,
                                            gather, scatter, _ptr(y), ldy, y_rows,
                                            _stream(stream)), "bnbx_gemm_nf4_experts")


def bnbx_gemm_nf4_experts_dx(dy, lddy: int, dy_rows: int, packed, state: Nf4State,
                             plan: RowGroupsDesc, N: int, K: int, gather: int, scatter: int, dx,
                             lddx: int, dx_rows: int, stream=None) -> None:
    _check(rows_lib().bnbx_gemm_nf4_experts_dx(_ptr(dy), lddy, dy_rows, _ptr(packed), state, plan,
                                               N, K, gather, scatter, _ptr(dx), lddx, dx_rows,
                                               _stream(stream)), "bnbx_gemm_nf4_experts_dx")


def bnbx_gemm_nf4_adapters_workspace_bytes(rows: int, r: int) -> int:
    return rows_lib().bnbx_gemm_nf4_adapters_workspace_bytes(rows, r)


def bnbx_gemm_nf4_adapters(x, ldx: int, packed, state: Nf4State, plan: RowGroupsDesc, N: int,
                           K: int, adapters: AdaptersDesc, y, ldy: int, workspace=None,
                           workspace_bytes: int = 0, stream=None) -> None:
    _check(rows_lib().bnbx_gemm_nf4_adapters(_ptr(x), ldx, _ptr(packed), state, plan, N, K,
                                             adapters, _ptr(y), ldy, _ptr(workspace),
                                             workspace_bytes, _stream(stream)),
           "bnbx_gemm_nf4_adapters")


def bnbx_quantize_rows_int8(x, ldx: int, q: Int8RowsDesc, stream=None) -> None:
    _check(int8_lib().bnbx_quantize_rows_int8(_ptr(x), ldx, q, _stream(stream)),
           "bnbx_quantize_rows_int8")


def bnbx_dequantize_rows_int8(q: Int8RowsDesc, out, ldo: int, stream=None) -> None:
    _check(int8_lib().bnbx_dequantize_rows_int8(q, _ptr(out), ldo, _stream(stream)),
           "bnbx_dequantize_rows_int8")


def bnbx_gemm_int8_workspace_bytes(M: int, N: int, K: int) -> int:
    return int8_lib().bnbx_gemm_int8_workspace_bytes(M, N, K)


def bnbx_gemm_int8(x: Int8RowsDesc, w: Int8RowsDesc, y, ldy: int, workspace=None,
                   workspace_bytes: int = 0, stream=None) -> None:
    _check(int8_lib().bnbx_gemm_int8(x, w, _ptr(y), ldy, _ptr(workspace), workspace_bytes,
                                     _stream(stream)), "bnbx_gemm_int8")


def bnbx_linear_int8_workspace_bytes(M: int, N: int, K: int, saved: int = 0) -> int:
    return int8_lib().bnbx_linear_int8_workspace_bytes(M, N, K, saved)


def bnbx_linear_int8(x, ldx: int, M: int, w: Int8RowsDesc, saved: Int8RowsDesc | None, y,
                     ldy: int, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(int8_lib().bnbx_linear_int8(_ptr(x), ldx, M, w, saved, _ptr(y), ldy, _ptr(workspace),
                                       workspace_bytes, _stream(stream)), "bnbx_linear_int8")


def bnbx_gemm_int8_dx_workspace_bytes(M: int, N: int, K: int) -> int:
    return int8_lib().bnbx_gemm_int8_dx_workspace_bytes(M, N, K)


def bnbx_gemm_int8_dx(dy, lddy: int, M: int, w: Int8RowsDesc, dx, lddx: int, workspace=None,
                      workspace_bytes: int = 0, stream=None) -> None:
    _check(int8_lib().bnbx_gemm_int8_dx(_ptr(dy), lddy, M, w, _ptr(dx), lddx, _ptr(workspace),
                                        workspace_bytes, _stream(stream)), "bnbx_gemm_int8_dx")


def bnbx_gemm_int8_dw_workspace_bytes(M: int, N: int, K: int) -> int:
    return int8_lib().bnbx_gemm_int8_dw_workspace_bytes(M, N, K)


def bnbx_gemm_int8_dw(dy, lddy: int, N: int, x: Int8RowsDesc, dw, lddw: int, out_dtype: int,
                      workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(int8_lib().bnbx_gemm_int8_dw(_ptr(dy), lddy, N, x, _ptr(dw), lddw, out_dtype,
                                        _ptr(workspace), workspace_bytes, _stream(stream)),
           "bnbx_gemm_int8_dw")
