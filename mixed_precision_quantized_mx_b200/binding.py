"""Thin ctypes binding of the C ABI in include/mx.h.

Argument marshalling only: every function forwards torch tensors' device
pointers, sizes and the current CUDA stream to the function of the same name in
libmx.so.  There is no host-side computation and no fallback: if the library is
missing, or a call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmx.so")

MX_OK = 0
STATUS_NAMES = {
    0: "MX_OK", 1: "MX_ERR_INVALID_ARG", 2: "MX_ERR_UNSUPPORTED", 3: "MX_ERR_ALIGNMENT",
    4: "MX_ERR_CUDA", 5: "MX_ERR_TIMEOUT", 6: "MX_ERR_BAD_BLOB", 7: "MX_ERR_WORKSPACE",
}
MX_F32, MX_F16, MX_BF16 = 0, 1, 2
FP4_E4M3_16, FP4_E8M0_32 = 0, 1          # mx_fp4_format
TILE_ROWS, KBLOCK, HEADER_BYTES = 128, 128, 256
PATH_AUTO, PATH_SPLITK, PATH_TENSOR, PATH_ROWS, PATH_PAIR, PATH_PAIR256, PATH_TC_DECODE = 0, 1, 2, 3, 4, 5, 6

EXPORTED = ("mx_version", "mx_last_error", "mx_layout_init", "mx_layout_from_header",
            "mx_pack_weights", "mx_quant_act", "mx_gemm_workspace_size", "mx_gemm_select_path",
            "mx_gemm", "mx_linear_workspace_size", "mx_linear", "mx_linear_noalloc",
            "mx_quant_act_grouped", "mx_copy_mapped", "mx_saliency", "mx_select_top_workspace_size",
            "mx_select_top", "mx_bw_layout_init", "mx_bw_pack", "mx_bw_gemm",
            "mx_fp4_layout_init", "mx_fp4_layout_from_header", "mx_fp4_gscale", "mx_fp4_quant",
            "mx_fp4_quant_sorted", "mx_fp4_dequant", "mx_fp4_gemm", "mx_fp4_gemm_sorted",
            "mx_fp4_linear_workspace_size", "mx_fp4_linear", "mx_fp4_linear_sorted_workspace_size",
            "mx_fp4_linear_sorted", "mx_fp4_experts_workspace_size", "mx_fp4_experts", "mx_experts_layout_init", "mx_experts_sort", "mx_experts_gather",
            "mx_experts_gather_bwd", "mx_experts_combine", "mx_experts_combine_bwd")


class MXError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn}: {STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class Layout(ctypes.Structure):
    """mirror of mx_layout"""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("N", "K", "group", "n8", "n4", "G", "t8", "t4", "kblocks", "reserved0")] + \
               [(n, ctypes.c_uint64) for n in
                ("off_rowmap", "off_scales8", "off_codes8", "off_scales4", "off_zeros4",
                 "off_codes4", "total_bytes")]


class BwLayout(ctypes.Structure):
    """mirror of mx_bw_layout (block-wise bit widths)"""
    _fields_ = [(n, ctypes.c_int32) for n in ("N", "K", "NB", "KB")] + \
               [("table", ctypes.c_uint8 * 4), ("reserved0", ctypes.c_int32)] + \
               [(n, ctypes.c_uint64) for n in
                ("off_meta", "off_offsets", "off_scales", "off_zeros", "off_codes", "code_bytes", "total_bytes")]


class GemmOpts(ctypes.Structure):
    """mirror of mx_gemm_opts"""
    _fields_ = [("path", ctypes.c_int32), ("split", ctypes.c_int32),
                ("debug_partials", ctypes.c_void_p), ("status", ctypes.c_void_p),
                ("wait_timeout_us", ctypes.c_int32), ("test_stall", ctypes.c_int32),
                ("act_group", ctypes.c_int32)]


class Fp4Layout(ctypes.Structure):
    """mirror of mx_fp4_layout (microscaled 4-bit matrices)"""
    _fields_ = [(n, ctypes.c_int32) for n in
                ("rows", "K", "format", "groups", "block", "tiles", "kblocks", "tile_bytes")] + \
               [(n, ctypes.c_uint64) for n in ("off_gscale", "off_data", "total_bytes")]


class Fp4Opts(ctypes.Structure):
    """mirror of mx_fp4_opts"""
    _fields_ = [("path", ctypes.c_int32), ("split", ctypes.c_int32), ("status", ctypes.c_void_p),
                ("wait_timeout_us", ctypes.c_int32), ("test_stall", ctypes.c_int32)]


class ExpertsLayout(ctypes.Structure):
    """mirror of mx_experts_layout"""
    _fields_ = [(n, ctypes.c_int32) for n in ("T", "k", "E", "n", "max_rows", "reserved0")] + \
               [(n, ctypes.c_uint64) for n in
                ("off_order", "off_pos", "off_dest", "off_offsets", "off_tiles", "total_bytes")]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libmx.so (built in-tree); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m mixed_precision_quantized_mx_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, I64, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
    L.mx_version.restype = I
    L.mx_last_error.restype = ctypes.c_char_p
    L.mx_layout_init.argtypes = [I, I, I, I, ctypes.POINTER(Layout)]
    L.mx_layout_from_header.argtypes = [P, Z, ctypes.POINTER(Layout)]
    L.mx_pack_weights.argtypes = [ctypes.POINTER(Layout), P, I, I64, P, P, P, P]
    L.mx_quant_act.argtypes = [P, I, I, I, I64, P, P, P]
    L.mx_quant_act_grouped.argtypes = [P, I, I, I, I64, I, P, P, P]
    L.mx_gemm_workspace_size.argtypes = [ctypes.POINTER(Layout), I, ctypes.POINTER(GemmOpts),
                                         ctypes.POINTER(Z)]
    L.mx_gemm_select_path.argtypes = [ctypes.POINTER(Layout), I, ctypes.POINTER(GemmOpts)]
    L.mx_gemm_select_path.restype = I
    L.mx_gemm.argtypes = [ctypes.POINTER(Layout), P, P, P, I, P, I64, P, Z,
                          ctypes.POINTER(GemmOpts), P]
    L.mx_linear_workspace_size.argtypes = [ctypes.POINTER(Layout), I, I, ctypes.POINTER(GemmOpts),
                                           ctypes.POINTER(Z)]
    L.mx_linear.argtypes = [ctypes.POINTER(Layout), P, P, I, I, I64, P, I64, P, Z,
                            ctypes.POINTER(GemmOpts), P]
    L.mx_linear_noalloc.argtypes = [ctypes.POINTER(Layout), P, P, I, I, I64, P, I64,
                                    ctypes.POINTER(GemmOpts), P]
    L.mx_copy_mapped.argtypes = [P, P, Z, P]
    L.mx_saliency.argtypes = [P, I, I64, P, I, I64, I, I, I, P, P]
    L.mx_select_top_workspace_size.argtypes = [I64, ctypes.POINTER(Z)]
    L.mx_select_top.argtypes = [P, I64, I64, P, P, Z, P]
    L.mx_bw_layout_init.argtypes = [I, I, P, P, ctypes.POINTER(BwLayout)]
    L.mx_bw_pack.argtypes = [ctypes.POINTER(BwLayout), P, P, I, I64, P, P]
    L.mx_bw_gemm.argtypes = [ctypes.POINTER(BwLayout), P, P, P, I, P, I64, P, P]
    F, X, FO = ctypes.POINTER(Fp4Layout), ctypes.POINTER(ExpertsLayout), ctypes.POINTER(Fp4Opts)
    L.mx_fp4_layout_init.argtypes = [I, I, I, I, F]
    L.mx_fp4_layout_from_header.argtypes = [P, Z, F]
    L.mx_fp4_gscale.argtypes = [F, P, I, I64, I64, P, P]
    L.mx_fp4_quant.argtypes = [F, P, I, I64, I64, P, P, P]
    L.mx_fp4_quant_sorted.argtypes = [F, X, P, I, P, I, I64, P, P, P]
    L.mx_fp4_dequant.argtypes = [F, P, P, I, I64, I64, P]
    L.mx_fp4_gemm.argtypes = [F, P, F, P, P, I, I64, FO, P]
    L.mx_fp4_gemm_sorted.argtypes = [F, P, F, P, X, P, P, I, I64, FO, P]
    L.mx_fp4_linear_workspace_size.argtypes = [F, I, FO, ctypes.POINTER(Z)]
    L.mx_fp4_linear.argtypes = [F, P, P, I, I, I64, P, P, I, I64, P, Z, FO, P]
    L.mx_fp4_linear_sorted_workspace_size.argtypes = [F, X, FO, ctypes.POINTER(Z)]
    L.mx_fp4_linear_sorted.argtypes = [F, P, X, P, I, P, I, I64, P, P, I, I64, P, Z, FO, P]
    L.mx_fp4_experts_workspace_size.argtypes = [F, X, FO, ctypes.POINTER(Z)]
    L.mx_fp4_experts.argtypes = [F, P, X, P, P, I, I64, P, P, P, I, I64, P, Z, FO, P]
    L.mx_experts_layout_init.argtypes = [I, I, I, X]
    L.mx_experts_sort.argtypes = [X, P, P, P]
    L.mx_experts_gather.argtypes = [X, P, P, I, I, I64, P, I64, P]
    L.mx_experts_gather_bwd.argtypes = [X, P, P, I, I, I64, P, I64, P]
    L.mx_experts_combine.argtypes = [X, P, P, I, I, I64, P, P, I, I64, P]
    L.mx_experts_combine_bwd.argtypes = [X, P, P, P, I, I, I64, I64, P, P, I64, P, P]
    for n in EXPORTED:
        if n.startswith(("mx_fp4_", "mx_experts_")):
            getattr(L, n).restype = I
    for n in ("mx_layout_init", "mx_layout_from_header", "mx_pack_weights", "mx_quant_act",
              "mx_quant_act_grouped", "mx_gemm_workspace_size", "mx_gemm", "mx_linear_workspace_size", "mx_linear",
              "mx_linear_noalloc", "mx_copy_mapped", "mx_saliency", "mx_select_top_workspace_size",
              "mx_select_top", "mx_bw_layout_init", "mx_bw_pack", "mx_bw_gemm"):
        getattr(L, n).restype = I
    _lib = L
    return L


def _check(st: int, fn: str):
    if st != MX_OK:
        raise MXError(st, fn, lib().mx_last_error().decode())


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


# the current device's current stream, without building a Stream object; names of torch's own, which
# another version may lack
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int | None:
    if stream is None:
        if _current_device is None or _current_stream is None:
            return torch.cuda.current_stream().cuda_stream
        return _current_stream(_current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(like: torch.Tensor, shape, stream, dtype=None, zeros: bool = False) -> torch.Tensor:
    """A tensor beside `like` for a call on `stream`: allocated (and zeroed) there, since memory of the
    current stream may still be in use by work in front of the call."""
    make = like.new_zeros if zeros else like.new_empty
    if stream is None:
        return make(shape, dtype=dtype)
    with torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream), device=like.device)):
        return make(shape, dtype=dtype)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float16:
        return MX_F16
    if t.dtype == torch.float32:
        return MX_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _opts(path=0, split=0, debug_partials=None, status=None, wait_timeout_us=0,
          test_stall=0, act_group=0) -> GemmOpts:
    return GemmOpts(path, split, _ptr(debug_partials), _ptr(status), wait_timeout_us, test_stall, act_group)


# ------------------------------------------------------------------ entry points
def mx_version() -> int:
    return lib().mx_version()


def mx_layout_init(N: int, K: int, group: int, n8: int) -> Layout:
    L = Layout()
    _check(lib().mx_layout_init(N, K, group, n8, ctypes.byref(L)), "mx_layout_init")
    return L


def mx_layout_from_header(header) -> Layout:
    """header: bytes, or a host uint8 tensor holding the blob's first 256 bytes."""
    if isinstance(header, torch.Tensor):
        header = bytes(header[:HEADER_BYTES].cpu().numpy().tobytes())
    buf = ctypes.create_string_buffer(bytes(header), len(header))
    L = Layout()
    _check(lib().mx_layout_from_header(buf, len(header), ctypes.byref(L)), "mx_layout_from_header")
    return L


def mx_pack_weights(L: Layout, W: torch.Tensor, is8: torch.Tensor, blob: torch.Tensor,
                    status: torch.Tensor | None = None, stream=None) -> None:
    assert W.dim() == 2 and W.stride(1) == 1
    _check(lib().mx_pack_weights(ctypes.byref(L), _ptr(W), _dtype_code(W), W.stride(0), _ptr(is8),
                                 _ptr(blob), _ptr(status), _stream(stream)), "mx_pack_weights")


def mx_quant_act(X: torch.Tensor, Aq: torch.Tensor, s_a: torch.Tensor, stream=None) -> None:
    assert X.dim() == 2 and X.stride(1) == 1
    M, K = X.shape
    _check(lib().mx_quant_act(_ptr(X), _dtype_code(X), M, K, X.stride(0), _ptr(Aq), _ptr(s_a),
                              _stream(stream)), "mx_quant_act")


def mx_quant_act_grouped(X: torch.Tensor, Aq: torch.Tensor, s_a: torch.Tensor, act_group: int,
                         stream=None) -> None:
    """s_a: fp16 [M] (act_group 0) or [M, K / act_group]."""
    assert X.dim() == 2 and X.stride(1) == 1
    M, K = X.shape
    _check(lib().mx_quant_act_grouped(_ptr(X), _dtype_code(X), M, K, X.stride(0), act_group, _ptr(Aq),
                                      _ptr(s_a), _stream(stream)), "mx_quant_act_grouped")


def mx_gemm_workspace_size(L: Layout, M: int, path: int = 0, split: int = 0) -> int:
    n = ctypes.c_size_t(0)
    o = _opts(path, split)
    _check(lib().mx_gemm_workspace_size(ctypes.byref(L), M, ctypes.byref(o), ctypes.byref(n)),
           "mx_gemm_workspace_size")
    return n.value


def mx_gemm_select_path(L: Layout, M: int, path: int = 0, split: int = 0) -> int:
    o = _opts(path, split)
    r = lib().mx_gemm_select_path(ctypes.byref(L), M, ctypes.byref(o))
    if r < 0:
        _check(-r, "mx_gemm_select_path")
    return r


def mx_gemm(L: Layout, blob: torch.Tensor, Aq: torch.Tensor, s_a: torch.Tensor, Y: torch.Tensor,
            workspace: torch.Tensor | None = None, path: int = 0, split: int = 0,
            debug_partials: torch.Tensor | None = None, status: torch.Tensor | None = None,
            wait_timeout_us: int = 0, test_stall: int = 0, act_group: int = 0, stream=None) -> None:
    M = Aq.shape[0]
    o = _opts(path, split, debug_partials, status, wait_timeout_us, test_stall, act_group)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mx_gemm(ctypes.byref(L), _ptr(blob), _ptr(Aq), _ptr(s_a), M, _ptr(Y), Y.stride(0),
                         _ptr(workspace), ws_bytes, ctypes.byref(o), _stream(stream)), "mx_gemm")


def mx_linear_workspace_size(L: Layout, M: int, xdtype=torch.float16, path: int = 0, split: int = 0,
                             act_group: int = 0) -> int:
    n = ctypes.c_size_t(0)
    o = _opts(path, split, act_group=act_group)
    code = MX_F16 if xdtype == torch.float16 else MX_F32
    _check(lib().mx_linear_workspace_size(ctypes.byref(L), M, code, ctypes.byref(o), ctypes.byref(n)),
           "mx_linear_workspace_size")
    return n.value


def mx_linear(L: Layout, blob: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
              workspace: torch.Tensor | None = None, path: int = 0, split: int = 0,
              debug_partials: torch.Tensor | None = None, status: torch.Tensor | None = None,
              act_group: int = 0, stream=None) -> None:
    assert X.dim() == 2 and X.stride(1) == 1
    M = X.shape[0]
    o = _opts(path, split, debug_partials, status, act_group=act_group)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().mx_linear(ctypes.byref(L), _ptr(blob), _ptr(X), _dtype_code(X), M, X.stride(0),
                           _ptr(Y), Y.stride(0), _ptr(workspace), ws_bytes, ctypes.byref(o),
                           _stream(stream)), "mx_linear")


NOALLOC_SCRATCH_BYTES = 4 << 20      # MX_NOALLOC_SCRATCH_BYTES


def mx_linear_noalloc(L: Layout, blob: torch.Tensor, X: torch.Tensor, Y: torch.Tensor, path: int = 0,
                      split: int = 0, debug_partials: torch.Tensor | None = None,
                      status: torch.Tensor | None = None, act_group: int = 0, stream=None) -> None:
    assert X.dim() == 2 and X.stride(1) == 1
    o = _opts(path, split, debug_partials, status, act_group=act_group)
    _check(lib().mx_linear_noalloc(ctypes.byref(L), _ptr(blob), _ptr(X), _dtype_code(X), X.shape[0],
                                   X.stride(0), _ptr(Y), Y.stride(0), ctypes.byref(o), _stream(stream)),
           "mx_linear_noalloc")


def mx_copy_mapped(dst: torch.Tensor, src: torch.Tensor, stream=None) -> None:
    """Copy src into dst with a kernel; either may be pinned host memory (see mx.h)."""
    if dst.nbytes != src.nbytes:
        raise ValueError(f"mx_copy_mapped: {dst.nbytes} bytes into {src.nbytes}")
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("mx_copy_mapped: contiguous tensors only")
    for t, n in ((dst, "dst"), (src, "src")):
        if not t.is_cuda and not t.is_pinned():
            raise ValueError(f"mx_copy_mapped: {n} is pageable host memory (pin it first)")
    _check(lib().mx_copy_mapped(_ptr(dst), _ptr(src), dst.nbytes, _stream(stream)), "mx_copy_mapped")


def mx_saliency(W: torch.Tensor, G: torch.Tensor, group: int, S: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Per-row channel saliency of one layer (see mx.h); returns S (device fp32 [N])."""
    assert W.dim() == 2 and W.stride(1) == 1 and G.shape == W.shape and G.stride(1) == 1
    N, K = W.shape
    if S is None:
        S = torch.empty(N, dtype=torch.float32, device=W.device)
    _check(lib().mx_saliency(_ptr(W), _dtype_code(W), W.stride(0), _ptr(G), _dtype_code(G), G.stride(0), N, K,
                             group, _ptr(S), _stream(stream)), "mx_saliency")
    return S


def mx_select_top(S: torch.Tensor, n_top: int, is8: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The n_top largest of the concatenated scores, ties to the lower index (see mx.h);
    returns the uint8 mask."""
    assert S.dim() == 1 and S.dtype == torch.float32 and S.is_contiguous()
    n = S.numel()
    if is8 is None:
        is8 = torch.empty(n, dtype=torch.uint8, device=S.device)
    nb = ctypes.c_size_t(0)
    _check(lib().mx_select_top_workspace_size(n, ctypes.byref(nb)), "mx_select_top_workspace_size")
    ws = torch.empty(max(nb.value, 16), dtype=torch.uint8, device=S.device)
    _check(lib().mx_select_top(_ptr(S), n, n_top, _ptr(is8), _ptr(ws), ws.numel(), _stream(stream)),
           "mx_select_top")
    return is8


# ------------------------------------------------------------------ block-wise bit widths
def _host_bytes(a) -> ctypes.Array:
    b = bytes(np.ascontiguousarray(np.asarray(a, dtype=np.uint8)).tobytes())
    return (ctypes.c_uint8 * max(1, len(b))).from_buffer_copy(b if b else b"\0")


def mx_bw_layout_init(N: int, K: int, table, meta) -> BwLayout:
    """Geometry of a block-wise layer (see mx_blockwise.h); table: four widths, meta: the
    packed 2-bit block codes (host bytes)."""
    L = BwLayout()
    _check(lib().mx_bw_layout_init(N, K, _host_bytes(table), _host_bytes(meta), ctypes.byref(L)),
           "mx_bw_layout_init")
    return L


def mx_bw_pack(L: BwLayout, meta, W: torch.Tensor, blob: torch.Tensor, stream=None) -> None:
    assert W.dim() == 2 and W.stride(1) == 1 and tuple(W.shape) == (L.N, L.K)
    assert blob.numel() * blob.element_size() >= L.total_bytes
    _check(lib().mx_bw_pack(ctypes.byref(L), _host_bytes(meta), _ptr(W), _dtype_code(W), W.stride(0), _ptr(blob),
                            _stream(stream)), "mx_bw_pack")


def mx_bw_gemm(L: BwLayout, blob: torch.Tensor, Aq: torch.Tensor, s_a: torch.Tensor, Y: torch.Tensor,
               partials: torch.Tensor | None = None, stream=None) -> None:
    assert Aq.dim() == 2 and Aq.is_contiguous() and Aq.dtype == torch.int8 and Aq.shape[1] == L.K
    assert s_a.dtype == torch.float16 and Y.dtype == torch.float16 and Y.stride(1) == 1
    M = Aq.shape[0]
    assert blob.numel() * blob.element_size() >= L.total_bytes and s_a.numel() >= M
    assert Y.shape[0] >= M and Y.shape[1] >= L.N
    assert partials is None or (partials.dtype == torch.int32 and partials.is_contiguous()
                                and partials.numel() >= M * L.N * L.KB)
    _check(lib().mx_bw_gemm(ctypes.byref(L), _ptr(blob), _ptr(Aq), _ptr(s_a), Aq.shape[0], _ptr(Y), Y.stride(0),
                            _ptr(partials), _stream(stream)), "mx_bw_gemm")


# ------------------------------------------------------------------ microscaled 4-bit floating point
_DTYPES = {torch.float32: MX_F32, torch.float16: MX_F16, torch.bfloat16: MX_BF16}


def _code(dtype: torch.dtype) -> int:
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype} (float32, float16 or bfloat16)")
    return _DTYPES[dtype]


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _rows(t: torch.Tensor, name: str, rows: int, cols: int) -> int:
    """Row stride of a [rows, cols] matrix with contiguous rows."""
    if t.shape != (rows, cols):
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.is_contiguous():
        return cols
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: columns must be contiguous")
    # the stride of a single row means nothing; torch may give any
    return ld if rows > 1 or ld > cols else cols


def _matrices(t: torch.Tensor, name: str, L: Fp4Layout) -> tuple[int, int]:
    """(row stride, matrix stride) of [rows, K], or [groups, rows, K]."""
    if t.dim() == 2 and L.groups == 1:
        return _rows(t, name, L.rows, L.K), 0
    if t.dim() != 3 or t.shape[0] != L.groups:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {(L.groups, L.rows, L.K)}")
    return _rows(t[0], name, L.rows, L.K), t.stride(0)


def _vec(t: torch.Tensor | None, name: str, n: int, dtype=torch.float32) -> int | None:
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous {dtype} values needed")
    return t.data_ptr()


def _blob(t: torch.Tensor, name: str, nbytes: int) -> int:
    if t.nbytes < nbytes or not t.is_contiguous():
        raise ValueError(f"{name}: {nbytes} contiguous bytes needed")
    return t.data_ptr()


# options are values alone: a layer passes the same ones in every call
_made_fp4_opts = functools.lru_cache(maxsize=256)(Fp4Opts)


def _fp4_opts(path: int, split: int, status, wait_timeout_us: int, test_stall: int) -> Fp4Opts | None:
    if not (path or split or status is not None or wait_timeout_us or test_stall):
        return None
    return _made_fp4_opts(path, split, _ptr(status), wait_timeout_us, test_stall)


def mx_fp4_layout_init(rows: int, K: int, format: int = FP4_E4M3_16, groups: int = 1) -> Fp4Layout:
    L = Fp4Layout()
    _check(lib().mx_fp4_layout_init(rows, K, format, groups, ctypes.byref(L)), "mx_fp4_layout_init")
    return L


def mx_fp4_layout_from_header(header) -> Fp4Layout:
    """header: bytes, or a host uint8 tensor holding the blob's first 256 bytes."""
    if isinstance(header, torch.Tensor):
        header = bytes(header[:HEADER_BYTES].cpu().numpy().tobytes())
    buf = ctypes.create_string_buffer(bytes(header), len(header))
    L = Fp4Layout()
    _check(lib().mx_fp4_layout_from_header(buf, len(header), ctypes.byref(L)), "mx_fp4_layout_from_header")
    return L


def mx_fp4_gscale(L: Fp4Layout, X: torch.Tensor, gscale: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The scale of each of the layout's matrices (see mx_fp4.h); returns fp32 [groups]."""
    ldx, gsx = _matrices(X, "X", L)
    if gscale is None:
        gscale = _new(X, L.groups, stream, torch.float32)
    _check(lib().mx_fp4_gscale(L, X.data_ptr(), _code(X.dtype), ldx, gsx, _vec(gscale, "gscale", L.groups),
                               _stream(stream)), "mx_fp4_gscale")
    return gscale


def mx_fp4_quant(L: Fp4Layout, X: torch.Tensor, blob: torch.Tensor, gscale: torch.Tensor | None = None,
                 stream=None) -> None:
    """X [rows, K] (or [groups, rows, K]) into blob."""
    ldx, gsx = _matrices(X, "X", L)
    _check(lib().mx_fp4_quant(L, X.data_ptr(), _code(X.dtype), ldx, gsx, _vec(gscale, "gscale", L.groups),
                              _blob(blob, "blob", L.total_bytes), _stream(stream)), "mx_fp4_quant")


def mx_fp4_dequant(L: Fp4Layout, blob: torch.Tensor, dtype=torch.float32, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """The blob's values, [rows, K] (or [groups, rows, K]) of dtype."""
    if out is None:
        shape = (L.rows, L.K) if L.groups == 1 else (L.groups, L.rows, L.K)
        out = _new(blob, shape, stream, dtype)
    ldo, gso = _matrices(out, "out", L)
    _check(lib().mx_fp4_dequant(L, _blob(blob, "blob", L.total_bytes), out.data_ptr(), _code(out.dtype), ldo, gso,
                                _stream(stream)), "mx_fp4_dequant")
    return out


def mx_fp4_gemm(LW: Fp4Layout, wblob: torch.Tensor, LA: Fp4Layout, ablob: torch.Tensor, Y: torch.Tensor,
                path: int = 0, split: int = 0, status: torch.Tensor | None = None, wait_timeout_us: int = 0,
                test_stall: int = 0, stream=None) -> None:
    """Y [LA.rows, LW.rows] = A W^T."""
    ldy = _rows(Y, "Y", LA.rows, LW.rows)
    _check(lib().mx_fp4_gemm(LW, _blob(wblob, "weight blob", LW.total_bytes), LA,
                             _blob(ablob, "activation blob", LA.total_bytes), Y.data_ptr(), _code(Y.dtype), ldy,
                             _fp4_opts(path, split, status, wait_timeout_us, test_stall), _stream(stream)),
           "mx_fp4_gemm")


def mx_fp4_linear_workspace_size(LW: Fp4Layout, M: int, path: int = 0, split: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx_fp4_linear_workspace_size(LW, M, _fp4_opts(path, split, None, 0, 0), ctypes.byref(n)),
           "mx_fp4_linear_workspace_size")
    return n.value


def mx_fp4_linear(LW: Fp4Layout, wblob: torch.Tensor, X: torch.Tensor, Y: torch.Tensor,
                  workspace: torch.Tensor | None = None, gscale: torch.Tensor | None = None, path: int = 0, split: int = 0,
                  status: torch.Tensor | None = None, stream=None, wait_timeout_us: int = 0, test_stall: int = 0) -> None:
    """Y [M, LW.rows] = X W^T (see mx_fp4.h)."""
    M = X.shape[0]
    ldx, ldy = _rows(X, "X", M, LW.K), _rows(Y, "Y", M, LW.rows)
    _check(lib().mx_fp4_linear(LW, _blob(wblob, "weight blob", LW.total_bytes), X.data_ptr(), _code(X.dtype), M, ldx,
                               _vec(gscale, "gscale", 1), Y.data_ptr(), _code(Y.dtype), ldy, _ptr(workspace),
                               0 if workspace is None else workspace.nbytes,
                               _fp4_opts(path, split, status, wait_timeout_us, test_stall), _stream(stream)),
           "mx_fp4_linear")


# ------------------------------------------------------------------ experts
def mx_experts_layout_init(T: int, k: int, E: int) -> ExpertsLayout:
    P = ExpertsLayout()
    _check(lib().mx_experts_layout_init(T, k, E, ctypes.byref(P)), "mx_experts_layout_init")
    return P


class ExpertsPlan:
    """A plan buffer (see mx_experts.h) and its sections as int32 tensors."""

    def __init__(self, P: ExpertsLayout, device="cuda", buffer: torch.Tensor | None = None):
        self.P = P
        self.buffer = torch.empty(P.total_bytes, dtype=torch.uint8, device=device) if buffer is None else buffer
        self.ptr = _blob(self.buffer, "plan", P.total_bytes)

    def _section(self, off: int, n: int) -> torch.Tensor:
        return self.buffer[off:off + 4 * n].view(torch.int32)

    @functools.cached_property
    def order(self) -> torch.Tensor:
        """Slot of each sorted row, -1 behind the last."""
        return self._section(self.P.off_order, self.P.n)

    @functools.cached_property
    def pos(self) -> torch.Tensor:
        """Sorted row of each slot, -1 where it is dropped."""
        return self._section(self.P.off_pos, self.P.n)

    @functools.cached_property
    def dest(self) -> torch.Tensor:
        """Row of each slot in the tiled activations, -1 where it is dropped."""
        return self._section(self.P.off_dest, self.P.n)

    @functools.cached_property
    def offsets(self) -> torch.Tensor:
        """First sorted row of each expert; the last entry is the number of kept rows."""
        return self._section(self.P.off_offsets, self.P.E + 1)

    @functools.cached_property
    def tiles(self) -> torch.Tensor:
        """First 128-row tile of each expert."""
        return self._section(self.P.off_tiles, self.P.E + 1)


def mx_experts_sort(plan: ExpertsPlan, ids: torch.Tensor, stream=None) -> None:
    """ids int32 [T, k] into plan."""
    _check(lib().mx_experts_sort(plan.P, _vec(ids, "ids", plan.P.n, torch.int32), plan.ptr, _stream(stream)),
           "mx_experts_sort")


def mx_experts_gather(plan: ExpertsPlan, X: torch.Tensor, Xs: torch.Tensor, stream=None) -> None:
    """Xs [n, H]: the token rows X [T, H] in sorted order; rows behind the kept ones stay as they are."""
    H = X.shape[1]
    _need(X.dtype == Xs.dtype, "X and Xs must have one dtype")
    _check(lib().mx_experts_gather(plan.P, plan.ptr, X.data_ptr(), _code(X.dtype), H, _rows(X, "X", plan.P.T, H),
                                   Xs.data_ptr(), _rows(Xs, "Xs", plan.P.n, H), _stream(stream)), "mx_experts_gather")


def mx_experts_gather_bwd(plan: ExpertsPlan, dXs: torch.Tensor, dX: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor:
    """dX [T, H] of mx_experts_gather from dXs [n, H]."""
    P, H = plan.P, dXs.shape[1]
    if dX is None:
        dX, ldx = _new(dXs, (P.T, H), stream), H
    else:
        _need(dX.dtype == dXs.dtype, "dX and dXs must have one dtype")
        ldx = _rows(dX, "dX", P.T, H)
    _check(lib().mx_experts_gather_bwd(P, plan.ptr, dXs.data_ptr(), _code(dXs.dtype), H, _rows(dXs, "dXs", P.n, H),
                                       dX.data_ptr(), ldx, _stream(stream)), "mx_experts_gather_bwd")
    return dX


def mx_experts_combine(plan: ExpertsPlan, Ys: torch.Tensor, w: torch.Tensor, Y: torch.Tensor | None = None,
                       out_dtype=None, stream=None) -> torch.Tensor:
    """Y [T, H] = per token the weighted sum of its rows of Ys [n, H]; w fp32 [T, k]."""
    P, H = plan.P, Ys.shape[1]
    if Y is None:
        Y, ldy = _new(Ys, (P.T, H), stream, out_dtype), H
    else:
        ldy = _rows(Y, "Y", P.T, H)
    _check(lib().mx_experts_combine(P, plan.ptr, Ys.data_ptr(), _code(Ys.dtype), H, _rows(Ys, "Ys", P.n, H),
                                    _vec(w, "w", P.n), Y.data_ptr(), _code(Y.dtype), ldy, _stream(stream)),
           "mx_experts_combine")
    return Y


def mx_experts_combine_bwd(plan: ExpertsPlan, dY: torch.Tensor, Ys: torch.Tensor, w: torch.Tensor,
                           dYs: torch.Tensor | None = None, dw: torch.Tensor | None = None,
                           stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """(dYs, dw) of mx_experts_combine; rows of dYs behind the kept ones stay as they are
    (zero when dYs is not given)."""
    P, H = plan.P, Ys.shape[1]
    if dYs is None:
        dYs = _new(Ys, (P.n, H), stream, zeros=True)
    if dw is None:
        dw = _new(w, w.shape, stream)
    _need(dY.dtype == Ys.dtype == dYs.dtype, "dY, Ys and dYs must have one dtype")
    _check(lib().mx_experts_combine_bwd(P, plan.ptr, dY.data_ptr(), Ys.data_ptr(), _code(Ys.dtype), H,
                                        _rows(dY, "dY", P.T, H), _rows(Ys, "Ys", P.n, H), _vec(w, "w", P.n),
                                        dYs.data_ptr(), _rows(dYs, "dYs", P.n, H), _vec(dw, "dw", P.n),
                                        _stream(stream)), "mx_experts_combine_bwd")
    return dYs, dw


def mx_fp4_quant_sorted(L: Fp4Layout, plan: ExpertsPlan, X: torch.Tensor, blob: torch.Tensor, sorted: bool = False,
                        gscale: torch.Tensor | None = None, stream=None) -> None:
    """Token rows X [T, K] (or sorted rows [n, K]) into expert-ordered tiles."""
    ldx = _rows(X, "X", plan.P.n if sorted else plan.P.T, L.K)
    _check(lib().mx_fp4_quant_sorted(L, plan.P, plan.ptr, int(sorted), X.data_ptr(), _code(X.dtype), ldx,
                                     _vec(gscale, "gscale", 1), _blob(blob, "blob", L.total_bytes), _stream(stream)),
           "mx_fp4_quant_sorted")


def mx_fp4_gemm_sorted(LW: Fp4Layout, wblob: torch.Tensor, LA: Fp4Layout, ablob: torch.Tensor, plan: ExpertsPlan,
                       Y: torch.Tensor, path: int = 0, split: int = 0, status: torch.Tensor | None = None,
                       wait_timeout_us: int = 0, test_stall: int = 0, stream=None) -> None:
    """Y [n, LW.rows]: each expert's product over its sorted rows."""
    ldy = _rows(Y, "Y", plan.P.n, LW.rows)
    _check(lib().mx_fp4_gemm_sorted(LW, _blob(wblob, "weight blob", LW.total_bytes), LA,
                                    _blob(ablob, "activation blob", LA.total_bytes), plan.P, plan.ptr, Y.data_ptr(),
                                    _code(Y.dtype), ldy, _fp4_opts(path, split, status, wait_timeout_us, test_stall),
                                    _stream(stream)), "mx_fp4_gemm_sorted")


def mx_fp4_linear_sorted_workspace_size(LW: Fp4Layout, P: ExpertsLayout, path: int = 0, split: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx_fp4_linear_sorted_workspace_size(LW, P, _fp4_opts(path, split, None, 0, 0), ctypes.byref(n)),
           "mx_fp4_linear_sorted_workspace_size")
    return n.value


def mx_fp4_linear_sorted(LW: Fp4Layout, wblob: torch.Tensor, plan: ExpertsPlan, X: torch.Tensor, Y: torch.Tensor,
                         workspace: torch.Tensor | None = None, sorted: bool = False, gscale: torch.Tensor | None = None,
                         path: int = 0, split: int = 0, status: torch.Tensor | None = None, stream=None,
                         wait_timeout_us: int = 0, test_stall: int = 0) -> None:
    """mx_fp4_quant_sorted and mx_fp4_gemm_sorted in one call."""
    ldx = _rows(X, "X", plan.P.n if sorted else plan.P.T, LW.K)
    ldy = _rows(Y, "Y", plan.P.n, LW.rows)
    _check(lib().mx_fp4_linear_sorted(LW, _blob(wblob, "weight blob", LW.total_bytes), plan.P, plan.ptr, int(sorted),
                                      X.data_ptr(), _code(X.dtype), ldx, _vec(gscale, "gscale", 1), Y.data_ptr(),
                                      _code(Y.dtype), ldy, _ptr(workspace),
                                      0 if workspace is None else workspace.nbytes,
                                      _fp4_opts(path, split, status, wait_timeout_us, test_stall), _stream(stream)),
           "mx_fp4_linear_sorted")


def mx_fp4_experts_workspace_size(LW: Fp4Layout, P: ExpertsLayout, path: int = 0, split: int = 0) -> int:
    n = ctypes.c_size_t(0)
    _check(lib().mx_fp4_experts_workspace_size(LW, P, _fp4_opts(path, split, None, 0, 0), ctypes.byref(n)),
           "mx_fp4_experts_workspace_size")
    return n.value


def mx_fp4_experts(LW: Fp4Layout, wblob: torch.Tensor, P: ExpertsLayout, ids: torch.Tensor, X: torch.Tensor,
                   w: torch.Tensor, Y: torch.Tensor, workspace: torch.Tensor, gscale: torch.Tensor | None = None,
                   path: int = 0, split: int = 0, status: torch.Tensor | None = None, stream=None,
                   wait_timeout_us: int = 0, test_stall: int = 0) -> None:
    """Y [T, LW.rows]: sort, one projection per expert and weighted sum (see mx_fp4.h)."""
    _check(lib().mx_fp4_experts(LW, _blob(wblob, "weight blob", LW.total_bytes), P, _vec(ids, "ids", P.n, torch.int32),
                                X.data_ptr(), _code(X.dtype), _rows(X, "X", P.T, LW.K), _vec(gscale, "gscale", 1),
                                _vec(w, "w", P.n), Y.data_ptr(), _code(Y.dtype), _rows(Y, "Y", P.T, LW.rows),
                                _ptr(workspace), 0 if workspace is None else workspace.nbytes,
                                _fp4_opts(path, split, status, wait_timeout_us, test_stall), _stream(stream)),
           "mx_fp4_experts")
