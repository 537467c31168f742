"""Thin ctypes binding of ``libnvfp4rs.so`` (declared in ``include/nvfp4rs.h``).

Argument marshalling only: every function here checks that tensors are CUDA,
contiguous and of the right dtype, turns them into device pointers, passes the
current torch stream, and raises ``NVFP4Error`` on a non-OK status. All of the
method's work happens in the library's kernels. If the library is not built,
every call raises; there is no fallback.

Names follow the C entry points. Tensors:
  x            bf16 [rows, K]
  row_amax     fp32 [rows]          col_amax  fp32 [E*K]
  row_data     uint8 [rows, K/2]    row_scale uint8 [rows, K/16]   row_s2 fp32 [rows]
  col_data     uint8 [rows*K/2]     col_scale uint8 [rows*K/16]    col_s2 fp32 [E*K]
(colwise buffers hold each group's transposed [K, m_g/2] / [K, m_g/16] slice
at byte offsets K*o_g/2 and K*o_g/16).
"""
from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional, Sequence

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# NVFP4RS_LIBRARY names another build of the same library to load instead
# (the bounds-checked debug build, libnvfp4rs_debug.so, for instance)
LIB_PATH = os.environ.get("NVFP4RS_LIBRARY") or os.path.join(HERE, "libnvfp4rs.so")

NVFP4_OK = 0
NVFP4_ERR_INVALID_ARG = 1
NVFP4_ERR_UNSUPPORTED = 2
NVFP4_ERR_CUDA = 3
NVFP4_ERR_ROUTING = 4
NVFP4_ERR_TIMEOUT = 5
NVFP4_MAX_GROUPS = 1024
NVFP4_SCALE_COMPACT = 0
NVFP4_SCALE_TILED_128X4 = 1
NVFP4_OUT_F32 = 0
NVFP4_OUT_BF16 = 1

_lib = None


class NVFP4Error(RuntimeError):
    def __init__(self, what: str, status: int):
        super().__init__(f"{what}: {status_name(status)} ({status})")
        self.status = status


class Outputs(ctypes.Structure):
    """Mirror of ``nvfp4_outputs``."""
    _fields_ = [("row_data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("row_s2", ctypes.c_void_p), ("col_data", ctypes.c_void_p),
                ("col_scale", ctypes.c_void_p), ("col_s2", ctypes.c_void_p),
                ("scale_layout", ctypes.c_int32)]


class MxOutputs(ctypes.Structure):
    """Mirror of ``nvfp4_mx_outputs``."""
    _fields_ = [("row_data", ctypes.c_void_p), ("row_scale", ctypes.c_void_p),
                ("col_data", ctypes.c_void_p), ("col_scale", ctypes.c_void_p)]


class Matrix(ctypes.Structure):
    """Mirror of ``nvfp4_matrix``."""
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("scale_layout", ctypes.c_int32)]


def lib():
    """Open the library (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               f"`python -m nvfp4_row_scaled_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        L.nvfp4_group_amax.argtypes = [vp, i64, i64, vp, i32, vp, vp, vp]
        L.nvfp4_group_cast.argtypes = [vp, i64, i64, vp, i32, vp, vp, ctypes.POINTER(Outputs), vp]
        L.nvfp4_group_amax_graphsafe.argtypes = [vp, i64, i64, vp, vp, i32, vp, vp, vp, vp]
        L.nvfp4_group_cast_graphsafe.argtypes = [vp, i64, i64, vp, vp, i32, vp, vp,
                                                 ctypes.POINTER(Outputs), vp, vp]
        L.nvfp4_dequantize.argtypes = [vp, vp, vp, i64, i64, vp, vp]
        sz = ctypes.c_size_t
        L.nvfp4_group_quantize_workspace_bytes.argtypes = [i64, i32]
        L.nvfp4_group_quantize_workspace_bytes.restype = sz
        L.nvfp4_group_quantize.argtypes = [vp, i64, i64, vp, i32, vp, vp, ctypes.POINTER(Outputs),
                                           vp, sz, vp]
        L.nvfp4_group_quantize_graphsafe.argtypes = [vp, i64, i64, vp, vp, i32, vp, vp,
                                                     ctypes.POINTER(Outputs), vp, sz, vp, vp]
        L.nvfp4_mx_group_cast.argtypes = [vp, i64, i64, vp, i32, ctypes.POINTER(MxOutputs), vp]
        L.nvfp4_mx_group_cast_graphsafe.argtypes = [vp, i64, i64, vp, vp, i32, ctypes.POINTER(MxOutputs),
                                                    vp, vp]
        L.nvfp4_mx_dequantize.argtypes = [vp, vp, i64, i64, vp, vp]
        for f in ("nvfp4_mx_group_cast", "nvfp4_mx_group_cast_graphsafe", "nvfp4_mx_dequantize"):
            getattr(L, f).restype = ctypes.c_int
        L.nvfp4_row_post_scale.argtypes = [vp, i64, i64, vp, vp, vp, i32, vp]
        L.nvfp4_row_post_scale.restype = ctypes.c_int
        L.nvfp4_group_quantize_noalloc.argtypes = [vp, i64, i64, vp, i32, vp, vp,
                                                   ctypes.POINTER(Outputs), vp]
        mp = ctypes.POINTER(Matrix)
        L.nvfp4_group_gemm.argtypes = [mp, i64, i64, vp, i32, mp, i64, vp, i32, vp]
        L.nvfp4_group_gemm_graphsafe.argtypes = [mp, i64, i64, vp, vp, i32, mp, i64, vp, i32, vp, vp]
        L.nvfp4_group_gated_gemm.argtypes = [mp, i64, i64, vp, i32, mp, i64, vp, vp, vp]
        L.nvfp4_group_gated_gemm_graphsafe.argtypes = [mp, i64, i64, vp, vp, i32, mp, i64, vp, vp, vp, vp]
        L.nvfp4_group_wgrad.argtypes = [mp, mp, i64, vp, i32, i64, i64, vp, i32, vp]
        L.nvfp4_group_wgrad_graphsafe.argtypes = [mp, mp, i64, vp, vp, i32, i64, i64, vp, i32, vp, vp]
        L.nvfp4_group_gated_backward.argtypes = [vp, vp, i64, i64, vp, i32, vp, vp, vp, vp]
        L.nvfp4_group_gated_backward_graphsafe.argtypes = [vp, vp, i64, i64, vp, vp, i32, vp, vp, vp, vp, vp]
        L.nvfp4_adapter_workspace_bytes.argtypes = [i64, i32]
        L.nvfp4_adapter_workspace_bytes.restype = sz
        L.nvfp4_adapter_gemm.argtypes = [vp, mp, i64, i64, mp, i64, vp, vp, vp, i32, i32, vp, vp, i32, vp, sz, vp, vp]
        for f in ("nvfp4_group_gemm", "nvfp4_group_gemm_graphsafe", "nvfp4_group_gated_gemm",
                  "nvfp4_group_gated_gemm_graphsafe", "nvfp4_group_wgrad", "nvfp4_group_wgrad_graphsafe",
                  "nvfp4_group_gated_backward", "nvfp4_group_gated_backward_graphsafe", "nvfp4_adapter_gemm"):
            getattr(L, f).restype = ctypes.c_int
        for f in ("nvfp4_group_amax", "nvfp4_group_cast", "nvfp4_group_amax_graphsafe",
                  "nvfp4_group_cast_graphsafe", "nvfp4_dequantize", "nvfp4_group_quantize",
                  "nvfp4_group_quantize_graphsafe", "nvfp4_group_quantize_noalloc"):
            getattr(L, f).restype = ctypes.c_int
        L.nvfp4_status_string.argtypes = [ctypes.c_int]
        L.nvfp4_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_name(status: int) -> str:
    return lib().nvfp4_status_string(int(status)).decode()


# ----------------------------------------------------------- marshalling

def _dev(t: Optional[torch.Tensor], dtype: torch.dtype, name: str):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream: Optional[torch.cuda.Stream]):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _splits(m_splits: Sequence[int]):
    arr = (ctypes.c_int64 * max(len(m_splits), 1))(*[int(m) for m in m_splits])
    return arr, len(m_splits)


def _outputs(out: Dict[str, torch.Tensor], scale_layout: int = NVFP4_SCALE_COMPACT) -> Outputs:
    o = Outputs()
    o.scale_layout = int(scale_layout)
    for name, dt in (("row_data", torch.uint8), ("row_scale", torch.uint8), ("row_s2", torch.float32),
                     ("col_data", torch.uint8), ("col_scale", torch.uint8), ("col_s2", torch.float32)):
        p = _dev(out.get(name), dt, name)
        setattr(o, name, p.value if p is not None else None)
    return o


def _groups(first_dims: Optional[torch.Tensor], num_groups: Optional[int]) -> int:
    """Group count of a graph-safe call: first_dims.numel(), or num_groups for
    uniform groups (first_dims and tensor_offsets both None)."""
    if first_dims is not None:
        return first_dims.numel()
    if num_groups is None:
        raise ValueError("uniform groups (no first_dims) need num_groups")
    return int(num_groups)


def _check(rc: int, what: str):
    if rc != NVFP4_OK:
        raise NVFP4Error(what, rc)


# ------------------------------------------------------------ entry points

def nvfp4_group_amax(x: torch.Tensor, m_splits: Sequence[int], row_amax: Optional[torch.Tensor],
                     col_amax: Optional[torch.Tensor], stream=None) -> None:
    arr, E = _splits(m_splits)
    rc = lib().nvfp4_group_amax(_dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1], arr, E,
                                _dev(row_amax, torch.float32, "row_amax"),
                                _dev(col_amax, torch.float32, "col_amax"), _stream(stream))
    _check(rc, "nvfp4_group_amax")


def nvfp4_group_cast(x: torch.Tensor, m_splits: Sequence[int], row_amax: Optional[torch.Tensor],
                     col_amax: Optional[torch.Tensor], out: Dict[str, torch.Tensor],
                     stream=None, scale_layout: int = NVFP4_SCALE_COMPACT) -> None:
    arr, E = _splits(m_splits)
    o = _outputs(out, scale_layout)
    rc = lib().nvfp4_group_cast(_dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1], arr, E,
                                _dev(row_amax, torch.float32, "row_amax"),
                                _dev(col_amax, torch.float32, "col_amax"), ctypes.byref(o),
                                _stream(stream))
    _check(rc, "nvfp4_group_cast")


def nvfp4_group_amax_graphsafe(x: torch.Tensor, first_dims: torch.Tensor,
                               tensor_offsets: torch.Tensor, row_amax: Optional[torch.Tensor],
                               col_amax: Optional[torch.Tensor], status: torch.Tensor,
                               stream=None, num_groups: Optional[int] = None) -> None:
    rc = lib().nvfp4_group_amax_graphsafe(
        _dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1],
        _dev(first_dims, torch.int64, "first_dims"), _dev(tensor_offsets, torch.int64, "tensor_offsets"),
        _groups(first_dims, num_groups), _dev(row_amax, torch.float32, "row_amax"),
        _dev(col_amax, torch.float32, "col_amax"), _dev(status, torch.int32, "status"),
        _stream(stream))
    _check(rc, "nvfp4_group_amax_graphsafe")


def nvfp4_group_cast_graphsafe(x: torch.Tensor, first_dims: torch.Tensor,
                               tensor_offsets: torch.Tensor, row_amax: Optional[torch.Tensor],
                               col_amax: Optional[torch.Tensor], out: Dict[str, torch.Tensor],
                               status: torch.Tensor, stream=None,
                               scale_layout: int = NVFP4_SCALE_COMPACT,
                               num_groups: Optional[int] = None) -> None:
    o = _outputs(out, scale_layout)
    rc = lib().nvfp4_group_cast_graphsafe(
        _dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1],
        _dev(first_dims, torch.int64, "first_dims"), _dev(tensor_offsets, torch.int64, "tensor_offsets"),
        _groups(first_dims, num_groups), _dev(row_amax, torch.float32, "row_amax"),
        _dev(col_amax, torch.float32, "col_amax"), ctypes.byref(o),
        _dev(status, torch.int32, "status"), _stream(stream))
    _check(rc, "nvfp4_group_cast_graphsafe")


def nvfp4_group_quantize_workspace_bytes(capacity_rows: int, num_groups: int) -> int:
    return int(lib().nvfp4_group_quantize_workspace_bytes(int(capacity_rows), int(num_groups)))


def _workspace(ws: torch.Tensor):
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor")
    return ctypes.c_void_p(ws.data_ptr()), ws.numel() * ws.element_size()


def nvfp4_group_quantize(x: torch.Tensor, m_splits: Sequence[int], row_amax: Optional[torch.Tensor],
                         col_amax: Optional[torch.Tensor], out: Dict[str, torch.Tensor],
                         workspace: torch.Tensor, stream=None, scale_layout: int = NVFP4_SCALE_COMPACT) -> None:
    arr, E = _splits(m_splits)
    o = _outputs(out, scale_layout)
    wp, wb = _workspace(workspace)
    rc = lib().nvfp4_group_quantize(_dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1], arr, E,
                                    _dev(row_amax, torch.float32, "row_amax"),
                                    _dev(col_amax, torch.float32, "col_amax"), ctypes.byref(o),
                                    wp, wb, _stream(stream))
    _check(rc, "nvfp4_group_quantize")


def nvfp4_group_quantize_graphsafe(x: torch.Tensor, first_dims: torch.Tensor,
                                   tensor_offsets: torch.Tensor, row_amax: Optional[torch.Tensor],
                                   col_amax: Optional[torch.Tensor], out: Dict[str, torch.Tensor],
                                   workspace: torch.Tensor, status: torch.Tensor,
                                   stream=None, scale_layout: int = NVFP4_SCALE_COMPACT,
                                   num_groups: Optional[int] = None) -> None:
    o = _outputs(out, scale_layout)
    wp, wb = _workspace(workspace)
    rc = lib().nvfp4_group_quantize_graphsafe(
        _dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1],
        _dev(first_dims, torch.int64, "first_dims"), _dev(tensor_offsets, torch.int64, "tensor_offsets"),
        _groups(first_dims, num_groups), _dev(row_amax, torch.float32, "row_amax"),
        _dev(col_amax, torch.float32, "col_amax"), ctypes.byref(o), wp, wb,
        _dev(status, torch.int32, "status"), _stream(stream))
    _check(rc, "nvfp4_group_quantize_graphsafe")


def nvfp4_group_quantize_noalloc(x: torch.Tensor, m_splits: Sequence[int],
                                 row_amax: Optional[torch.Tensor], col_amax: Optional[torch.Tensor],
                                 out: Dict[str, torch.Tensor], stream=None, scale_layout: int = NVFP4_SCALE_COMPACT) -> None:
    """nvfp4_group_quantize with the library's static scratch (no workspace)."""
    arr, E = _splits(m_splits)
    o = _outputs(out, scale_layout)
    rc = lib().nvfp4_group_quantize_noalloc(_dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1], arr, E,
                                            _dev(row_amax, torch.float32, "row_amax"),
                                            _dev(col_amax, torch.float32, "col_amax"), ctypes.byref(o),
                                            _stream(stream))
    _check(rc, "nvfp4_group_quantize_noalloc")


def nvfp4_row_post_scale(gemm_out: torch.Tensor, row_amax: torch.Tensor, out: torch.Tensor,
                         bias: Optional[torch.Tensor] = None, stream=None) -> None:
    """out = gemm_out * row_amax[:, None] (+ bias), as fp32 or bf16 (out's dtype)."""
    if out.dtype == torch.float32:
        dt = NVFP4_OUT_F32
    elif out.dtype == torch.bfloat16:
        dt = NVFP4_OUT_BF16
    else:
        raise ValueError("out must be float32 or bfloat16")
    if out.shape != gemm_out.shape:
        raise ValueError("out must have gemm_out's shape")
    rows, cols = gemm_out.shape
    rc = lib().nvfp4_row_post_scale(_dev(gemm_out, torch.float32, "gemm_out"), rows, cols,
                                    _dev(row_amax, torch.float32, "row_amax"),
                                    _dev(bias, torch.float32, "bias"), _dev(out, out.dtype, "out"), dt,
                                    _stream(stream))
    _check(rc, "nvfp4_row_post_scale")


def _mx_outputs(out: Dict[str, torch.Tensor]) -> MxOutputs:
    o = MxOutputs()
    for name in ("row_data", "row_scale", "col_data", "col_scale"):
        p = _dev(out.get(name), torch.uint8, name)
        setattr(o, name, p.value if p is not None else None)
    return o


def nvfp4_mx_group_cast(x: torch.Tensor, m_splits: Sequence[int], out: Dict[str, torch.Tensor],
                        stream=None) -> None:
    arr, E = _splits(m_splits)
    o = _mx_outputs(out)
    rc = lib().nvfp4_mx_group_cast(_dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1], arr, E,
                                   ctypes.byref(o), _stream(stream))
    _check(rc, "nvfp4_mx_group_cast")


def nvfp4_mx_group_cast_graphsafe(x: torch.Tensor, first_dims: Optional[torch.Tensor],
                                  tensor_offsets: Optional[torch.Tensor], out: Dict[str, torch.Tensor],
                                  status: torch.Tensor, stream=None,
                                  num_groups: Optional[int] = None) -> None:
    o = _mx_outputs(out)
    rc = lib().nvfp4_mx_group_cast_graphsafe(
        _dev(x, torch.bfloat16, "x"), x.shape[0], x.shape[1],
        _dev(first_dims, torch.int64, "first_dims"), _dev(tensor_offsets, torch.int64, "tensor_offsets"),
        _groups(first_dims, num_groups), ctypes.byref(o), _dev(status, torch.int32, "status"), _stream(stream))
    _check(rc, "nvfp4_mx_group_cast_graphsafe")


def nvfp4_mx_dequantize(data: torch.Tensor, scale: torch.Tensor, rows: int, cols: int, out: torch.Tensor,
                        stream=None) -> None:
    rc = lib().nvfp4_mx_dequantize(_dev(data, torch.uint8, "data"), _dev(scale, torch.uint8, "scale"),
                                   int(rows), int(cols), _dev(out, torch.float32, "out"), _stream(stream))
    _check(rc, "nvfp4_mx_dequantize")


def alloc_mx_outputs(rows: int, K: int, device="cuda", row: bool = True,
                     col: bool = True) -> Dict[str, torch.Tensor]:
    """Uninitialised output buffers of the grouped MXFP4 cast for ``rows`` rows."""
    out: Dict[str, torch.Tensor] = {}
    if row:
        out["row_data"] = torch.empty(rows, K // 2, dtype=torch.uint8, device=device)
        out["row_scale"] = torch.empty(rows, K // 32, dtype=torch.uint8, device=device)
    if col:
        out["col_data"] = torch.empty(rows * K // 2, dtype=torch.uint8, device=device)
        out["col_scale"] = torch.empty(rows * K // 32, dtype=torch.uint8, device=device)
    return out


def nvfp4_dequantize(data: torch.Tensor, scale: torch.Tensor, s2: torch.Tensor, rows: int, cols: int,
                     out: torch.Tensor, stream=None) -> None:
    rc = lib().nvfp4_dequantize(_dev(data, torch.uint8, "data"), _dev(scale, torch.uint8, "scale"),
                                _dev(s2, torch.float32, "s2"), int(rows), int(cols),
                                _dev(out, torch.float32, "out"), _stream(stream))
    _check(rc, "nvfp4_dequantize")


# --------------------------------------------------- products of the casts

def matrix(data: torch.Tensor, scale: torch.Tensor, s2: torch.Tensor,
           scale_layout: int = NVFP4_SCALE_COMPACT) -> Dict[str, object]:
    """An NVFP4 operand of the products: codes, block scales (in
    ``scale_layout``) and one fp32 factor a row."""
    return {"data": data, "scale": scale, "s2": s2, "scale_layout": int(scale_layout)}


def row_matrix(out: Dict[str, torch.Tensor], scale_layout: int = NVFP4_SCALE_COMPACT) -> Dict[str, object]:
    """The rowwise outputs of a cast as an operand."""
    return matrix(out["row_data"], out["row_scale"], out["row_s2"], scale_layout)


def col_matrix(out: Dict[str, torch.Tensor], scale_layout: int = NVFP4_SCALE_COMPACT) -> Dict[str, object]:
    """The colwise outputs of a cast (each group's transpose) as an operand."""
    return matrix(out["col_data"], out["col_scale"], out["col_s2"], scale_layout)


def _matrix(m: Dict[str, object], rows: int, elements: int, name: str) -> Matrix:
    """``m`` checked to be ``rows`` factors and ``elements`` codes."""
    for key, n in (("data", elements // 2), ("scale", elements // 16), ("s2", rows)):
        if m[key].numel() != n:
            raise ValueError(f"{name}[{key!r}] must have {n} entries, got {m[key].numel()}")
    o = Matrix()
    o.data = _dev(m["data"], torch.uint8, f"{name}['data']").value
    o.scale = _dev(m["scale"], torch.uint8, f"{name}['scale']").value
    o.s2 = _dev(m["s2"], torch.float32, f"{name}['s2']").value
    o.scale_layout = int(m.get("scale_layout", NVFP4_SCALE_COMPACT))
    return o


def _same_device(ref: torch.Tensor, *tensors) -> torch.device:
    """The one CUDA device of all the tensors (None is skipped)."""
    for t in tensors:
        if t is not None and t.device != ref.device:
            raise ValueError(f"tensors are on {ref.device} and {t.device}")
    if not ref.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    return ref.device


def _parts(*ms):
    return [m[k] for m in ms for k in ("data", "scale", "s2")]


def _on(dev: torch.device, stream, what: str, call) -> None:
    """Run ``call(stream pointer)`` with ``dev`` current, on its current stream
    unless one is given."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.device(dev):
        rc = call(_stream(stream))
    _check(rc, what)


def _out_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float32:
        return NVFP4_OUT_F32
    if t.dtype == torch.bfloat16:
        return NVFP4_OUT_BF16
    raise ValueError(f"{name} must be float32 or bfloat16")


def _width(w: Dict[str, object], x: Dict[str, object], rows: int, what: str) -> int:
    """Contraction width of x [rows, K] against stacked weights w."""
    ref, n = (x, rows) if rows else (w, w["s2"].numel())
    total = 2 * ref["data"].numel()
    if n and total % n:
        raise ValueError(f"{what}: {total} codes are not {n} equal rows")
    return total // n if n else 0


def nvfp4_group_gemm(x: Dict[str, object], m_splits: Sequence[int], w: Dict[str, object], y: torch.Tensor,
                     stream=None) -> None:
    """y [rows, N] (bf16 or fp32) = X_g W_g^T for each group's rows of x [rows, K]
    and its matrix of w [E*N, K]. Input gradients: x the rowwise cast of dy, w
    the colwise cast of the weights."""
    arr, E = _splits(m_splits)
    rows, N = y.shape
    K = _width(w, x, rows, "nvfp4_group_gemm")
    dt = _out_dtype(y, "y")
    dev = _same_device(y, *_parts(x, w))
    xm, wm = _matrix(x, rows, rows * K, "x"), _matrix(w, E * N, E * N * K, "w")
    yp = _dev(y, y.dtype, "y")
    _on(dev, stream, "nvfp4_group_gemm", lambda s: lib().nvfp4_group_gemm(
        ctypes.byref(xm), rows, K, arr, E, ctypes.byref(wm), N, yp, dt, s))


def nvfp4_group_gemm_graphsafe(x: Dict[str, object], first_dims: Optional[torch.Tensor],
                               tensor_offsets: Optional[torch.Tensor], w: Dict[str, object], y: torch.Tensor,
                               status: torch.Tensor, stream=None, num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    rows, N = y.shape
    K = _width(w, x, rows, "nvfp4_group_gemm_graphsafe")
    dt = _out_dtype(y, "y")
    dev = _same_device(y, first_dims, tensor_offsets, status, *_parts(x, w))
    xm, wm = _matrix(x, rows, rows * K, "x"), _matrix(w, E * N, E * N * K, "w")
    fd, to, st, yp = _routing(first_dims, tensor_offsets, status, E) + (_dev(y, y.dtype, "y"),)
    _on(dev, stream, "nvfp4_group_gemm_graphsafe", lambda s: lib().nvfp4_group_gemm_graphsafe(
        ctypes.byref(xm), rows, K, fd, to, E, ctypes.byref(wm), N, yp, dt, st, s))


def _routing(first_dims, tensor_offsets, status, E: int):
    if tensor_offsets is not None and tensor_offsets.numel() != E + 1:
        raise ValueError(f"tensor_offsets must have {E + 1} entries")
    return (_dev(first_dims, torch.int64, "first_dims"), _dev(tensor_offsets, torch.int64, "tensor_offsets"),
            _dev(status, torch.int32, "status"))


def _gated(x, w, h, gate_up, E):
    rows, F = h.shape
    if gate_up is not None and tuple(gate_up.shape) != (rows, 2 * F):
        raise ValueError("gate_up must be [rows, 2F]")
    K = _width(w, x, rows, "nvfp4_group_gated_gemm")
    return (rows, F, K, _matrix(x, rows, rows * K, "x"), _matrix(w, E * 2 * F, E * 2 * F * K, "w"),
            _dev(h, torch.bfloat16, "h"), _dev(gate_up, torch.bfloat16, "gate_up"))


def nvfp4_group_gated_gemm(x: Dict[str, object], m_splits: Sequence[int], w: Dict[str, object], h: torch.Tensor,
                           gate_up: Optional[torch.Tensor] = None, stream=None) -> None:
    """h [rows, F] = silu(X_g Wgate_g^T) * (X_g Wup_g^T); w [E*2F, K] holds each
    group's gate rows, then its up rows. gate_up [rows, 2F], if given, takes the
    two projections (bf16) for the gradient."""
    arr, E = _splits(m_splits)
    dev = _same_device(h, gate_up, *_parts(x, w))
    rows, F, K, xm, wm, hp, gp = _gated(x, w, h, gate_up, E)
    _on(dev, stream, "nvfp4_group_gated_gemm", lambda s: lib().nvfp4_group_gated_gemm(
        ctypes.byref(xm), rows, K, arr, E, ctypes.byref(wm), F, hp, gp, s))


def nvfp4_group_gated_gemm_graphsafe(x: Dict[str, object], first_dims: Optional[torch.Tensor],
                                     tensor_offsets: Optional[torch.Tensor], w: Dict[str, object], h: torch.Tensor,
                                     status: torch.Tensor, gate_up: Optional[torch.Tensor] = None, stream=None,
                                     num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    dev = _same_device(h, gate_up, first_dims, tensor_offsets, status, *_parts(x, w))
    rows, F, K, xm, wm, hp, gp = _gated(x, w, h, gate_up, E)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E)
    _on(dev, stream, "nvfp4_group_gated_gemm_graphsafe", lambda s: lib().nvfp4_group_gated_gemm_graphsafe(
        ctypes.byref(xm), rows, K, fd, to, E, ctypes.byref(wm), F, hp, gp, st, s))


def _wgrad(dy, x, dw, rows):
    E, N, K = dw.shape
    return (E, N, K, _matrix(dy, E * N, rows * N, "dy"), _matrix(x, E * K, rows * K, "x"),
            _dev(dw, dw.dtype, "dw"), _out_dtype(dw, "dw"))


def nvfp4_group_wgrad(dy: Dict[str, object], x: Dict[str, object], m_splits: Sequence[int], dw: torch.Tensor,
                      stream=None) -> None:
    """dw [E, N, K] (bf16 or fp32) = dY_g^T X_g from the colwise casts of dy
    [rows, N] and x [rows, K]; zero for an empty group."""
    arr, E = _splits(m_splits)
    if dw.shape[0] != E:
        raise ValueError(f"dw must have {E} matrices")
    rows = sum(int(m) for m in m_splits)
    dev = _same_device(dw, *_parts(dy, x))
    E, N, K, dm, xm, wp, dt = _wgrad(dy, x, dw, rows)
    _on(dev, stream, "nvfp4_group_wgrad", lambda s: lib().nvfp4_group_wgrad(
        ctypes.byref(dm), ctypes.byref(xm), rows, arr, E, N, K, wp, dt, s))


def nvfp4_group_wgrad_graphsafe(dy: Dict[str, object], x: Dict[str, object], capacity_rows: int,
                                first_dims: Optional[torch.Tensor], tensor_offsets: Optional[torch.Tensor],
                                dw: torch.Tensor, status: torch.Tensor, stream=None,
                                num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    if dw.shape[0] != E:
        raise ValueError(f"dw must have {E} matrices")
    rows = int(capacity_rows)
    dev = _same_device(dw, first_dims, tensor_offsets, status, *_parts(dy, x))
    E, N, K, dm, xm, wp, dt = _wgrad(dy, x, dw, rows)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E)
    _on(dev, stream, "nvfp4_group_wgrad_graphsafe", lambda s: lib().nvfp4_group_wgrad_graphsafe(
        ctypes.byref(dm), ctypes.byref(xm), rows, fd, to, E, N, K, wp, dt, st, s))


def _gated_backward(dh, gate_up, d_gate_up, row_amax, col_amax, E):
    rows, F = dh.shape
    for t, name in ((gate_up, "gate_up"), (d_gate_up, "d_gate_up")):
        if tuple(t.shape) != (rows, 2 * F):
            raise ValueError(f"{name} must be [rows, 2F]")
    for t, n, name in ((row_amax, rows, "row_amax"), (col_amax, E * 2 * F, "col_amax")):
        if t is not None and t.numel() != n:
            raise ValueError(f"{name} must have {n} entries")
    return (rows, F, _dev(dh, torch.bfloat16, "dh"), _dev(gate_up, torch.bfloat16, "gate_up"),
            _dev(d_gate_up, torch.bfloat16, "d_gate_up"), _dev(row_amax, torch.float32, "row_amax"),
            _dev(col_amax, torch.float32, "col_amax"))


def nvfp4_group_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, m_splits: Sequence[int],
                               d_gate_up: torch.Tensor, row_amax: Optional[torch.Tensor] = None,
                               col_amax: Optional[torch.Tensor] = None, stream=None) -> None:
    """d_gate_up [rows, 2F] from dh [rows, F] and the saved gate_up [rows, 2F]
    of nvfp4_group_gated_gemm, with the row amax [rows] and per-group column
    amax [E*2F] its cast takes. d_gate_up may be gate_up."""
    arr, E = _splits(m_splits)
    dev = _same_device(dh, gate_up, d_gate_up, row_amax, col_amax)
    rows, F, dp, gp, op, rp, cp = _gated_backward(dh, gate_up, d_gate_up, row_amax, col_amax, E)
    _on(dev, stream, "nvfp4_group_gated_backward", lambda s: lib().nvfp4_group_gated_backward(
        dp, gp, rows, F, arr, E, op, rp, cp, s))


def nvfp4_group_gated_backward_graphsafe(dh: torch.Tensor, gate_up: torch.Tensor, first_dims: Optional[torch.Tensor],
                                         tensor_offsets: Optional[torch.Tensor], d_gate_up: torch.Tensor,
                                         status: torch.Tensor, row_amax: Optional[torch.Tensor] = None,
                                         col_amax: Optional[torch.Tensor] = None, stream=None,
                                         num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    dev = _same_device(dh, gate_up, d_gate_up, row_amax, col_amax, first_dims, tensor_offsets, status)
    rows, F, dp, gp, op, rp, cp = _gated_backward(dh, gate_up, d_gate_up, row_amax, col_amax, E)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E)
    _on(dev, stream, "nvfp4_group_gated_backward_graphsafe", lambda s: lib().nvfp4_group_gated_backward_graphsafe(
        dp, gp, rows, F, fd, to, E, op, rp, cp, st, s))


def nvfp4_adapter_workspace_bytes(rows: int, rank: int) -> int:
    return int(lib().nvfp4_adapter_workspace_bytes(int(rows), int(rank)))


def nvfp4_adapter_gemm(x_bf16: torch.Tensor, x: Dict[str, object], w: Dict[str, object], a: torch.Tensor,
                       b: torch.Tensor, factor: torch.Tensor, ids: torch.Tensor, y: torch.Tensor,
                       workspace: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """y [rows, N] = X W^T + factor[i] (x A_i^T) B_i^T with i = ids[t] (-1: none).
    x_bf16 [rows, K] and its rowwise cast x, w [N, K], a [L, R, K], b [L, N, R],
    factor [L], ids int32 [rows]; workspace from alloc_adapter_workspace."""
    rows, K = x_bf16.shape
    L, R = a.shape[0], a.shape[1]
    N = y.shape[1]
    if y.shape[0] != rows or ids.numel() != rows or factor.numel() != L:
        raise ValueError("y and ids must have a row for each of x_bf16's, factor an entry for each adapter")
    if tuple(a.shape) != (L, R, K) or tuple(b.shape) != (L, N, R):
        raise ValueError("a must be [L, R, K] and b [L, N, R]")
    dt = _out_dtype(y, "y")
    dev = _same_device(y, x_bf16, a, b, factor, ids, workspace, status, *_parts(x, w))
    xm, wm = _matrix(x, rows, rows * K, "x"), _matrix(w, N, N * K, "w")
    wp, wb = _workspace(workspace)
    ptrs = (_dev(x_bf16, torch.bfloat16, "x_bf16"), _dev(a, torch.bfloat16, "a"), _dev(b, torch.bfloat16, "b"),
            _dev(factor, torch.float32, "factor"), _dev(ids, torch.int32, "ids"), _dev(y, y.dtype, "y"),
            _dev(status, torch.int32, "status"))
    xp, ap, bp, fp, ip, yp, st = ptrs
    _on(dev, stream, "nvfp4_adapter_gemm", lambda s: lib().nvfp4_adapter_gemm(
        xp, ctypes.byref(xm), rows, K, ctypes.byref(wm), N, ap, bp, fp, L, R, ip, yp, dt, wp, wb, st, s))


def alloc_adapter_workspace(rows: int, rank: int, device="cuda") -> torch.Tensor:
    """Workspace of nvfp4_adapter_gemm (uint8, uninitialised)."""
    return torch.empty(nvfp4_adapter_workspace_bytes(rows, rank), dtype=torch.uint8, device=device)


# -------------------------------------------------------- buffer helpers

def alloc_amax(rows: int, K: int, E: int, device="cuda"):
    """Uninitialised row_amax [rows] and col_amax [E*K] (fp32)."""
    return (torch.empty(rows, dtype=torch.float32, device=device),
            torch.empty(E * K, dtype=torch.float32, device=device))


def alloc_outputs(rows: int, K: int, E: int, device="cuda", row: bool = True,
                  col: bool = True) -> Dict[str, torch.Tensor]:
    """Uninitialised output buffers of the grouped cast for ``rows`` rows."""
    out: Dict[str, torch.Tensor] = {}
    if row:
        out["row_data"] = torch.empty(rows, K // 2, dtype=torch.uint8, device=device)
        out["row_scale"] = torch.empty(rows, K // 16, dtype=torch.uint8, device=device)
        out["row_s2"] = torch.empty(rows, dtype=torch.float32, device=device)
    if col:
        out["col_data"] = torch.empty(rows * K // 2, dtype=torch.uint8, device=device)
        out["col_scale"] = torch.empty(rows * K // 16, dtype=torch.uint8, device=device)
        out["col_s2"] = torch.empty(E * K, dtype=torch.float32, device=device)
    return out


def alloc_workspace(capacity_rows: int, num_groups: int, device="cuda") -> torch.Tensor:
    """Workspace of the one-launch calls (uint8; its contents need no
    initialisation, the calls zero what they use)."""
    return torch.empty(nvfp4_group_quantize_workspace_bytes(capacity_rows, num_groups),
                       dtype=torch.uint8, device=device)


def routing_tensors(m_splits: Sequence[int], K: int, device="cuda"):
    """Device first_dims [E] and tensor_offsets [E+1] (element offsets) of a
    host split list -- the graph-safe routing format."""
    fd = torch.tensor([int(m) for m in m_splits], dtype=torch.int64)
    offs = torch.zeros(len(m_splits) + 1, dtype=torch.int64)
    offs[1:] = torch.cumsum(fd, 0) * K
    return fd.to(device), offs.to(device)
