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

import array
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


def _ptr(t: Optional[torch.Tensor], dtype: torch.dtype, dev: torch.device, name: str) -> Optional[int]:
    """Device address of a contiguous tensor of ``dtype`` on ``dev``."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _cuda(t: torch.Tensor, name: str) -> torch.device:
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    return dev


def _matrix(m: Dict[str, object], rows: int, elements: int, dev: torch.device, name: str) -> Matrix:
    """``m`` checked to be ``rows`` factors and ``elements`` codes on ``dev``."""
    data, scale, s2 = m["data"], m["scale"], m["s2"]
    if data.numel() * 2 != elements or scale.numel() * 16 != elements or s2.numel() != rows:
        raise ValueError(f"{name} must hold {elements // 2} bytes of codes, {elements // 16} scales and {rows} factors, got "
                         f"{data.numel()}, {scale.numel()} and {s2.numel()}")
    return Matrix(_ptr(data, torch.uint8, dev, name), _ptr(scale, torch.uint8, dev, name),
                  _ptr(s2, torch.float32, dev, name), m.get("scale_layout", NVFP4_SCALE_COMPACT))


def _split_array(m_splits: Sequence[int]):
    """Host array of group sizes (kept alive by the caller during the call)."""
    arr = array.array("q", m_splits)
    return arr, arr.buffer_info()[0], len(arr)


def _run(dev: torch.device, stream: Optional[torch.cuda.Stream], what: str, entry, *args) -> None:
    """``entry(*args, stream)`` with ``dev`` current, on its current stream unless
    one is given."""
    if stream is None:
        s = torch._C._cuda_getCurrentRawStream(dev.index)
    elif stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors on {dev}")
    else:
        s = stream.cuda_stream
    if torch._C._cuda_getDevice() == dev.index:
        rc = entry(*args, s)
    else:
        with torch.cuda.device(dev):
            rc = entry(*args, s)
    if rc != NVFP4_OK:
        raise NVFP4Error(what, rc)


def _out_dtype(t: torch.Tensor, name: str) -> int:
    if t.dtype == torch.float32:
        return NVFP4_OUT_F32
    if t.dtype == torch.bfloat16:
        return NVFP4_OUT_BF16
    raise ValueError(f"{name} must be float32 or bfloat16")


def _width(w: Dict[str, object], x: Dict[str, object], rows: int) -> int:
    """Contraction width of x [rows, K] against stacked weights w."""
    m, n = (x, rows) if rows else (w, w["s2"].numel())
    total = 2 * m["data"].numel()
    if n and total % n:
        raise ValueError(f"{total} codes are not {n} equal rows")
    return total // n if n else 0


def _routing(first_dims: Optional[torch.Tensor], tensor_offsets: Optional[torch.Tensor], status: torch.Tensor, E: int,
             dev: torch.device):
    if tensor_offsets is not None and tensor_offsets.numel() != E + 1:
        raise ValueError(f"tensor_offsets must have {E + 1} entries")
    if status.numel() < 1:
        raise ValueError("status must have an entry")
    return (_ptr(first_dims, torch.int64, dev, "first_dims"), _ptr(tensor_offsets, torch.int64, dev, "tensor_offsets"),
            _ptr(status, torch.int32, dev, "status"))


def _gemm_args(x, w, y: torch.Tensor, E: int):
    dev = _cuda(y, "y")
    rows, N = y.shape
    K = _width(w, x, rows)
    return (dev, rows, N, K, _matrix(x, rows, rows * K, dev, "x"), _matrix(w, E * N, E * N * K, dev, "w"),
            _ptr(y, y.dtype, dev, "y"), _out_dtype(y, "y"))


def nvfp4_group_gemm(x: Dict[str, object], m_splits: Sequence[int], w: Dict[str, object], y: torch.Tensor,
                     stream=None) -> None:
    """y [rows, N] (bf16 or fp32) = X_g W_g^T for each group's rows of x [rows, K]
    and its matrix of w [E*N, K]. Input gradients: x the rowwise cast of dy, w
    the colwise cast of the weights."""
    arr, ap, E = _split_array(m_splits)
    dev, rows, N, K, xm, wm, yp, dt = _gemm_args(x, w, y, E)
    _run(dev, stream, "nvfp4_group_gemm", lib().nvfp4_group_gemm, xm, rows, K, ap, E, wm, N, yp, dt)


def nvfp4_group_gemm_graphsafe(x: Dict[str, object], first_dims: Optional[torch.Tensor],
                               tensor_offsets: Optional[torch.Tensor], w: Dict[str, object], y: torch.Tensor,
                               status: torch.Tensor, stream=None, num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    dev, rows, N, K, xm, wm, yp, dt = _gemm_args(x, w, y, E)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E, dev)
    _run(dev, stream, "nvfp4_group_gemm_graphsafe", lib().nvfp4_group_gemm_graphsafe, xm, rows, K, fd, to, E, wm, N, yp, dt,
         st)


def _gated_args(x, w, h: torch.Tensor, gate_up: Optional[torch.Tensor], E: int):
    dev = _cuda(h, "h")
    rows, F = h.shape
    if gate_up is not None and tuple(gate_up.shape) != (rows, 2 * F):
        raise ValueError("gate_up must be [rows, 2F]")
    K = _width(w, x, rows)
    return (dev, rows, F, K, _matrix(x, rows, rows * K, dev, "x"), _matrix(w, E * 2 * F, E * 2 * F * K, dev, "w"),
            _ptr(h, torch.bfloat16, dev, "h"), _ptr(gate_up, torch.bfloat16, dev, "gate_up"))


def nvfp4_group_gated_gemm(x: Dict[str, object], m_splits: Sequence[int], w: Dict[str, object], h: torch.Tensor,
                           gate_up: Optional[torch.Tensor] = None, stream=None) -> None:
    """h [rows, F] = silu(X_g Wgate_g^T) * (X_g Wup_g^T); w [E*2F, K] holds each
    group's gate rows, then its up rows. gate_up [rows, 2F], if given, takes the
    two projections (bf16) for the gradient."""
    arr, ap, E = _split_array(m_splits)
    dev, rows, F, K, xm, wm, hp, gp = _gated_args(x, w, h, gate_up, E)
    _run(dev, stream, "nvfp4_group_gated_gemm", lib().nvfp4_group_gated_gemm, xm, rows, K, ap, E, wm, F, hp, gp)


def nvfp4_group_gated_gemm_graphsafe(x: Dict[str, object], first_dims: Optional[torch.Tensor],
                                     tensor_offsets: Optional[torch.Tensor], w: Dict[str, object], h: torch.Tensor,
                                     status: torch.Tensor, gate_up: Optional[torch.Tensor] = None, stream=None,
                                     num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    dev, rows, F, K, xm, wm, hp, gp = _gated_args(x, w, h, gate_up, E)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E, dev)
    _run(dev, stream, "nvfp4_group_gated_gemm_graphsafe", lib().nvfp4_group_gated_gemm_graphsafe, xm, rows, K, fd, to, E, wm,
         F, hp, gp, st)


def _wgrad_args(dy, x, dw: torch.Tensor, rows: int, groups: int):
    dev = _cuda(dw, "dw")
    E, N, K = dw.shape
    if E != groups:
        raise ValueError(f"dw must have {groups} matrices")
    return (dev, E, N, K, _matrix(dy, E * N, rows * N, dev, "dy"), _matrix(x, E * K, rows * K, dev, "x"),
            _ptr(dw, dw.dtype, dev, "dw"), _out_dtype(dw, "dw"))


def nvfp4_group_wgrad(dy: Dict[str, object], x: Dict[str, object], m_splits: Sequence[int], dw: torch.Tensor,
                      stream=None) -> None:
    """dw [E, N, K] (bf16 or fp32) = dY_g^T X_g from the colwise casts of dy
    [rows, N] and x [rows, K]; zero for an empty group."""
    arr, ap, groups = _split_array(m_splits)
    rows = sum(arr)
    dev, E, N, K, dm, xm, wp, dt = _wgrad_args(dy, x, dw, rows, groups)
    _run(dev, stream, "nvfp4_group_wgrad", lib().nvfp4_group_wgrad, dm, xm, rows, ap, E, N, K, wp, dt)


def nvfp4_group_wgrad_graphsafe(dy: Dict[str, object], x: Dict[str, object], capacity_rows: int,
                                first_dims: Optional[torch.Tensor], tensor_offsets: Optional[torch.Tensor],
                                dw: torch.Tensor, status: torch.Tensor, stream=None,
                                num_groups: Optional[int] = None) -> None:
    rows = int(capacity_rows)
    dev, E, N, K, dm, xm, wp, dt = _wgrad_args(dy, x, dw, rows, _groups(first_dims, num_groups))
    fd, to, st = _routing(first_dims, tensor_offsets, status, E, dev)
    _run(dev, stream, "nvfp4_group_wgrad_graphsafe", lib().nvfp4_group_wgrad_graphsafe, dm, xm, rows, fd, to, E, N, K, wp, dt,
         st)


def _gated_backward_args(dh, gate_up, d_gate_up, row_amax, col_amax, E: int):
    dev = _cuda(dh, "dh")
    rows, F = dh.shape
    for t, name in ((gate_up, "gate_up"), (d_gate_up, "d_gate_up")):
        if tuple(t.shape) != (rows, 2 * F):
            raise ValueError(f"{name} must be [rows, 2F]")
    for t, n, name in ((row_amax, rows, "row_amax"), (col_amax, E * 2 * F, "col_amax")):
        if t is not None and t.numel() != n:
            raise ValueError(f"{name} must have {n} entries")
    return (dev, rows, F, _ptr(dh, torch.bfloat16, dev, "dh"), _ptr(gate_up, torch.bfloat16, dev, "gate_up"),
            _ptr(d_gate_up, torch.bfloat16, dev, "d_gate_up"), _ptr(row_amax, torch.float32, dev, "row_amax"),
            _ptr(col_amax, torch.float32, dev, "col_amax"))


def nvfp4_group_gated_backward(dh: torch.Tensor, gate_up: torch.Tensor, m_splits: Sequence[int],
                               d_gate_up: torch.Tensor, row_amax: Optional[torch.Tensor] = None,
                               col_amax: Optional[torch.Tensor] = None, stream=None) -> None:
    """d_gate_up [rows, 2F] from dh [rows, F] and the saved gate_up [rows, 2F]
    of nvfp4_group_gated_gemm, with the row amax [rows] and per-group column
    amax [E*2F] its cast takes. d_gate_up may be gate_up."""
    arr, ap, E = _split_array(m_splits)
    dev, rows, F, dp, gp, op, rp, cp = _gated_backward_args(dh, gate_up, d_gate_up, row_amax, col_amax, E)
    _run(dev, stream, "nvfp4_group_gated_backward", lib().nvfp4_group_gated_backward, dp, gp, rows, F, ap, E, op, rp, cp)


def nvfp4_group_gated_backward_graphsafe(dh: torch.Tensor, gate_up: torch.Tensor, first_dims: Optional[torch.Tensor],
                                         tensor_offsets: Optional[torch.Tensor], d_gate_up: torch.Tensor,
                                         status: torch.Tensor, row_amax: Optional[torch.Tensor] = None,
                                         col_amax: Optional[torch.Tensor] = None, stream=None,
                                         num_groups: Optional[int] = None) -> None:
    E = _groups(first_dims, num_groups)
    dev, rows, F, dp, gp, op, rp, cp = _gated_backward_args(dh, gate_up, d_gate_up, row_amax, col_amax, E)
    fd, to, st = _routing(first_dims, tensor_offsets, status, E, dev)
    _run(dev, stream, "nvfp4_group_gated_backward_graphsafe", lib().nvfp4_group_gated_backward_graphsafe, dp, gp, rows, F, fd,
         to, E, op, rp, cp, st)


def nvfp4_adapter_workspace_bytes(rows: int, rank: int) -> int:
    return int(lib().nvfp4_adapter_workspace_bytes(int(rows), int(rank)))


def nvfp4_adapter_gemm(x_bf16: torch.Tensor, x: Dict[str, object], w: Dict[str, object], a: torch.Tensor,
                       b: torch.Tensor, factor: torch.Tensor, ids: torch.Tensor, y: torch.Tensor,
                       workspace: torch.Tensor, status: torch.Tensor, stream=None) -> None:
    """y [rows, N] = X W^T + factor[i] (x A_i^T) B_i^T with i = ids[t] (-1: none).
    x_bf16 [rows, K] and its rowwise cast x, w [N, K], a [L, R, K], b [L, N, R],
    factor [L], ids int32 [rows]; workspace from alloc_adapter_workspace."""
    dev = _cuda(y, "y")
    rows, K = x_bf16.shape
    N, (L, R) = y.shape[1], a.shape[:2]
    if y.shape[0] != rows or ids.numel() != rows or factor.numel() != L or status.numel() < 1:
        raise ValueError("y and ids must have a row for each of x_bf16's, factor an entry for each adapter")
    if a.shape[2] != K or tuple(b.shape) != (L, N, R):
        raise ValueError("a must be [L, R, K] and b [L, N, R]")
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and on {dev}")
    _run(dev, stream, "nvfp4_adapter_gemm", lib().nvfp4_adapter_gemm, _ptr(x_bf16, torch.bfloat16, dev, "x_bf16"),
         _matrix(x, rows, rows * K, dev, "x"), rows, K, _matrix(w, N, N * K, dev, "w"), N,
         _ptr(a, torch.bfloat16, dev, "a"), _ptr(b, torch.bfloat16, dev, "b"), _ptr(factor, torch.float32, dev, "factor"),
         L, R, _ptr(ids, torch.int32, dev, "ids"), _ptr(y, y.dtype, dev, "y"), _out_dtype(y, "y"),
         workspace.data_ptr(), workspace.numel() * workspace.element_size(), _ptr(status, torch.int32, dev, "status"))


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
