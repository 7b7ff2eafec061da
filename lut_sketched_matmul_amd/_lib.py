"""ctypes binding of ``libsketchmm.so`` (the C ABI in ``include/sketch_matmul.h``).

Argument marshalling only: every step of the sketched matmul runs in the HIP
library. PyTorch provides device memory (``tensor.data_ptr()``) and the
current HIP stream; nothing here computes on the host, and there is no
fallback: when the library is missing or its call fails, an exception is
raised.
"""
from __future__ import annotations

import ctypes
import os
import re
from typing import Optional, Tuple

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB_PATH = os.path.join(PKG, "libsketchmm.so")
HEADER = os.path.join(ROOT, "include", "sketch_matmul.h")

SKM_F32, SKM_F16, SKM_BF16 = 0, 1, 2
STATUS = {
    0: "SKM_OK", -1: "SKM_EINVAL", -2: "SKM_EUNSUPPORTED", -3: "SKM_EALIGN",
    -4: "SKM_EWORKSPACE", -5: "SKM_EHIP", -6: "SKM_EALIAS",
}


class SketchError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({text})")
        self.status = status


_lib = None

_c_i64 = ctypes.c_int64
_c_int = ctypes.c_int
_c_vp = ctypes.c_void_p
_c_size = ctypes.c_size_t
_c_f32 = ctypes.c_float

_SIGNATURES = {
    "sketch_matmul_fwd": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int,
                                   _c_vp, _c_vp, _c_size, _c_vp]),
    "sketch_matmul_fwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int]),
    "sketch_matmul_fwd_multi": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_i64, _c_i64, _c_i64,
                                         _c_int, _c_int, _c_vp, _c_vp]),
    "sketch_matmul_bwd": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int, _c_int,
                                   _c_vp, _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_matmul_bwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int]),
    "sketch_matmul_bwd_noalloc": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64, _c_int,
                                           _c_int, _c_vp, _c_vp, _c_int, _c_vp]),
    "sketch_dequant": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_vp]),
    "sketch_unpack_indices": (_c_int, [_c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_vp]),
    "sketch_lut_adam_step": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_i64, _c_i64, _c_f32, _c_f32,
                                      _c_f32, _c_f32, _c_f32, _c_f32, _c_vp]),
    "sketch_lut_sgd_step": (_c_int, [_c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_i64, _c_f32, _c_f32, _c_f32, _c_f32,
                                     _c_vp]),
    "sketch_column_weights": (_c_int, [_c_vp, _c_i64, _c_vp, _c_vp]),
    "sketch_lloyd": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_vp, _c_int, _c_vp]),
    "sketch_map_workspace": (_c_size, [_c_i64]),
    "sketch_map": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_size,
                            _c_vp]),
    "sketch_hessian_factor_workspace": (_c_size, [_c_i64]),
    "sketch_hessian_factor": (_c_int, [_c_vp, _c_i64, ctypes.c_double, _c_vp, _c_vp, _c_size, _c_vp]),
    "sketch_act_quant": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "sketch_act_dequant": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_int, _c_vp]),
    "sketch_matmul_bwd_ckpt": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_i64,
                                        _c_int, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_matmul_bwd_ckpt_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int,
                                                   _c_int]),
    "sketch_norm_fwd": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64, _c_i64, _c_int, _c_f32, _c_vp, _c_vp,
                                 _c_vp, _c_vp, _c_vp, _c_vp]),
    "sketch_norm_bwd": (_c_int, [_c_vp, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_vp, _c_i64,
                                 _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_norm_bwd_workspace": (_c_size, [_c_i64, _c_i64]),
    "sketch_xent_fwd": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_i64, _c_i64, _c_i64, _c_i64, _c_int,
                                 _c_int, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "sketch_xent_fwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int]),
    "sketch_xent_mean": (_c_int, [_c_vp, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp, _c_vp]),
    "sketch_xent_bwd": (_c_int, [_c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_i64, _c_vp, _c_vp, _c_i64, _c_i64,
                                 _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_xent_bwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "sketch_dropout": (_c_int, [_c_vp, _c_int, _c_vp, _c_i64, ctypes.c_double, _c_vp, _c_vp, _c_vp]),
    "sketch_adapter_fwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_vp, _c_vp, ctypes.c_double, _c_vp,
                                    _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "sketch_adapter_fwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int]),
    "sketch_adapter_bwd": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_int, _c_vp, _c_int, _c_vp, _c_vp,
                                    ctypes.c_double, _c_vp, _c_i64, _c_i64, _c_i64, _c_int, _c_vp, _c_vp, _c_vp,
                                    _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_adapter_bwd_workspace": (_c_size, [_c_i64, _c_i64, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_int,
                                               _c_int]),
    "sketch_rotary_fwd": (_c_int, [_c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_vp, _c_vp,
                                   _c_i64, _c_int, _c_int, _c_int, _c_int, _c_f32, _c_vp, _c_i64, _c_vp, _c_i64,
                                   _c_vp]),
    "sketch_rotary_bwd": (_c_int, [_c_vp, _c_i64, _c_int, _c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_i64, _c_vp, _c_i64,
                                   _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_int, _c_int, _c_int, _c_int, _c_f32, _c_vp,
                                   _c_i64, _c_vp, _c_i64, _c_vp, _c_vp, _c_int, _c_vp, _c_size, _c_vp]),
    "sketch_rotary_bwd_workspace": (_c_size, [_c_int]),
    "sketch_status_str": (ctypes.c_char_p, [_c_int]),
    "sketch_version": (_c_int, []),
}


def library_path() -> str:
    return os.environ.get("SKETCHMM_LIB", LIB_PATH)


def lib() -> ctypes.CDLL:
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} not found: build it with `python -m lut_sketched_matmul_amd.build`")
        handle = ctypes.CDLL(path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def header_functions() -> list:
    """Names of the functions declared in include/sketch_matmul.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sketch_\w+)\s*\(", text)))


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise SketchError(fn, status, lib().sketch_status_str(status).decode())


# --------------------------------------------------------------------------
# torch-facing wrappers
# --------------------------------------------------------------------------

_torch_module = None
_dtype_codes = {}


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _dtype_codes.update({torch.float32: SKM_F32, torch.float16: SKM_F16, torch.bfloat16: SKM_BF16})
        _torch_module = torch
    return _torch_module


def dtype_code(t) -> int:
    _torch()
    code = _dtype_codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _stream_ptr(stream) -> int:
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _require_device(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


# The C ABI takes raw pointers and sizes, so it cannot see a tensor's extent:
# every tensor's shape (or element count) and dtype is checked against the
# sizes passed with it before the call, so that a wrong buffer is an exception
# here and never an out-of-bounds access on the device.

_FLOAT_DTYPES = ("float32", "float16", "bfloat16")


_dtype_names = {}


def _dtype_name(t) -> str:
    name = _dtype_names.get(t.dtype)
    if name is None:
        name = _dtype_names[t.dtype] = str(t.dtype).replace("torch.", "")
    return name


def _expect(t, name: str, shape=None, numel=None, dtypes=None):
    if t is None:
        return
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")
    if dtypes is not None and _dtype_name(t) not in dtypes:
        raise TypeError(f"{name} has dtype {_dtype_name(t)}, expected one of {dtypes}")


def _check_bits(b: int, d: int):
    if b not in (2, 3, 4):
        raise ValueError(f"bit width b = {b}: supported are 2, 3 and 4")
    if d < 0 or (d * b) % 8:
        raise ValueError(f"d = {d} columns of {b} bits do not fill whole bytes")


def _check_sketch(idx_packed, lut, n: int, d: int, b: int, gpr: int, n_sets=None, lut_name="lut"):
    """idx_packed [n, d*b/8] uint8 and tables of n (x n_sets) rows of gpr groups of 2^b entries."""
    _check_bits(b, d)
    if gpr < 1:
        raise ValueError(f"gpr = {gpr} must be at least 1")
    _expect(idx_packed, "idx_packed", shape=(n, d * b // 8), dtypes=("uint8",))
    count = n * gpr * (1 << b) * (1 if n_sets is None else n_sets)
    _expect(lut, lut_name, numel=count, dtypes=_FLOAT_DTYPES)
    if n_sets is not None and (lut.dim() < 1 or lut.shape[0] != n_sets):
        raise ValueError(f"{lut_name} must have the table sets as its first dimension")


def _matrix(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got {t.dim()} dimensions")
    return t.shape


def _gradient(out, shape, accumulate: bool, device):
    """The fp32 output a call writes, or adds to: `out`, else a new one (of zeros when there is to be added)."""
    if out is not None:
        return out
    torch = _torch()
    return (torch.zeros if accumulate else torch.empty)(shape, dtype=torch.float32, device=device)


def sketch_matmul_fwd_workspace(m: int, n: int, d: int, b: int, gpr: int, x_dtype: int, lut_dtype: int) -> int:
    """Bytes of device workspace sketch_matmul_fwd needs for these sizes and dtypes."""
    return int(lib().sketch_matmul_fwd_workspace(m, n, d, b, gpr, x_dtype, lut_dtype))


def _workspace(ws, need: int, device):
    """The caller's workspace (checked), or a new one of `need` bytes, or None."""
    torch = _torch()
    if ws is not None:
        if ws.numel() * ws.element_size() < need:
            raise ValueError(f"workspace of {ws.numel() * ws.element_size()} bytes, {need} needed")
        return ws
    return torch.empty(need, dtype=torch.uint8, device=device) if need else None


def sketch_matmul_fwd(X, idx_packed, lut, b: int, gpr: int, out=None, workspace=None, stream=None):
    """Y = X W^T with W[i, j] = lut[i, j // (d/gpr), idx[i, j]].

    X [m, d] (f32/f16/bf16), idx_packed [n, d*b/8] uint8, lut [n, gpr, 2^b].
    Returns Y [m, n] in X's dtype. workspace: optional uint8 device buffer of
    at least sketch_matmul_fwd_workspace(...) bytes (allocated here when
    needed and omitted).
    """
    torch = _torch()
    m, d = _matrix(X, "X")
    n = idx_packed.shape[0]
    _expect(X, "X", dtypes=_FLOAT_DTYPES)
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _expect(out, "out", shape=(m, n), dtypes=(_dtype_name(X),))
    _expect(workspace, "workspace", dtypes=("uint8",))
    _require_device(X, idx_packed, lut, out, workspace)
    if out is None:
        out = torch.empty((m, n), dtype=X.dtype, device=X.device)
    ws = _workspace(workspace, sketch_matmul_fwd_workspace(m, n, d, b, gpr, dtype_code(X), dtype_code(lut)),
                    X.device)
    st = lib().sketch_matmul_fwd(X.data_ptr(), dtype_code(X), idx_packed.data_ptr(), lut.data_ptr(),
                                 dtype_code(lut), m, n, d, b, gpr, out.data_ptr() if out.numel() else None,
                                 ws.data_ptr() if ws is not None else None, ws.numel() if ws is not None else 0,
                                 _stream_ptr(stream))
    _check("sketch_matmul_fwd", st)
    return out


def sketch_matmul_fwd_multi(X, idx_packed, luts, lut_set, b: int, gpr: int, out=None, stream=None):
    """Y[t] = X[t] W_{lut_set[t]}^T: one table set per token over shared indices.

    X [m, d] (f16/bf16, m <= 16), idx_packed [n, d*b/8] uint8, luts [n_sets, n,
    gpr, 2^b], lut_set [m] int32 (device). Returns Y [m, n] in X's dtype.
    """
    torch = _torch()
    m, d = _matrix(X, "X")
    n = idx_packed.shape[0]
    _expect(X, "X", dtypes=_FLOAT_DTYPES)
    if luts.dim() < 1:
        raise ValueError("luts must have the table sets as its first dimension")
    _check_sketch(idx_packed, luts, n, d, b, gpr, n_sets=luts.shape[0], lut_name="luts")
    if lut_set.dtype != torch.int32 or lut_set.numel() != m:
        raise ValueError("lut_set must be an int32 tensor with one entry per token")
    _expect(out, "out", shape=(m, n), dtypes=(_dtype_name(X),))
    _require_device(X, idx_packed, luts, lut_set, out)
    if out is None:
        out = torch.empty((m, n), dtype=X.dtype, device=X.device)
    st = lib().sketch_matmul_fwd_multi(X.data_ptr(), dtype_code(X), idx_packed.data_ptr(), luts.data_ptr(),
                                       dtype_code(luts), lut_set.data_ptr() if m else None, luts.shape[0], m, n, d,
                                       b, gpr, out.data_ptr() if out.numel() else None, _stream_ptr(stream))
    _check("sketch_matmul_fwd_multi", st)
    return out


def sketch_matmul_bwd_workspace(m: int, n: int, d: int, b: int, gpr: int, io_dtype: int, lut_dtype: int) -> int:
    """Bytes of device workspace sketch_matmul_bwd needs for these sizes and dtypes."""
    return int(lib().sketch_matmul_bwd_workspace(m, n, d, b, gpr, io_dtype, lut_dtype))


def sketch_matmul_bwd(dY, X, idx_packed, lut, b: int, gpr: int, d: Optional[int] = None,
                      need_dx: bool = True, need_dlut: bool = True, dlut_out=None, accumulate: bool = False,
                      workspace=None, stream=None) -> Tuple[object, object]:
    """(dX, dLUT) of the sketched matmul; both fp32. dLUT sums shared entries.

    dY [m, n], X [m, d] in the same dtype (X may be None when need_dlut is
    False; then d must be given), idx_packed [n, d*b/8] uint8, lut [n, gpr,
    2^b]. dlut_out: optional fp32 [n, gpr, 2^b] to write (accumulate=True adds
    to it). workspace: optional uint8 device buffer of at least
    sketch_matmul_bwd_workspace(...) bytes (allocated here when omitted).
    """
    torch = _torch()
    m, n = _matrix(dY, "dY")
    _expect(dY, "dY", dtypes=_FLOAT_DTYPES)
    if X is not None:
        mx, dx_cols = _matrix(X, "X")
        if d is not None and d != dx_cols:
            raise ValueError(f"d = {d} does not match X's {dx_cols} columns")
        d = dx_cols
        _expect(X, "X", shape=(m, d), dtypes=(_dtype_name(dY),))
    elif need_dlut:
        raise ValueError("the table gradient needs X")
    if d is None:
        raise ValueError("d must be given when X is None")
    K = 1 << b
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _expect(dlut_out, "dlut_out", shape=(n, gpr, K), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    _require_device(dY, X, idx_packed, lut, dlut_out, workspace)
    dX = torch.empty((m, d), dtype=torch.float32, device=dY.device) if need_dx else None
    dL = None
    if need_dlut:
        with torch.cuda.stream(stream):  # (where a new output's zeros have to be written)
            dL = _gradient(dlut_out, (n, gpr, K), accumulate, dY.device)
    workspace = _workspace(workspace, sketch_matmul_bwd_workspace(m, n, d, b, gpr, dtype_code(dY), dtype_code(lut)),
                           dY.device)
    st = lib().sketch_matmul_bwd(
        dY.data_ptr() if dY.numel() else None, X.data_ptr() if (X is not None and X.numel()) else None,
        dtype_code(dY), idx_packed.data_ptr(), lut.data_ptr(), dtype_code(lut), m, n, d, b, gpr,
        dX.data_ptr() if (dX is not None and dX.numel()) else None, dL.data_ptr() if dL is not None else None,
        1 if accumulate else 0, workspace.data_ptr() if workspace is not None else None,
        workspace.numel() if workspace is not None else 0, _stream_ptr(stream))
    _check("sketch_matmul_bwd", st)
    return dX, dL


def sketch_matmul_bwd_noalloc(dY, X, idx_packed, lut, b: int, gpr: int, dx_out=None, dlut_out=None,
                              accumulate: bool = False, stream=None) -> None:
    """The backward pass into caller-given outputs with the library's own scratch (no allocation at all).

    dY [m, n], X [m, d] in the same dtype, idx_packed [n, d*b/8] uint8, lut [n, gpr, 2^b]; dx_out fp32
    [m, d] and dlut_out fp32 [n, gpr, 2^b] are written when given (at least one of them). Nothing is
    allocated here or in the library; calls that overlap in time on one GPU race on its scratch.
    """
    m, n = _matrix(dY, "dY")
    mx, d = _matrix(X, "X")
    _expect(dY, "dY", dtypes=_FLOAT_DTYPES)
    _expect(X, "X", shape=(m, d), dtypes=(_dtype_name(dY),))
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _expect(dx_out, "dx_out", shape=(m, d), dtypes=("float32",))
    _expect(dlut_out, "dlut_out", shape=(n, gpr, 1 << b), dtypes=("float32",))
    if dx_out is None and dlut_out is None:
        raise ValueError("give dx_out, dlut_out or both")
    _require_device(dY, X, idx_packed, lut, dx_out, dlut_out)
    st = lib().sketch_matmul_bwd_noalloc(
        dY.data_ptr() if dY.numel() else None, X.data_ptr() if X.numel() else None, dtype_code(dY),
        idx_packed.data_ptr(), lut.data_ptr(), dtype_code(lut), m, n, d, b, gpr,
        dx_out.data_ptr() if (dx_out is not None and dx_out.numel()) else None,
        dlut_out.data_ptr() if dlut_out is not None else None, 1 if accumulate else 0, _stream_ptr(stream))
    _check("sketch_matmul_bwd_noalloc", st)


def sketch_dequant(idx_packed, lut, d: int, b: int, gpr: int, stream=None):
    """Dense W [n, d] in the table dtype (a checking aid)."""
    torch = _torch()
    n = idx_packed.shape[0]
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _require_device(idx_packed, lut)
    W = torch.empty((n, d), dtype=lut.dtype, device=lut.device)
    st = lib().sketch_dequant(idx_packed.data_ptr(), lut.data_ptr(), dtype_code(lut), n, d, b, gpr, W.data_ptr(),
                              _stream_ptr(stream))
    _check("sketch_dequant", st)
    return W


def sketch_unpack_indices(idx_packed, d: int, b: int, stream=None):
    """One uint8 per weight: idx [n, d] (a checking aid)."""
    torch = _torch()
    n = idx_packed.shape[0]
    _check_bits(b, d)
    _expect(idx_packed, "idx_packed", shape=(n, d * b // 8), dtypes=("uint8",))
    _require_device(idx_packed)
    out = torch.empty((n, d), dtype=torch.uint8, device=idx_packed.device)
    st = lib().sketch_unpack_indices(idx_packed.data_ptr(), n, d, b, out.data_ptr(), _stream_ptr(stream))
    _check("sketch_unpack_indices", st)
    return out


def _copy_args(lut):
    """(pointer, dtype code) of an optional 16-bit compute copy."""
    if lut is None:
        return None, SKM_F16
    return lut.data_ptr(), dtype_code(lut)


def _check_f32(*ts):
    torch = _torch()
    for t in ts:
        if t is not None and t.dtype != torch.float32:
            raise TypeError("master tables, gradients and optimizer state are fp32")


def sketch_lut_adam_step(master, grad, exp_avg, exp_avg_sq, step: int, lr: float, beta1: float = 0.9,
                         beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.0,
                         grad_scale: float = 1.0, lut=None, stream=None) -> None:
    """One fused Adam(W) step on fp32 master tables; writes the 16-bit copy `lut` if given."""
    _require_device(master, grad, exp_avg, exp_avg_sq, lut)
    _check_f32(master, grad, exp_avg, exp_avg_sq)
    count = master.numel()
    for t in (grad, exp_avg, exp_avg_sq, lut):
        if t is not None and t.numel() != count:
            raise ValueError("all buffers must have the master's number of entries")
    lp, ldt = _copy_args(lut)
    st = lib().sketch_lut_adam_step(master.data_ptr(), lp, ldt, grad.data_ptr(), exp_avg.data_ptr(),
                                    exp_avg_sq.data_ptr(), count, step, lr, beta1, beta2, eps, weight_decay,
                                    grad_scale, _stream_ptr(stream))
    _check("sketch_lut_adam_step", st)


def sketch_lut_sgd_step(master, grad, lr: float, momentum: float = 0.0, weight_decay: float = 0.0,
                        grad_scale: float = 1.0, momentum_buf=None, lut=None, stream=None) -> None:
    """One fused SGD step on fp32 master tables; writes the 16-bit copy `lut` if given."""
    _require_device(master, grad, momentum_buf, lut)
    _check_f32(master, grad, momentum_buf)
    count = master.numel()
    for t in (grad, momentum_buf, lut):
        if t is not None and t.numel() != count:
            raise ValueError("all buffers must have the master's number of entries")
    lp, ldt = _copy_args(lut)
    st = lib().sketch_lut_sgd_step(master.data_ptr(), lp, ldt, grad.data_ptr(),
                                   momentum_buf.data_ptr() if momentum_buf is not None else None, count, lr,
                                   momentum, weight_decay, grad_scale, _stream_ptr(stream))
    _check("sketch_lut_sgd_step", st)


def sketch_column_weights(U, stream=None):
    """h[j] = 1 / [H^-1]_jj from the upper factor U (H^-1 = U^T U), fp32 [d]."""
    torch = _torch()
    d = U.shape[0]
    _expect(U, "U", shape=(d, d))
    _check_f32(U)
    _require_device(U)
    h = torch.empty(d, dtype=torch.float32, device=U.device)
    _check("sketch_column_weights", lib().sketch_column_weights(U.data_ptr(), d, h.data_ptr(), _stream_ptr(stream)))
    return h


def sketch_lloyd(W, h, b: int, gpr: int, iters: int, lut_dtype=None, out=None, stream=None):
    """Weighted Lloyd tables [n, gpr, 2^b] (fp32 unless lut_dtype / out say otherwise)."""
    torch = _torch()
    n, d = _matrix(W, "W")
    _check_f32(W, h)
    _check_bits(b, d)
    _expect(h, "h", numel=d)
    _expect(out, "out", numel=n * gpr * (1 << b), dtypes=_FLOAT_DTYPES)
    _require_device(W, h, out)
    if out is None:
        out = torch.empty((n, gpr, 1 << b), dtype=lut_dtype or torch.float32, device=W.device)
    st = lib().sketch_lloyd(W.data_ptr(), h.data_ptr(), n, d, b, gpr, iters, out.data_ptr(), dtype_code(out),
                            _stream_ptr(stream))
    _check("sketch_lloyd", st)
    return out


def sketch_map(W_work, U, lut, b: int, gpr: int, out=None, workspace=None, stream=None):
    """Error-compensated mapping -> idx_packed [n, d*b/8] uint8. W_work (fp32 [n, d]) is overwritten."""
    torch = _torch()
    n, d = _matrix(W_work, "W_work")
    _check_f32(W_work, U)
    _expect(U, "U", shape=(d, d))
    _check_sketch(out, lut, n, d, b, gpr)
    _require_device(W_work, U, lut, out, workspace)
    if out is None:
        out = torch.empty((n, d * b // 8), dtype=torch.uint8, device=W_work.device)
    ws = lib().sketch_map_workspace(n)
    if workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=W_work.device)
    st = lib().sketch_map(W_work.data_ptr(), U.data_ptr(), lut.data_ptr(), dtype_code(lut), n, d, b, gpr,
                          out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                          _stream_ptr(stream))
    _check("sketch_map", st)
    return out


def sketch_hessian_factor(H, damp: float = 0.01, out=None, workspace=None, stream=None):
    """U [d, d] fp32, upper triangular, with U^T U = (H + damp * mean(diag H) * I)^-1, from the float64 Gram
    matrix H [d, d] of the sample inputs (only its entries with i <= j are read)."""
    torch = _torch()
    d, d2 = _matrix(H, "H")
    if d != d2:
        raise ValueError(f"H must be square, got {tuple(H.shape)}")
    _expect(H, "H", dtypes=("float64",))
    _expect(out, "out", shape=(d, d), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    _require_device(H, out, workspace)
    if out is None:
        out = torch.empty((d, d), dtype=torch.float32, device=H.device)
    ws = _workspace(workspace, lib().sketch_hessian_factor_workspace(d), H.device)
    st = lib().sketch_hessian_factor(H.data_ptr(), d, float(damp), out.data_ptr(),
                                     ws.data_ptr() if ws is not None else None,
                                     ws.numel() if ws is not None else 0, _stream_ptr(stream))
    _check("sketch_hessian_factor", st)
    return out


# --------------------------------------------------------------------------
# 8-bit activation checkpoints, norms
# --------------------------------------------------------------------------

def _enter(stream, first, *others):
    """(raw stream, context): makes the tensors' device and the stream a call runs on current.

    The tensors must live on one GPU and be contiguous. `stream` (None = the device's current stream) becomes
    current too, so that outputs and workspaces allocated before :func:`_leave` belong to the stream that uses
    them; ordering the inputs before it is the caller's. The context is None when nothing had to change.
    """
    torch = _torch()
    index = first.get_device()
    for t in (first, *others):
        if t is not None:
            if not t.is_cuda:
                raise ValueError("tensors must live on the GPU")
            if not t.is_contiguous():
                raise ValueError("tensors must be contiguous")
            if t.get_device() != index:
                raise ValueError(f"tensors on cuda:{index} and cuda:{t.get_device()}")
    context = None
    if stream is not None:
        if stream.device_index != index:
            raise ValueError(f"a stream of cuda:{stream.device_index} for tensors on cuda:{index}")
        context = torch.cuda.stream(stream)
    elif torch._C._cuda_getDevice() != index:
        context = torch.cuda.device(index)
    if context is not None:
        context.__enter__()
    # (the raw handle: building a Stream object costs as much as half a launch)
    return torch._C._cuda_getCurrentRawStream(index), context


def _leave(context):
    if context is not None:
        context.__exit__(None, None, None)


def _ptr(t):
    """The tensor's address (None for no tensor; an empty one's is null too)."""
    return None if t is None else t.data_ptr()


def _size(t) -> int:
    return t.numel() * t.element_size() if t is not None else 0


def _check_ckpt(codes, scales, m: int, d: int):
    _expect(codes, "codes", shape=(m, d), dtypes=("int8",))
    _expect(scales, "scales", shape=(m, d // 32), dtypes=("uint8",))


def sketch_act_quant(X, codes=None, scales=None, stream=None) -> Tuple[object, object]:
    """The 8-bit checkpoint of X [m, d] (f32/f16/bf16, d % 32 == 0): (codes int8 [m, d], scales uint8 [m, d/32]).

    value = codes * 2^(scales - 127), one exponent per 32 columns; a block with an infinity or NaN reads back
    as NaN. codes / scales: optional outputs.
    """
    torch = _torch()
    m, d = _matrix(X, "X")
    if d < 32 or d % 32:
        raise ValueError(f"X has {d} columns: a checkpoint takes whole blocks of 32")
    _check_ckpt(codes, scales, m, d)
    sp, context = _enter(stream, X, codes, scales)
    try:
        if codes is None:
            codes = X.new_empty((m, d), dtype=torch.int8)
        if scales is None:
            scales = X.new_empty((m, d // 32), dtype=torch.uint8)
        st = lib().sketch_act_quant(_ptr(X), dtype_code(X), m, d, _ptr(codes), _ptr(scales), sp)
    finally:
        _leave(context)
    _check("sketch_act_quant", st)
    return codes, scales


def sketch_act_dequant(codes, scales, dtype, out=None, stream=None):
    """X [m, d] in `dtype` from its checkpoint (exact in the dtype that was quantised)."""
    torch = _torch()
    m, d = _matrix(codes, "codes")
    if d < 32 or d % 32:
        raise ValueError(f"codes has {d} columns: a checkpoint takes whole blocks of 32")
    _check_ckpt(codes, scales, m, d)
    if out is None and dtype not in (torch.float32, torch.float16, torch.bfloat16):
        raise TypeError(f"unsupported dtype {dtype}")
    _expect(out, "out", shape=(m, d), dtypes=(str(dtype).replace("torch.", ""),))
    sp, context = _enter(stream, codes, scales, out)
    try:
        if out is None:
            out = codes.new_empty((m, d), dtype=dtype)
        st = lib().sketch_act_dequant(_ptr(codes), _ptr(scales), m, d, _ptr(out), dtype_code(out), sp)
    finally:
        _leave(context)
    _check("sketch_act_dequant", st)
    return out


def sketch_matmul_bwd_ckpt_workspace(m: int, n: int, d: int, b: int, gpr: int, io_dtype: int, lut_dtype: int,
                                     need_dx: bool = True, need_dlut: bool = True) -> int:
    """Bytes of device workspace sketch_matmul_bwd_ckpt needs for these sizes and dtypes."""
    return int(lib().sketch_matmul_bwd_ckpt_workspace(m, n, d, b, gpr, io_dtype, lut_dtype, 1 if need_dx else 0,
                                                      1 if need_dlut else 0))


def sketch_matmul_bwd_ckpt(dY, codes, scales, idx_packed, lut, b: int, gpr: int, need_dx: bool = True,
                           need_dlut: bool = True, dlut_out=None, accumulate: bool = False, workspace=None,
                           stream=None) -> Tuple[object, object]:
    """(dX, dLUT) of the sketched matmul, both fp32, with X given as its 8-bit checkpoint.

    dY [m, n] (its dtype is the activations'), codes [m, d] int8 and scales [m, d/32] uint8 of
    sketch_act_quant or sketch_norm_fwd; the rest as for sketch_matmul_bwd.
    """
    torch = _torch()
    m, n = _matrix(dY, "dY")
    _, d = _matrix(codes, "codes")
    _expect(dY, "dY", dtypes=_FLOAT_DTYPES)
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _check_ckpt(codes, scales, m, d)
    K = 1 << b
    _expect(dlut_out, "dlut_out", shape=(n, gpr, K), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    io, lt = dtype_code(dY), dtype_code(lut)
    sp, context = _enter(stream, dY, codes, scales, idx_packed, lut, dlut_out, workspace)
    try:
        dX = torch.empty((m, d), dtype=torch.float32, device=dY.device) if need_dx else None
        dL = None
        if need_dlut:
            dL = _gradient(dlut_out, (n, gpr, K), accumulate, dY.device)
        ws = _workspace(workspace, sketch_matmul_bwd_ckpt_workspace(m, n, d, b, gpr, io, lt, need_dx, need_dlut),
                        dY.device)
        st = lib().sketch_matmul_bwd_ckpt(_ptr(dY), _ptr(codes), _ptr(scales), io, idx_packed.data_ptr(),
                                          lut.data_ptr(), lt, m, n, d, b, gpr, _ptr(dX), _ptr(dL),
                                          1 if accumulate else 0, _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_matmul_bwd_ckpt", st)
    return dX, dL


_NORM_KINDS = {"rms": 0, "layer": 1}


def _norm_kind(kind: str) -> int:
    if kind not in _NORM_KINDS:
        raise ValueError(f"kind = {kind!r}: supported are 'layer' and 'rms'")
    return _NORM_KINDS[kind]


def _check_params(xt, d: int, *named):
    """weight / bias of a norm: [d], fp32 or the activations' dtype xt, one dtype for both. Returns its code."""
    code = SKM_F32
    first = None
    for name, t in named:
        if t is None:
            continue
        _expect(t, name, shape=(d,), dtypes=None if t.dtype == xt else ("float32", str(xt).replace("torch.", "")))
        if first is not None and t.dtype != first:
            raise TypeError("weight and bias must have one dtype")
        first = t.dtype
        code = dtype_code(t)
    return code


def sketch_norm_fwd(X, weight=None, bias=None, kind: str = "layer", eps: float = 1e-5, checkpoint: bool = False,
                    out=None, stream=None):
    """(Y, mean, rstd, codes, scales): layer norm or rms norm of the rows of X [m, d].

    Y = (x - mean) rstd weight + bias in X's dtype (f32/f16/bf16); mean (None for kind "rms") and rstd fp32 [m].
    weight / bias: [d] fp32 or X's dtype, None = ones / zeros. checkpoint: also write the 8-bit checkpoint of Y
    in the same pass (d % 32 == 0), else codes and scales are None.
    """
    torch = _torch()
    m, d = _matrix(X, "X")
    k = _norm_kind(kind)
    _expect(X, "X", dtypes=_FLOAT_DTYPES)
    pc = _check_params(X.dtype, d, ("weight", weight), ("bias", bias))
    if checkpoint and d % 32:
        raise ValueError(f"X has {d} columns: a checkpoint takes whole blocks of 32")
    _expect(out, "out", shape=(m, d), dtypes=(_dtype_name(X),))
    sp, context = _enter(stream, X, weight, bias, out)
    try:
        if out is None:
            out = torch.empty_like(X)
        mean = X.new_empty(m, dtype=torch.float32) if k else None
        rstd = X.new_empty(m, dtype=torch.float32)
        codes = scales = None
        if checkpoint:
            codes = X.new_empty((m, d), dtype=torch.int8)
            scales = X.new_empty((m, d // 32), dtype=torch.uint8)
        st = lib().sketch_norm_fwd(_ptr(X), dtype_code(X), _ptr(weight), _ptr(bias), pc, m, d, k, eps, _ptr(out),
                                   _ptr(mean), _ptr(rstd), _ptr(codes), _ptr(scales), sp)
    finally:
        _leave(context)
    _check("sketch_norm_fwd", st)
    return out, mean, rstd, codes, scales


def sketch_norm_bwd_workspace(m: int, d: int) -> int:
    """Bytes of device workspace sketch_norm_bwd needs for dweight / dbias of these sizes."""
    return int(lib().sketch_norm_bwd_workspace(m, d))


def sketch_norm_bwd(dY, X, weight, mean, rstd, kind: str = "layer", need_dx: bool = True, need_dw: bool = True,
                    need_db: bool = True, dw_out=None, db_out=None, accumulate: bool = False, x_dtype=None,
                    workspace=None, stream=None):
    """(dX, dweight, dbias) of sketch_norm_fwd; None where not asked for.

    X: the forward's input [m, d], or its 8-bit checkpoint as a pair (codes, scales), then x_dtype is the
    activations' dtype (dY's if omitted). dY [m, d] fp32 or the activations' dtype; dX in the activations'
    dtype, dweight and dbias fp32 [d] (dw_out / db_out: optional outputs, accumulate=True adds to them). mean
    is None for kind "rms". workspace: optional uint8 buffer of sketch_norm_bwd_workspace(m, d) bytes.
    """
    torch = _torch()
    k = _norm_kind(kind)
    m, d = _matrix(dY, "dY")
    codes = scales = None
    if isinstance(X, (tuple, list)):
        codes, scales = X
        X = None
        if d % 32:
            raise ValueError(f"dY has {d} columns: a checkpoint takes whole blocks of 32")
        _check_ckpt(codes, scales, m, d)
        xt = x_dtype if x_dtype is not None else dY.dtype
    else:
        _expect(X, "X", shape=(m, d))
        xt = X.dtype
        if x_dtype is not None and x_dtype != xt:
            raise TypeError(f"X has dtype {xt}, expected {x_dtype}")
    xc = _dtype_codes.get(xt)
    if xc is None:
        raise TypeError(f"X has dtype {xt}, expected one of {_FLOAT_DTYPES}")
    if dY.dtype != xt:
        _expect(dY, "dY", dtypes=("float32", str(xt).replace("torch.", "")))
    pc = _check_params(xt, d, ("weight", weight))
    if k and mean is None:
        raise ValueError("a layer norm's backward needs the mean")
    if not k:
        mean = None
    _expect(mean, "mean", shape=(m,), dtypes=("float32",))
    _expect(rstd, "rstd", shape=(m,), dtypes=("float32",))
    _expect(dw_out, "dw_out", shape=(d,), dtypes=("float32",))
    _expect(db_out, "db_out", shape=(d,), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    sp, context = _enter(stream, dY, X, codes, scales, weight, mean, rstd, dw_out, db_out, workspace)
    try:
        dev = dY.device
        dX = torch.empty((m, d), dtype=xt, device=dev) if need_dx else None
        dw = db = None
        if need_dw:
            dw = _gradient(dw_out, (d,), accumulate, dev)
        if need_db:
            db = _gradient(db_out, (d,), accumulate, dev)
        need = sketch_norm_bwd_workspace(m, d) if need_dw or need_db else 0
        ws = _workspace(workspace, need, dev)
        st = lib().sketch_norm_bwd(_ptr(dY), dtype_code(dY), _ptr(X), xc, _ptr(codes), _ptr(scales),
                                   _ptr(weight), pc, _ptr(mean), _ptr(rstd), m, d, k, _ptr(dX), _ptr(dw), _ptr(db),
                                   1 if accumulate else 0, _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_norm_bwd", st)
    return dX, dw, db


# --------------------------------------------------------------------------
# cross entropy of a sketched head
# --------------------------------------------------------------------------

def _check_xent(X, idx_packed, lut, targets, b: int, gpr: int, **vectors):
    m, d = _matrix(X, "X")
    n = idx_packed.shape[0]
    _expect(X, "X", dtypes=("float16", "bfloat16"))
    _check_sketch(idx_packed, lut, n, d, b, gpr)
    _expect(lut, "lut", dtypes=("float16", "bfloat16"))
    _expect(targets, "targets", shape=(m,), dtypes=("int64",))
    for name, t in vectors.items():
        _expect(t, name, shape=(m,), dtypes=("float32",))
    return m, n, d


def sketch_xent_fwd_workspace(m: int, n: int, d: int, b: int, gpr: int, x_dtype: int, lut_dtype: int) -> int:
    """Bytes of device workspace sketch_xent_fwd needs for these sizes and dtypes."""
    return int(lib().sketch_xent_fwd_workspace(m, n, d, b, gpr, x_dtype, lut_dtype))


def sketch_xent_fwd(X, idx_packed, lut, targets, b: int, gpr: int, ignore_index: int = -100, workspace=None,
                    stream=None) -> Tuple[object, object]:
    """(loss, lse), fp32 [m]: softmax cross entropy of the logits X W^T, which are never stored.

    X [m, d] f16/bf16, idx_packed [n, d*b/8] uint8 and lut [n, gpr, 2^b] the sketched head of n words (f16 X
    needs f16 tables), targets [m] int64. Tokens whose target is ignore_index have loss and lse 0; any other
    target outside [0, n) gives loss NaN.
    """
    torch = _torch()
    m, n, d = _check_xent(X, idx_packed, lut, targets, b, gpr)
    _expect(workspace, "workspace", dtypes=("uint8",))
    xc, lc = dtype_code(X), dtype_code(lut)
    sp, context = _enter(stream, X, idx_packed, lut, targets, workspace)
    try:
        loss = torch.empty(m, dtype=torch.float32, device=X.device)
        lse = torch.empty(m, dtype=torch.float32, device=X.device)
        ws = _workspace(workspace, sketch_xent_fwd_workspace(m, n, d, b, gpr, xc, lc), X.device)
        st = lib().sketch_xent_fwd(_ptr(X), xc, idx_packed.data_ptr(), lut.data_ptr(), lc, _ptr(targets), ignore_index,
                                   m, n, d, b, gpr, _ptr(loss), _ptr(lse), _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_xent_fwd", st)
    return loss, lse


def sketch_xent_mean(loss, targets, ignore_index: int = -100, stream=None) -> Tuple[object, object]:
    """(mean, weight): the mean (fp32, 0 dimensions) of the losses whose target is not ignore_index, and every
    token's weight in it, fp32 [m] (0 for ignored tokens; mean and weights 0 when all are)."""
    torch = _torch()
    if loss.dim() != 1 or loss.numel() < 1:
        raise ValueError(f"loss must be a vector of at least one token, got {tuple(loss.shape)}")
    m = loss.numel()
    _expect(loss, "loss", dtypes=("float32",))
    _expect(targets, "targets", shape=(m,), dtypes=("int64",))
    sp, context = _enter(stream, loss, targets)
    try:
        mean = loss.new_empty(())
        weight = torch.empty_like(loss)
        st = lib().sketch_xent_mean(loss.data_ptr(), targets.data_ptr(), ignore_index, m, mean.data_ptr(),
                                    weight.data_ptr(), sp)
    finally:
        _leave(context)
    _check("sketch_xent_mean", st)
    return mean, weight


def sketch_xent_bwd_workspace(m: int, n: int, d: int, b: int, gpr: int, x_dtype: int, lut_dtype: int,
                              need_dx: bool = True, need_dlut: bool = True) -> int:
    """Bytes of device workspace sketch_xent_bwd needs for these sizes and dtypes."""
    return int(lib().sketch_xent_bwd_workspace(m, n, d, b, gpr, x_dtype, lut_dtype, 1 if need_dx else 0,
                                               1 if need_dlut else 0))


def sketch_xent_bwd(X, idx_packed, lut, targets, lse, dloss, b: int, gpr: int, ignore_index: int = -100,
                    need_dx: bool = True, need_dlut: bool = True, dlut_out=None, accumulate: bool = False,
                    workspace=None, stream=None) -> Tuple[object, object]:
    """(dX, dLUT) of sketch_xent_fwd's losses: dX [m, d] in X's dtype, dLUT fp32 [n, gpr, 2^b]; None if not asked.

    lse [m] as sketch_xent_fwd gave it, dloss [m] fp32 the gradient of every token's loss. dlut_out: optional
    fp32 [n, gpr, 2^b] to write (accumulate=True adds to it; to zeros without it). The other arguments are the forward's.
    """
    torch = _torch()
    m, n, d = _check_xent(X, idx_packed, lut, targets, b, gpr, lse=lse, dloss=dloss)
    K = 1 << b
    _expect(dlut_out, "dlut_out", shape=(n, gpr, K), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    xc, lc = dtype_code(X), dtype_code(lut)
    sp, context = _enter(stream, X, idx_packed, lut, targets, lse, dloss, dlut_out, workspace)
    try:
        dX = torch.empty((m, d), dtype=X.dtype, device=X.device) if need_dx else None
        dL = None
        if need_dlut:
            dL = _gradient(dlut_out, (n, gpr, K), accumulate, X.device)
        ws = _workspace(workspace, sketch_xent_bwd_workspace(m, n, d, b, gpr, xc, lc, need_dx, need_dlut), X.device)
        st = lib().sketch_xent_bwd(_ptr(X), xc, idx_packed.data_ptr(), lut.data_ptr(), lc, _ptr(targets), ignore_index,
                                   _ptr(lse), _ptr(dloss), m, n, d, b, gpr, _ptr(dX), _ptr(dL),
                                   1 if accumulate else 0, _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_xent_bwd", st)
    return dX, dL


# --------------------------------------------------------------------------
# dropout, low-rank adapters, norm and rotation of heads
# --------------------------------------------------------------------------

# These calls are short on the device, so what is right is found in one expression; the checks one by one word the error.

def _check_dropout(p: float, seed):
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p = {p} is not a probability")
    if seed is None:
        if p * 65536 + 0.5 >= 1.0:
            raise ValueError("dropout needs a seed")
    else:
        _expect(seed, "seed", shape=(2,), dtypes=("int64",))


def sketch_dropout(X, p: float, seed=None, residual=None, out=None, stream=None):
    """residual + dropout(X): every value of X is 0 with probability p, else divided by 1 - p (p to 2^-16).

    X (f32/f16/bf16, any shape), residual and out of X's shape and dtype. seed: int64 [2] on the GPU, (key, stream
    number), read when the work runs; the mask is computed from it and from a value's number and is never stored, so
    the gradient of X is the same call on the gradient.
    """
    torch = _torch()
    dt, code = X.dtype, _dtype_codes.get(X.dtype)
    if code is None:
        _expect(X, "X", dtypes=_FLOAT_DTYPES)
    _check_dropout(p, seed)
    for name, t in (("residual", residual), ("out", out)):
        if t is not None and (t.dtype is not dt or t.shape != X.shape):
            _expect(t, name, shape=X.shape, dtypes=(_dtype_name(X),))
    sp, context = _enter(stream, X, residual, seed, out)
    try:
        if out is None:
            out = torch.empty_like(X)
        st = lib().sketch_dropout(_ptr(X), code, _ptr(residual), X.numel(), p, _ptr(seed), _ptr(out), sp)
    finally:
        _leave(context)
    _check("sketch_dropout", st)
    return out


def _check_adapter(X, A, B, adapter, scale):
    """(m, n, d, r, n_adapters) of X [m, d], A [n_adapters, r, d], B [n_adapters, n, r] in one 16-bit dtype."""
    torch = _torch()
    m, d = _matrix(X, "X")
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A and B must have the adapters as the first of three dimensions")
    S, r, da = A.shape
    sb, n, rb = B.shape
    dt = X.dtype
    if not (da == d and sb == S and rb == r and A.dtype is dt and B.dtype is dt
            and (dt is torch.float16 or dt is torch.bfloat16)
            and (adapter is None or (adapter.dtype is torch.int32 and adapter.shape == (m,)))
            and (scale is None or (scale.dtype is torch.float32 and scale.shape == (S,)))):
        name = (_dtype_name(X),)
        _expect(X, "X", dtypes=("float16", "bfloat16"))
        _expect(A, "A", shape=(S, r, d), dtypes=name)
        _expect(B, "B", shape=(S, n, r), dtypes=name)
        _expect(adapter, "adapter", shape=(m,), dtypes=("int32",))
        _expect(scale, "scale", shape=(S,), dtypes=("float32",))
    return m, n, d, r, S


def sketch_adapter_fwd_workspace(m: int, n: int, d: int, r: int, n_adapters: int, has_ids: bool = True,
                                 has_dropout: bool = True) -> int:
    """Bytes of device workspace sketch_adapter_fwd needs for these sizes (has_ids: with a token's adapter given;
    has_dropout: with p > 0; a few tokens without dropout need none)."""
    return int(lib().sketch_adapter_fwd_workspace(m, n, d, r, n_adapters, 1 if has_ids else 0, 1 if has_dropout else 0))


def sketch_adapter_fwd(X, A, B, base=None, adapter=None, scale=None, p: float = 0.0, seed=None, out=None,
                       need_h: bool = False, workspace=None, stream=None) -> Tuple[object, object]:
    """(Y, H): Y[t] = base[t] + scale[s] B[s] H[t], H[t] = A[s] dropout(X[t]), s = adapter[t].

    X [m, d], A [n_adapters, r, d], B [n_adapters, n, r] and base [m, n] (None = zeros) f16 or bf16, all the same.
    adapter int32 [m]: a token's adapter, outside [0, n_adapters) = none (None: all have adapter 0); scale fp32
    [n_adapters] (None = ones). p, seed: dropout of X as in sketch_dropout. out: optional output, may be base itself.
    need_h: also return H, fp32 [m, r], which the backward pass takes (None otherwise).
    """
    torch = _torch()
    m, n, d, r, S = _check_adapter(X, A, B, adapter, scale)
    _check_dropout(p, seed)
    for name, t in (("base", base), ("out", out)):
        if t is not None and (t.dtype is not X.dtype or t.shape != (m, n)):
            _expect(t, name, shape=(m, n), dtypes=(_dtype_name(X),))
    if workspace is not None:
        _expect(workspace, "workspace", dtypes=("uint8",))
    sp, context = _enter(stream, X, A, B, base, adapter, scale, seed, out, workspace)
    try:
        if out is None:
            out = X.new_empty((m, n))
        H = X.new_empty((m, r), dtype=torch.float32) if need_h else None
        ws = _workspace(workspace, sketch_adapter_fwd_workspace(m, n, d, r, S, adapter is not None, p > 0.0), X.device)
        st = lib().sketch_adapter_fwd(_ptr(X), _ptr(A), _ptr(B), dtype_code(X), _ptr(adapter), S, _ptr(scale),
                                      _ptr(base), p, _ptr(seed), m, n, d, r, _ptr(out), _ptr(H), _ptr(ws), _size(ws),
                                      sp)
    finally:
        _leave(context)
    _check("sketch_adapter_fwd", st)
    return out, H


def sketch_adapter_bwd_workspace(m: int, n: int, d: int, r: int, n_adapters: int, has_ids: bool = True,
                                 need_dx: bool = True, need_da: bool = True, need_db: bool = True) -> int:
    """Bytes of device workspace sketch_adapter_bwd needs for these sizes."""
    return int(lib().sketch_adapter_bwd_workspace(m, n, d, r, n_adapters, 1 if has_ids else 0, 1 if need_dx else 0,
                                                  1 if need_da else 0, 1 if need_db else 0))


def sketch_adapter_bwd(dY, X, H, A, B, base_dx=None, adapter=None, scale=None, p: float = 0.0, seed=None,
                       need_dx: bool = True, need_da: bool = True, need_db: bool = True, da_out=None, db_out=None,
                       accumulate: bool = False, workspace=None, stream=None):
    """(dX, dA, dB) of sketch_adapter_fwd; None where not asked for.

    dY [m, n] in X's dtype, H as the forward gave it (None if dB is not asked for), the other arguments the forward's.
    dX [m, d] in X's dtype is base_dx (fp32 [m, d], None = zeros) plus the adapters' part; dA, dB fp32 in the shapes
    of A and B (da_out / db_out: optional outputs, accumulate=True adds to them). At most 4096 adapters (the forward
    takes 2^20), and (n / 128 + d / 128) (m / 128 + 1 + min(m, n_adapters)) blocks below 2^24.
    """
    torch = _torch()
    m, n, d, r, S = _check_adapter(X, A, B, adapter, scale)
    if S > 4096:
        raise ValueError(f"{S} adapters: a backward call takes at most 4096")
    if (-(-n // 128) - (-d // 128)) * (m // 128 + 1 + min(m, S)) >= 1 << 24:
        raise ValueError(f"{m} tokens of {S} adapters with {n} rows and {d} columns: a backward call takes less than 2^24 "
                         "blocks of 128 rows or columns and 128 tokens or an adapter's")
    _check_dropout(p, seed)
    _expect(dY, "dY", shape=(m, n), dtypes=(_dtype_name(X),))
    if need_db and H is None:
        raise ValueError("the gradient of B needs H")
    _expect(H, "H", shape=(m, r), dtypes=("float32",))
    _expect(base_dx, "base_dx", shape=(m, d), dtypes=("float32",))
    _expect(da_out, "da_out", shape=(S, r, d), dtypes=("float32",))
    _expect(db_out, "db_out", shape=(S, n, r), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    sp, context = _enter(stream, dY, X, H, A, B, base_dx, adapter, scale, seed, da_out, db_out, workspace)
    try:
        dev = X.device
        dX = torch.empty_like(X) if need_dx else None
        dA = dB = None
        if need_da:
            dA = _gradient(da_out, (S, r, d), accumulate, dev)
        if need_db:
            dB = _gradient(db_out, (S, n, r), accumulate, dev)
        ws = _workspace(workspace, sketch_adapter_bwd_workspace(m, n, d, r, S, adapter is not None, need_dx, need_da,
                                                                need_db), dev)
        st = lib().sketch_adapter_bwd(_ptr(dY), _ptr(X), _ptr(H), _ptr(A), _ptr(B), dtype_code(X), _ptr(adapter), S,
                                      _ptr(scale), _ptr(base_dx), p, _ptr(seed), m, n, d, r, _ptr(dX), _ptr(dA),
                                      _ptr(dB), 1 if accumulate else 0, _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_adapter_bwd", st)
    return dX, dA, dB


_PAIRS = {"halves": 0, "neighbours": 1}


def _pairs(pairs: str) -> int:
    if pairs not in _PAIRS:
        raise ValueError(f"pairs = {pairs!r}: supported are 'halves' and 'neighbours'")
    return _PAIRS[pairs]


def _head_rows(t, name: str, like=None):
    """(address, elements from token to token) of heads [m, heads, head_dim] whose heads lie side by side."""
    if t is None:
        return None, 0
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions (tokens, heads, columns), got {t.dim()}")
    if like is not None and (t.shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device()):
        _expect(t, name, shape=like.shape, dtypes=(_dtype_name(like),))
        raise ValueError(f"{name} must live where the heads do")
    if not t.is_cuda:
        raise ValueError("tensors must live on the GPU")
    m, h, dh = t.shape
    ld, sh, sc = t.stride()
    if (dh > 1 and sc != 1) or (h > 1 and sh != dh) or (m > 1 and ld < h * dh):
        raise ValueError(f"{name}: the heads of a token must lie side by side")
    return t.data_ptr(), (ld if m > 1 else h * dh)


def _check_rotary(q, k, positions, inv_freq, q_weight, k_weight, eps):
    torch = _torch()
    qp, ldq = _head_rows(q, "q")
    m, hq, dh = q.shape
    dt, index = q.dtype, q.get_device()
    kp, ldk, hk = None, 0, 0
    if k is not None:
        kp, ldk = _head_rows(k, "k")
        hk = k.shape[1]
        if k.dtype is not dt or k.shape != (m, hk, dh):
            _expect(k, "k", shape=(m, hk, dh), dtypes=(_dtype_name(q),))
        if k.get_device() != index:
            raise ValueError("q and k must live on one GPU")
    if dt not in _dtype_codes:
        _expect(q, "q", dtypes=_FLOAT_DTYPES)
    if positions.dtype is not torch.int64 or positions.shape != (m,):
        _expect(positions, "positions", shape=(m,), dtypes=("int64",))
    if inv_freq.dtype is not torch.float64:
        _expect(inv_freq, "inv_freq", dtypes=("float64",))
    if inv_freq.dim() != 1 or not 1 <= inv_freq.numel() <= dh // 2:
        raise ValueError(f"inv_freq must be a vector of 1 to {dh // 2} frequencies, got {tuple(inv_freq.shape)}")
    if q_weight is not None or k_weight is not None:
        if eps is None:
            raise ValueError("weights belong to a norm: give its eps")
        _expect(q_weight, "q_weight", shape=(dh,), dtypes=("float32",))
        _expect(k_weight, "k_weight", shape=(dh,), dtypes=("float32",))
    if positions.get_device() != index:
        raise ValueError("positions must live where the heads do")
    return m, hq, hk, dh, qp, ldq, kp, ldk


def _head_outputs(q, k, q_out, k_out, m: int, hq: int, hk: int, dh: int):
    """The outputs beside q and k (new ones where none are given) and their addresses and strides."""
    if q_out is None:
        q_out = q.new_empty((m, hq, dh))
        qo, ldqo = q_out.data_ptr(), hq * dh
    else:
        qo, ldqo = _head_rows(q_out, "q_out", q)
    ko, ldko = None, 0
    if k is not None:
        if k_out is None:
            k_out = q.new_empty((m, hk, dh))
            ko, ldko = k_out.data_ptr(), hk * dh
        else:
            ko, ldko = _head_rows(k_out, "k_out", k)
    return q_out, k_out, qo, ldqo, ko, ldko


def sketch_rotary_fwd(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: Optional[float] = None,
                      pairs: str = "halves", q_out=None, k_out=None, stream=None) -> Tuple[object, object]:
    """(q', k'): the heads q [m, heads, head_dim] and k (None = none) normed and turned by their positions.

    f32/f16/bf16; rows may be strided (the q and k columns of a joined projection). positions int64 [m], inv_freq
    float64 [rot_dim / 2]: pair i of a head turns by positions[t] * inv_freq[i], columns from rot_dim on stay. pairs:
    "halves" (i, i + rot_dim / 2) or "neighbours" (2 i, 2 i + 1). eps: of the root-mean-square norm of every head
    (None = no norm), q_weight / k_weight its fp32 [head_dim] weights (None = ones). q_out / k_out: optional outputs,
    also q and k themselves.
    """
    m, hq, hk, dh, qp, ldq, kp, ldk = _check_rotary(q, k, positions, inv_freq, q_weight, k_weight, eps)
    pc = _pairs(pairs)
    if k is None and k_out is not None:
        raise ValueError("k_out without k")
    sp, context = _enter(stream, positions, inv_freq, q_weight, k_weight)
    try:
        q_out, k_out, qo, ldqo, ko, ldko = _head_outputs(q, k, q_out, k_out, m, hq, hk, dh)
        st = lib().sketch_rotary_fwd(qp, ldq, hq, kp, ldk, hk, dtype_code(q), _ptr(positions), _ptr(inv_freq),
                                     _ptr(q_weight), _ptr(k_weight), m, dh, 2 * inv_freq.numel(), pc,
                                     0 if eps is None else 1, 0.0 if eps is None else eps, qo, ldqo, ko, ldko, sp)
    finally:
        _leave(context)
    _check("sketch_rotary_fwd", st)
    return q_out, k_out


def sketch_rotary_bwd_workspace(head_dim: int) -> int:
    """Bytes of device workspace sketch_rotary_bwd needs for weight gradients."""
    return int(lib().sketch_rotary_bwd_workspace(head_dim))


def sketch_rotary_bwd(dq, dk, q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: Optional[float] = None,
                      pairs: str = "halves", need_dw: bool = True, q_out=None, k_out=None, qw_out=None, kw_out=None,
                      accumulate: bool = False, workspace=None, stream=None):
    """(dq_in, dk_in, dq_weight, dk_weight) of sketch_rotary_fwd; the weights' gradients fp32 [head_dim], with a norm
    and need_dw only (else None).

    dq, dk: gradients of the outputs, strided rows of the heads' dtype; the other arguments the forward's. q_out /
    k_out: optional outputs for the heads' gradients (strided rows, e.g. of one joined buffer); qw_out / kw_out for
    the weights' (accumulate=True adds to them).
    """
    m, hq, hk, dh, qp, ldq, kp, ldk = _check_rotary(q, k, positions, inv_freq, q_weight, k_weight, eps)
    pc = _pairs(pairs)
    if (dk is None) != (k is None) or (k is None and (k_out is not None or kw_out is not None)):
        raise ValueError("dk, k_out and kw_out go with k")
    if eps is None and (qw_out is not None or kw_out is not None):
        raise ValueError("weights belong to a norm: give its eps")
    dqp, lddq = _head_rows(dq, "dq", q)
    dkp, lddk = _head_rows(dk, "dk", k)
    for name, t in (("qw_out", qw_out), ("kw_out", kw_out)):
        _expect(t, name, shape=(dh,), dtypes=("float32",))
    _expect(workspace, "workspace", dtypes=("uint8",))
    need_dw = need_dw and eps is not None
    sp, context = _enter(stream, positions, inv_freq, q_weight, k_weight, qw_out, kw_out, workspace)
    try:
        dev = q.device
        q_out, k_out, qo, ldqo, ko, ldko = _head_outputs(q, k, q_out, k_out, m, hq, hk, dh)
        dqw = dkw = ws = None
        if need_dw:
            dqw = _gradient(qw_out, (dh,), accumulate, dev)
            if k is not None:
                dkw = _gradient(kw_out, (dh,), accumulate, dev)
            ws = _workspace(workspace, sketch_rotary_bwd_workspace(dh), dev)
        st = lib().sketch_rotary_bwd(dqp, lddq, hq, dkp, lddk, hk, dtype_code(q), qp, ldq, kp, ldk, _ptr(positions),
                                     _ptr(inv_freq), _ptr(q_weight), _ptr(k_weight), m, dh, 2 * inv_freq.numel(), pc,
                                     0 if eps is None else 1, 0.0 if eps is None else eps, qo, ldqo, ko, ldko,
                                     _ptr(dqw), _ptr(dkw), 1 if accumulate else 0, _ptr(ws), _size(ws), sp)
    finally:
        _leave(context)
    _check("sketch_rotary_bwd", st)
    return q_out, k_out, dqw, dkw
