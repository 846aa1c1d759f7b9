"""Python binding of the t3 C ABI (include/t3.h): argument marshalling only.

Every product runs in the CUDA kernels of ``libt3.so``; this module checks
dtypes, shapes and devices, allocates outputs with torch when the caller does
not pass them, and forwards raw pointers and the current CUDA stream.  There
is no fallback: if the library is missing or cannot load, every call raises.

Function names follow the C ABI:
  t3_pack_ternary(w)                       host packer, w int8 [K][N]
  t3_pack_ternary_device(w, wp=None)       the same on the GPU (w a CUDA tensor)
  t3_gemm_fwd(A, Wp, K=None, C=None)       C  = A . W        (int32 [M][N])
  t3_gemm_bwd_dx(dY, Wp, K, dX=None)       dX = dY . W^T     (int32 [M][K])
  t3_gemm_bwd_dw(A, dY, dW=None)           dW = A^T . dY     (int32 [K][N])
  t3_quantize_rows_bf16(x)                 (int8 q, per-row scale) from bf16 x
  t3_gemm_fwd_bf16(x, Wp)                  the quantizer fused into the forward
  t3_dequant_i32(x, kind, row_scale, col_scale, out=None)   scaled float/bf16 output
  t3_gemm_fwd_scaled / t3_gemm_bwd_dx_scaled / t3_gemm_bwd_dw_scaled
                                           the products with that output
  t3_rmsnorm_quant(x, gamma, residual)     residual add, norm, int8 rows with scales
  t3_rmsnorm_bwd(dy, s, rstd, gamma)       its gradient
  t3_gated_scan_fwd(gate, cand, h0)        the gated linear recurrence (sequences, tokens)
  t3_gated_scan_bwd(gate, cand, h, dh)     its gradient
  t3_gemm_fwd_act(A, Wp, bias=, act=)      the forward with bias, activation, residual
  t3_act_bwd(dy, z, act)                   that epilogue's gradient
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libt3.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "t3.h")

T3_OK, T3_EINVAL, T3_EVALUE, T3_EOVERFLOW, T3_ECUDA, T3_ETIMEOUT, T3_EDEVICE = 0, -1, -2, -3, -4, -5, -6
T3_OUT_F32, T3_OUT_BF16, T3_OUT_F32_ADD = 0, 1, 2
T3_ACT_NONE, T3_ACT_RELU, T3_ACT_RELU2, T3_ACT_SILU, T3_ACT_GELU = 0, 1, 2, 3, 4

_lock = threading.Lock()
_lib = None


class T3Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def build(force: bool = False) -> str:
    """Compiles libt3.so for sm_103a (nvcc); returns its path."""
    from . import _build
    return _build.build(force=force)


def load():
    """Loads libt3.so (building it first if it is absent or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        from . import _build
        if not _build.up_to_date():
            _build.build()
        lib = ctypes.CDLL(LIB_PATH)
        p, i64 = ctypes.c_void_p, ctypes.c_int64
        lib.t3_pack_ternary.argtypes = [p, p, i64, i64]
        for name in ("t3_gemm_fwd", "t3_gemm_bwd_dx", "t3_gemm_bwd_dw"):
            f = getattr(lib, name)
            f.argtypes = [p, p, p, i64, i64, i64, p]
            f.restype = ctypes.c_int
        lib.t3_pack_ternary.restype = ctypes.c_int
        lib.t3_pack_ternary_device.argtypes = [p, p, i64, i64, p]
        lib.t3_pack_ternary_device.restype = ctypes.c_int
        lib.t3_quantize_rows_bf16.argtypes = [p, p, p, i64, i64, p]
        lib.t3_quantize_rows_bf16.restype = ctypes.c_int
        lib.t3_gemm_fwd_bf16.argtypes = [p, p, p, p, p, i64, i64, i64, p]
        lib.t3_gemm_fwd_bf16.restype = ctypes.c_int
        lib.t3_dequant_i32.argtypes = [p, p, i64, i64, p, p, ctypes.c_int, p]
        lib.t3_dequant_i32.restype = ctypes.c_int
        for name in ("t3_gemm_fwd_scaled", "t3_gemm_bwd_dx_scaled", "t3_gemm_bwd_dw_scaled"):
            f = getattr(lib, name)
            f.argtypes = [p, p, p, i64, i64, i64, p, p, ctypes.c_int, p, p]
            f.restype = ctypes.c_int
        lib.t3_gemm_bwd_dw_scaled_noalloc.argtypes = [p, p, p, i64, i64, i64, p, p, ctypes.c_int, p]
        lib.t3_gemm_bwd_dw_scaled_noalloc.restype = ctypes.c_int
        lib.t3_status_string.argtypes = [ctypes.c_int]
        lib.t3_status_string.restype = ctypes.c_char_p
        lib.t3_last_device_error.argtypes = [p, ctypes.POINTER(ctypes.c_int32)]
        lib.t3_last_device_error.restype = ctypes.c_int
        for f in (lib.t3_selftest_wait_timeout, lib.t3_selftest_scan_wait_timeout):
            f.argtypes = [i64, p]
            f.restype = ctypes.c_int
        lib.t3_set_small_product_limit.argtypes = [i64]
        lib.t3_set_small_product_limit.restype = i64
        i32 = ctypes.c_int
        for name, types in (
                ("t3_rmsnorm_quant", [p, i64, p, i64, p, ctypes.c_float, p, p, p, p, i64, i64, i64, i32, p]),
                ("t3_rmsnorm_bwd", [p, i64, p, i64, p, p, p, i64, p, i64, p, i64, i64, i32, p, p]),
                ("t3_gated_scan_fwd", [p, i64, p, i64, p, p, p, i64, p, i64, i64, i64, i32, p]),
                ("t3_gated_scan_bwd", [p, i64, p, i64, p, i64, p, i64, p, p, p, p, i64, p, i64, p,
                                       i64, i64, i64, i32, p]),
                ("t3_gemm_fwd_act", [p, p, p, i64, i64, i64, p, p, p, i32, p, p, i32, p, p, i64, p]),
                ("t3_act_bwd", [p, p, i32, p, p, i64, i64, i32, p, p])):
            f = getattr(lib, name)
            f.argtypes = types
            f.restype = ctypes.c_int
        for f in (lib.t3_gemm_fwd_act_scratch, lib.t3_gemm_fwd_act_scratch_now):
            f.argtypes = [i64, i64, i64]
            f.restype = i64
        lib.t3_gemm_fwd_act_workspace.argtypes = [p, p, p, i64, i64, i64, p, p, i32, i64]
        lib.t3_gemm_fwd_act_workspace.restype = i64
        lib.t3_colsum_workspace.argtypes = [i64, i64]
        lib.t3_colsum_workspace.restype = i64
        lib.t3_version.argtypes = []
        lib.t3_version.restype = ctypes.c_int
        _lib = lib
        return lib


def declared_functions() -> list[str]:
    """Names of the functions include/t3.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:int|const char\*)\s+(t3_\w+)\s*\(", text, re.M)))


def status_string(status: int) -> str:
    return load().t3_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != T3_OK:
        raise T3Error(status, where)


# ------------------------------------------------------------------- host ---

def t3_pack_ternary(w) -> np.ndarray:
    """Packs ternary w (int8 [K][N], values in {-1,0,+1}; numpy or CPU tensor)
    into Wp (uint8 [N][ceil(K/4)]) with the library's host packer."""
    if hasattr(w, "detach"):
        w = w.detach().cpu().numpy()
    w = np.ascontiguousarray(w)
    if w.dtype != np.int8 or w.ndim != 2:
        raise TypeError("w must be a 2-D int8 array [K][N]")
    K, N = w.shape
    wp = np.empty((N, (K + 3) // 4), dtype=np.uint8)
    rc = load().t3_pack_ternary(ctypes.c_void_p(w.ctypes.data), ctypes.c_void_p(wp.ctypes.data),
                                K, N)
    _check(rc, "t3_pack_ternary")
    return wp


# ----------------------------------------------------------------- device ---

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _dev_ptr(t, dtype, name):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr() if t.numel() else 0)


def _stream(t, stream):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(s.cuda_stream)


def t3_pack_ternary_device(w, wp=None, stream=None):
    """Packs ternary w (CUDA int8 tensor [K][N]) into Wp (CUDA uint8
    [N][ceil(K/4)]) on the GPU, asynchronously on `stream`.  A value outside
    {-1, 0, +1} packs as 0 and is reported by t3_last_device_error."""
    torch = _torch()
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise TypeError("w must be a 2-D CUDA int8 tensor [K][N]")
    K, N = w.shape
    if wp is None:
        wp = torch.empty((N, (K + 3) // 4), dtype=torch.uint8, device=w.device)
    if tuple(wp.shape) != (N, (K + 3) // 4):
        raise ValueError(f"wp must be [{N}][{(K + 3) // 4}], got {tuple(wp.shape)}")
    rc = load().t3_pack_ternary_device(_dev_ptr(w, torch.int8, "w"), _dev_ptr(wp, torch.uint8, "wp"),
                                       K, N, _stream(w, stream))
    _check(rc, "t3_pack_ternary_device")
    return wp


def t3_gemm_fwd(A, Wp, K: int | None = None, C=None, stream=None):
    """C[m][n] = sum_k A[m][k] W[k][n].  A int8 [M][K], Wp uint8 [N][ceil(K/4)]."""
    torch = _torch()
    M, Ka = A.shape
    K = Ka if K is None else K
    if Ka != K:
        raise ValueError("A must be [M][K]")
    N = Wp.shape[0]
    if Wp.dim() != 2 or Wp.shape[1] != (K + 3) // 4:
        raise ValueError("Wp must be [N][ceil(K/4)]")
    if C is None:
        _dev_ptr(A, torch.int8, "A")
        C = torch.empty((M, N), dtype=torch.int32, device=A.device)
    elif tuple(C.shape) != (M, N):
        raise ValueError("C must be [M][N]")
    args = (_dev_ptr(A, torch.int8, "A"), _dev_ptr(Wp, torch.uint8, "Wp"),
            _dev_ptr(C, torch.int32, "C"))
    with torch.cuda.device(A.device):
        rc = load().t3_gemm_fwd(*args, M, N, K, _stream(A, stream))
    _check(rc, "t3_gemm_fwd")
    return C


def t3_gemm_bwd_dx(dY, Wp, K: int, dX=None, stream=None):
    """dX[m][k] = sum_n dY[m][n] W[k][n].  dY int8 [M][N], Wp uint8 [N][ceil(K/4)]."""
    torch = _torch()
    M, N = dY.shape
    if Wp.dim() != 2 or tuple(Wp.shape) != (N, (K + 3) // 4):
        raise ValueError("Wp must be [N][ceil(K/4)]")
    if dX is None:
        _dev_ptr(dY, torch.int8, "dY")
        dX = torch.empty((M, K), dtype=torch.int32, device=dY.device)
    elif tuple(dX.shape) != (M, K):
        raise ValueError("dX must be [M][K]")
    args = (_dev_ptr(dY, torch.int8, "dY"), _dev_ptr(Wp, torch.uint8, "Wp"),
            _dev_ptr(dX, torch.int32, "dX"))
    with torch.cuda.device(dY.device):
        rc = load().t3_gemm_bwd_dx(*args, M, N, K, _stream(dY, stream))
    _check(rc, "t3_gemm_bwd_dx")
    return dX


def t3_gemm_bwd_dw(A, dY, dW=None, stream=None):
    """dW[k][n] = sum_m A[m][k] dY[m][n].  A int8 [M][K], dY int8 [M][N]."""
    torch = _torch()
    M, K = A.shape
    if dY.shape[0] != M:
        raise ValueError("A and dY must have the same number of rows")
    N = dY.shape[1]
    if dW is None:
        _dev_ptr(A, torch.int8, "A")
        dW = torch.empty((K, N), dtype=torch.int32, device=A.device)
    elif tuple(dW.shape) != (K, N):
        raise ValueError("dW must be [K][N]")
    args = (_dev_ptr(A, torch.int8, "A"), _dev_ptr(dY, torch.int8, "dY"),
            _dev_ptr(dW, torch.int32, "dW"))
    with torch.cuda.device(A.device):
        rc = load().t3_gemm_bwd_dw(*args, M, N, K, _stream(A, stream))
    _check(rc, "t3_gemm_bwd_dw")
    return dW


# ------------------------------------------------------------ scaled outputs

def _scaled_out(out, kind, rows, cols, device, name):
    torch = _torch()
    dtype = torch.bfloat16 if kind == T3_OUT_BF16 else torch.float32
    if kind not in (T3_OUT_F32, T3_OUT_BF16, T3_OUT_F32_ADD):
        raise ValueError(f"unknown output kind {kind}")
    if out is None:
        if kind == T3_OUT_F32_ADD:
            raise ValueError(f"{name}: the += kind needs the existing output")
        out = torch.empty((rows, cols), dtype=dtype, device=device)
    if tuple(out.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}]")
    return out, _dev_ptr(out, dtype, name)


def _scale_ptr(v, n, name):
    if v is None:
        return ctypes.c_void_p(0)
    if v.dim() != 1 or v.shape[0] != n:
        raise ValueError(f"{name} must have {n} entries")
    return _dev_ptr(v, _torch().float32, name)


def _ws_ptr(ws, rows, cols):
    if ws is None:
        return ctypes.c_void_p(0)
    if tuple(ws.shape) != (rows, cols):
        raise ValueError(f"workspace must be [{rows}][{cols}]")
    return _dev_ptr(ws, _torch().int32, "workspace")


def t3_quantize_rows_bf16(x, q=None, row_scale=None, stream=None):
    """(q, row_scale): bf16 x [M][K] quantized to int8 with one absmax scale
    per row (see include/t3.h)."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a 2-D CUDA bfloat16 tensor [M][K]")
    M, K = x.shape
    if q is None:
        q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if row_scale is None:
        row_scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    if tuple(q.shape) != (M, K) or tuple(row_scale.shape) != (M,):
        raise ValueError("q must be [M][K] and row_scale [M]")
    args = (_dev_ptr(x, torch.bfloat16, "x"), _dev_ptr(q, torch.int8, "q"),
            _dev_ptr(row_scale, torch.float32, "row_scale"), M, K, _stream(x, stream))
    with torch.cuda.device(x.device):
        rc = load().t3_quantize_rows_bf16(*args)
    _check(rc, "t3_quantize_rows_bf16")
    return q, row_scale


def t3_gemm_fwd_bf16(x, Wp, C=None, row_scale=None, row_inv=None, stream=None):
    """(C, row_scale, row_inv): the forward product of the row-quantized bf16
    activations x [M][K] with the packed weights Wp [N][ceil(K/4)], the
    quantizer fused into the product (see include/t3.h); C int32 [M][N]."""
    torch = _torch()
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise TypeError("x must be a 2-D CUDA bfloat16 tensor [M][K]")
    M, K = x.shape
    N = Wp.shape[0]
    if Wp.dim() != 2 or Wp.shape[1] != (K + 3) // 4:
        raise ValueError("Wp must be [N][ceil(K/4)]")
    if C is None:
        C = torch.empty((M, N), dtype=torch.int32, device=x.device)
    if row_scale is None:
        row_scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    if row_inv is None:
        row_inv = torch.empty((M,), dtype=torch.float32, device=x.device)
    if tuple(C.shape) != (M, N) or tuple(row_scale.shape) != (M,) or tuple(row_inv.shape) != (M,):
        raise ValueError("C must be [M][N], row_scale and row_inv [M]")
    args = (_dev_ptr(x, torch.bfloat16, "x"), _dev_ptr(Wp, torch.uint8, "Wp"),
            _dev_ptr(C, torch.int32, "C"), _dev_ptr(row_scale, torch.float32, "row_scale"),
            _dev_ptr(row_inv, torch.float32, "row_inv"), M, N, K, _stream(x, stream))
    with torch.cuda.device(x.device):
        rc = load().t3_gemm_fwd_bf16(*args)
    _check(rc, "t3_gemm_fwd_bf16")
    return C, row_scale, row_inv


def t3_dequant_i32(x, kind=T3_OUT_F32, row_scale=None, col_scale=None, out=None, stream=None):
    """out = ((float)x * row_scale[r]) * col_scale[c] as float (T3_OUT_F32),
    bf16 (T3_OUT_BF16) or added to `out` (T3_OUT_F32_ADD).  x int32 [R][C]."""
    torch = _torch()
    rows, cols = x.shape
    out, po = _scaled_out(out, kind, rows, cols, x.device, "out")
    args = (_dev_ptr(x, torch.int32, "x"), po, rows, cols, _scale_ptr(row_scale, rows, "row_scale"),
            _scale_ptr(col_scale, cols, "col_scale"), kind, _stream(x, stream))
    with torch.cuda.device(x.device):
        rc = load().t3_dequant_i32(*args)
    _check(rc, "t3_dequant_i32")
    return out


def t3_gemm_fwd_scaled(A, Wp, K=None, row_scale=None, col_scale=None, kind=T3_OUT_F32, C=None,
                       workspace=None, stream=None):
    """C (scaled, float or bf16 [M][N]) of A . W; row_scale [M], col_scale [N]."""
    torch = _torch()
    M, Ka = A.shape
    K = Ka if K is None else K
    if Ka != K:
        raise ValueError("A must be [M][K]")
    N = Wp.shape[0]
    if Wp.dim() != 2 or Wp.shape[1] != (K + 3) // 4:
        raise ValueError("Wp must be [N][ceil(K/4)]")
    C, pc = _scaled_out(C, kind, M, N, A.device, "C")
    args = (_dev_ptr(A, torch.int8, "A"), _dev_ptr(Wp, torch.uint8, "Wp"), pc, M, N, K,
            _scale_ptr(row_scale, M, "row_scale"), _scale_ptr(col_scale, N, "col_scale"), kind,
            _ws_ptr(workspace, M, N), _stream(A, stream))
    with torch.cuda.device(A.device):
        rc = load().t3_gemm_fwd_scaled(*args)
    _check(rc, "t3_gemm_fwd_scaled")
    return C


def t3_gemm_bwd_dx_scaled(dY, Wp, K: int, row_scale=None, col_scale=None, kind=T3_OUT_F32,
                          dX=None, workspace=None, stream=None):
    """dX (scaled, float or bf16 [M][K]) of dY . W^T; row_scale [M], col_scale [K]."""
    torch = _torch()
    M, N = dY.shape
    if Wp.dim() != 2 or tuple(Wp.shape) != (N, (K + 3) // 4):
        raise ValueError("Wp must be [N][ceil(K/4)]")
    dX, px = _scaled_out(dX, kind, M, K, dY.device, "dX")
    args = (_dev_ptr(dY, torch.int8, "dY"), _dev_ptr(Wp, torch.uint8, "Wp"), px, M, N, K,
            _scale_ptr(row_scale, M, "row_scale"), _scale_ptr(col_scale, K, "col_scale"), kind,
            _ws_ptr(workspace, M, K), _stream(dY, stream))
    with torch.cuda.device(dY.device):
        rc = load().t3_gemm_bwd_dx_scaled(*args)
    _check(rc, "t3_gemm_bwd_dx_scaled")
    return dX


def t3_gemm_bwd_dw_scaled(A, dY, row_scale=None, col_scale=None, kind=T3_OUT_F32, dW=None,
                          workspace=None, stream=None):
    """dW (scaled, float or bf16 [K][N]) of A^T . dY; row_scale [K] (A's column
    scales), col_scale [N] (dY's column scales)."""
    torch = _torch()
    M, K = A.shape
    if dY.shape[0] != M:
        raise ValueError("A and dY must have the same number of rows")
    N = dY.shape[1]
    dW, pw = _scaled_out(dW, kind, K, N, A.device, "dW")
    args = (_dev_ptr(A, torch.int8, "A"), _dev_ptr(dY, torch.int8, "dY"), pw, M, N, K,
            _scale_ptr(row_scale, K, "row_scale"), _scale_ptr(col_scale, N, "col_scale"), kind,
            _ws_ptr(workspace, K, N), _stream(A, stream))
    with torch.cuda.device(A.device):
        rc = load().t3_gemm_bwd_dw_scaled(*args)
    _check(rc, "t3_gemm_bwd_dw_scaled")
    return dW


def t3_gemm_bwd_dw_scaled_noalloc(A, dY, row_scale=None, col_scale=None, kind=T3_OUT_F32,
                                  dW=None, stream=None):
    """t3_gemm_bwd_dw_scaled with the int32 intermediate in the library's fixed
    per-device buffer (K * N <= 8,388,608; calls on one device must not overlap)."""
    torch = _torch()
    M, K = A.shape
    if dY.shape[0] != M:
        raise ValueError("A and dY must have the same number of rows")
    N = dY.shape[1]
    dW, pw = _scaled_out(dW, kind, K, N, A.device, "dW")
    args = (_dev_ptr(A, torch.int8, "A"), _dev_ptr(dY, torch.int8, "dY"), pw, M, N, K,
            _scale_ptr(row_scale, K, "row_scale"), _scale_ptr(col_scale, N, "col_scale"), kind,
            _stream(A, stream))
    with torch.cuda.device(A.device):
        rc = load().t3_gemm_bwd_dw_scaled_noalloc(*args)
    _check(rc, "t3_gemm_bwd_dw_scaled_noalloc")
    return dW


# ------------------------------------------- norm, recurrence, epilogue ---

# These calls may run once per token of a serving loop, on a few kilobytes: the
# checks below read each tensor property once and build nothing.

def _dtype_of(t, name):
    """The element type's code (T3_OUT_F32 or T3_OUT_BF16) of an activation tensor."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is torch.bfloat16:
        return T3_OUT_BF16
    if t.dtype is torch.float32:
        return T3_OUT_F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _rows(t, dtype, dev, shape, name, out=False):
    """(address, row stride) of a tensor [..., cols] on device number `dev`
    whose rows are evenly spaced; None gives (None, 0)."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return _spaced(t, shape, name, out)


def _spaced(t, shape, name, out=False):
    """The same for a tensor whose type, device and shape are the call's."""
    st = t.stride()
    cols = shape[-1]
    if st[-1] != 1 and cols > 1 and t.numel():
        raise ValueError(f"{name}: the elements of a row must be adjacent")
    if len(shape) == 2:
        ld = st[0] if shape[0] > 1 else cols
    else:  # [batch][length][width]: one stride serves both
        batch, length = shape[0], shape[1]
        ld = st[1] if length > 1 else st[0] if batch > 1 else cols
        if batch > 1 and length > 1 and st[0] != length * ld and cols:
            raise ValueError(f"{name}: sequences must be evenly spaced (stride {st[0]}, not {length * ld})")
    if ld < cols:
        if not t.numel():
            ld = cols
        elif out:
            raise ValueError(f"{name}: output rows must not overlap")
    return t.data_ptr(), ld


def _dense(t, dtype, dev, shape, name):
    """Address of a contiguous tensor on device number `dev`; None gives None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev:
        raise TypeError(f"{name} must be a {dtype} tensor on device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _marks(resets, dev, shape):
    """Address of the resets, uint8 or bool (what a comparison gives)."""
    torch = _torch()
    if resets is not None and resets.dtype is torch.bool:
        resets = resets.view(torch.uint8)
    return _dense(resets, torch.uint8, dev, shape, "resets")


_fns = {}
_raw_stream = _device = None


def _bind(name):
    """The library's function, and the current stream's handle and device without
    the objects and checks around them."""
    global _raw_stream, _device
    torch = _torch()
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda d: torch.cuda.current_stream(d).cuda_stream)
    _device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    fn = _fns[name] = getattr(load(), name)
    return fn


def _on(dev, name, *args):
    """The library's answer on device number `dev`."""
    fn = _fns.get(name) or _bind(name)
    if dev == _device():
        return fn(*args)
    with _torch().cuda.device(dev):
        return fn(*args)


def _launch(name, dev, stream, *args):
    """Calls the library on device number `dev`, on its current stream unless one is given."""
    fn = _fns.get(name) or _bind(name)
    s = _raw_stream(dev) if stream is None else stream.cuda_stream
    if dev == _device():
        rc = fn(*args, s)
    else:
        with _torch().cuda.device(dev):
            rc = fn(*args, s)
    if rc != T3_OK:
        raise T3Error(rc, name)


def _empty(shape, dtype, dev, stream):
    """An output or workspace for a call on `stream` (None: the current one):
    allocated on that stream, so that memory another stream still uses is not
    handed out, nor this memory to another stream while the call is running."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


_col_parts = None


def _workspace(workspace, rows, cols, dev, stream):
    """The column sums' partial rows: t3_colsum_workspace(rows, cols) floats, at
    most a fixed number of rows."""
    global _col_parts
    if _col_parts is None:
        _col_parts = load().t3_colsum_workspace((1 << 31) - 1, 1)
    n = min(rows, _col_parts) * cols
    torch = _torch()
    if workspace is None:
        return _empty(n, torch.float32, dev, stream)
    if workspace.dtype is not torch.float32 or workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError(f"workspace must be a contiguous float32 tensor on device {dev}")
    if workspace.numel() < n:
        raise ValueError(f"workspace needs {n} floats, has {workspace.numel()}")
    return workspace


def t3_rmsnorm_quant(x, gamma=None, residual=None, eps=1e-5, q=None, row_scale=None, rstd=None,
                     sum_out=None, stream=None):
    """(q, row_scale, rstd, s): s = x + residual in x's type, normalized by its
    root mean square, times gamma, as int8 rows with one scale each; rstd and s
    are what t3_rmsnorm_bwd takes (see include/t3.h).  x [rows][cols] bfloat16
    or float32, rows evenly spaced; gamma float32 [cols].  s is x itself
    without a residual and without sum_out; sum_out may be x or residual."""
    torch = _torch()
    dtype = _dtype_of(x, "x")
    shape, xt, dev, f32 = x.shape, x.dtype, x.get_device(), torch.float32
    if len(shape) != 2:
        raise TypeError("x must be 2-D [rows][cols]")
    rows, cols = shape
    if q is None:
        q = _empty(shape, torch.int8, dev, stream)
    if row_scale is None:
        row_scale = _empty(rows, f32, dev, stream)
    if rstd is None:
        rstd = _empty(rows, f32, dev, stream)
    if sum_out is None and residual is not None:
        sum_out = _empty(shape, xt, dev, stream)
    px, ldx = _spaced(x, shape, "x")
    pr, ldr = _rows(residual, xt, dev, shape, "residual")
    ps, lds = _rows(sum_out, xt, dev, shape, "sum_out", out=True)
    _launch("t3_rmsnorm_quant", dev, stream, px, ldx, pr, ldr, _dense(gamma, f32, dev, (cols,), "gamma"), eps,
            _dense(q, torch.int8, dev, shape, "q"), _dense(row_scale, f32, dev, (rows,), "row_scale"),
            _dense(rstd, f32, dev, (rows,), "rstd"), ps, lds, rows, cols, dtype)
    return q, row_scale, rstd, x if sum_out is None else sum_out


def t3_rmsnorm_bwd(dy, s, rstd, gamma=None, dsum=None, dx=None, dgamma=None, workspace=None, stream=None):
    """(dx, dgamma): the gradient of t3_rmsnorm_quant for dy, the gradient of
    the normalized rows, and dsum, that of s itself; s and rstd are the
    forward's.  dgamma is None without gamma.  dx may be dy or dsum."""
    torch = _torch()
    dtype = _dtype_of(dy, "dy")
    if dy.dim() != 2:
        raise TypeError("dy must be 2-D [rows][cols]")
    shape, xt, dev, f32 = dy.shape, dy.dtype, dy.get_device(), torch.float32
    rows, cols = shape
    if dx is None:
        dx = _empty(shape, xt, dev, stream)
    if dgamma is None and gamma is not None:
        dgamma = _empty(cols, f32, dev, stream)
    ws = None if dgamma is None else _workspace(workspace, rows, cols, dev, stream)
    pdy, lddy = _spaced(dy, shape, "dy")
    ps, lds = _rows(s, xt, dev, shape, "s")
    pd, ldd = _rows(dsum, xt, dev, shape, "dsum")
    px, ldx = _rows(dx, xt, dev, shape, "dx", out=True)
    _launch("t3_rmsnorm_bwd", dev, stream, pdy, lddy, ps, lds, _dense(rstd, f32, dev, (rows,), "rstd"),
            _dense(gamma, f32, dev, (cols,), "gamma"), pd, ldd, px, ldx,
            _dense(dgamma, f32, dev, (cols,), "dgamma"), rows, cols, dtype, None if ws is None else ws.data_ptr())
    return dx, dgamma


def t3_gated_scan_fwd(gate, cand, h0=None, resets=None, h=None, h_last=None, stream=None):
    """(h, h_last): h_t = a_t h_(t-1) + (1 - a_t) cand_t with a_t =
    sigmoid(gate_t) over [batch][length][width], from the float state h0
    [batch][width] (None: zeros); resets uint8 or bool [batch][length] marks
    tokens that start from zero.  gate and cand may be slices of one wider tensor.
    h_last (float32 [batch][width]) may be h0: the state advances in place."""
    torch = _torch()
    dtype = _dtype_of(gate, "gate")
    shape, xt, dev, f32 = gate.shape, gate.dtype, gate.get_device(), torch.float32
    if len(shape) != 3:
        raise TypeError("gate must be 3-D [batch][length][width]")
    batch, length, width = shape
    if h is None:
        h = _empty(shape, xt, dev, stream)
    if h_last is None:
        h_last = _empty((batch, width), f32, dev, stream)
    pg, ldg = _spaced(gate, shape, "gate")
    pc, ldc = _rows(cand, xt, dev, shape, "cand")
    ph, ldh = _rows(h, xt, dev, shape, "h", out=True)
    _launch("t3_gated_scan_fwd", dev, stream, pg, ldg, pc, ldc, _dense(h0, f32, dev, (batch, width), "h0"),
            _marks(resets, dev, (batch, length)), ph, ldh,
            _dense(h_last, f32, dev, (batch, width), "h_last"), batch, length, width, dtype)
    return h, h_last


def t3_gated_scan_bwd(gate, cand, h, dh, h0=None, resets=None, dh_last=None, dgate=None, dcand=None,
                      dh0=None, stream=None):
    """(dgate, dcand, dh0): the gradient of t3_gated_scan_fwd for dh, the
    gradient of h, and dh_last (float32 [batch][width] or None), that of
    h_last; h is the forward's output."""
    torch = _torch()
    dtype = _dtype_of(gate, "gate")
    shape, xt, dev, f32 = gate.shape, gate.dtype, gate.get_device(), torch.float32
    if len(shape) != 3:
        raise TypeError("gate must be 3-D [batch][length][width]")
    batch, length, width = shape
    if dgate is None:
        dgate = _empty(shape, xt, dev, stream)
    if dcand is None:
        dcand = _empty(shape, xt, dev, stream)
    if dh0 is None:
        dh0 = _empty((batch, width), f32, dev, stream)
    pg, ldg = _spaced(gate, shape, "gate")
    pc, ldc = _rows(cand, xt, dev, shape, "cand")
    ph, ldh = _rows(h, xt, dev, shape, "h")
    pd, ldd = _rows(dh, xt, dev, shape, "dh")
    pdg, lddg = _rows(dgate, xt, dev, shape, "dgate", out=True)
    pdc, lddc = _rows(dcand, xt, dev, shape, "dcand", out=True)
    _launch("t3_gated_scan_bwd", dev, stream, pg, ldg, pc, ldc, ph, ldh, pd, ldd,
            _dense(h0, f32, dev, (batch, width), "h0"),
            _marks(resets, dev, (batch, length)),
            _dense(dh_last, f32, dev, (batch, width), "dh_last"), pdg, lddg, pdc, lddc,
            _dense(dh0, f32, dev, (batch, width), "dh0"), batch, length, width, dtype)
    return dgate, dcand, dh0


def t3_gemm_fwd_act(A, Wp, K=None, row_scale=None, col_scale=None, bias=None, act=T3_ACT_NONE,
                    residual=None, kind=T3_OUT_F32, C=None, pre=None, workspace=None, scratch=None, stream=None):
    """C = act(z) + residual with z = A . W scaled per row and column plus
    bias; `pre`, when given, receives z for t3_act_bwd.  kind: T3_OUT_F32 or
    T3_OUT_BF16, the type of C, residual and pre [M][N].  workspace: int32
    [M][N] where t3_gemm_fwd_act_workspace asks for one, and scratch: uint8 of t3_gemm_fwd_act_scratch_now(M, N, K), are allocated
    where none is given."""
    torch = _torch()
    if not isinstance(A, torch.Tensor) or not A.is_cuda or A.dim() != 2 or Wp.dim() != 2:
        raise TypeError("A and Wp must be 2-D CUDA tensors")
    M, Ka = A.shape
    N, KB = Wp.shape
    K = Ka if K is None else K
    if Ka != K or KB != (K + 3) // 4:
        raise ValueError("A must be [M][K] and Wp [N][ceil(K/4)]")
    if kind not in (T3_OUT_F32, T3_OUT_BF16):
        raise ValueError(f"unknown output kind {kind}")
    dev, f32, shape = A.get_device(), torch.float32, (M, N)
    dtype = torch.bfloat16 if kind == T3_OUT_BF16 else f32
    if C is None:
        C = _empty(shape, dtype, dev, stream)
    room = 0
    if scratch is not None:
        room = scratch.numel()
        ps = _dense(scratch, torch.uint8, dev, (room,), "scratch")
        if ps % 16:
            room = 0  # the library does not use it either
    else:
        ps = None
        if M > 32 and (K % 64 or N % 8):
            room = load().t3_gemm_fwd_act_scratch_now(M, N, K)
            if room:
                scratch = _empty(room, torch.uint8, dev, stream)
                ps = scratch.data_ptr()
    pa, pw, pc = _dense(A, torch.int8, dev, (M, K), "A"), _dense(Wp, torch.uint8, dev, (N, KB), "Wp"), _dense(C, dtype, dev, shape, "C")
    pr, pp = _dense(residual, dtype, dev, shape, "residual"), _dense(pre, dtype, dev, shape, "pre")
    if workspace is None and kind == T3_OUT_BF16:
        n = _on(dev, "t3_gemm_fwd_act_workspace", pa, pw, pc, M, N, K, pr, pp, kind, room)
        if n < 0:
            raise T3Error(n, "t3_gemm_fwd_act_workspace")
        if n:
            workspace = _empty(shape, torch.int32, dev, stream)
    _launch("t3_gemm_fwd_act", dev, stream, pa, pw, pc, M, N, K,
            _dense(row_scale, f32, dev, (M,), "row_scale"), _dense(col_scale, f32, dev, (N,), "col_scale"),
            _dense(bias, f32, dev, (N,), "bias"), act, pr, pp, kind,
            _dense(workspace, torch.int32, dev, shape, "workspace"), ps, room)
    return C


def t3_act_bwd(dy, z, act, dz=None, dbias=None, workspace=None, stream=None):
    """(dz, dbias): dz = dy * act'(z) and, into dbias when one is given
    (float32 [cols]), its column sums; z is t3_gemm_fwd_act's pre.  dz may be
    dy."""
    torch = _torch()
    dtype = _dtype_of(dy, "dy")
    if dy.dim() != 2:
        raise TypeError("dy must be 2-D [rows][cols]")
    shape, xt, dev = dy.shape, dy.dtype, dy.get_device()
    rows, cols = shape
    if z is None and act != T3_ACT_NONE:
        raise ValueError("z is needed for this activation")
    if dz is None:
        dz = _empty(shape, xt, dev, stream)
    ws = None if dbias is None else _workspace(workspace, rows, cols, dev, stream)
    _launch("t3_act_bwd", dev, stream, _dense(dy, xt, dev, shape, "dy"), _dense(z, xt, dev, shape, "z"), act,
            _dense(dz, xt, dev, shape, "dz"), _dense(dbias, torch.float32, dev, (cols,), "dbias"), rows, cols, dtype,
            None if ws is None else ws.data_ptr())
    return dz, dbias


def t3_last_device_error(stream=None):
    """(status, detail): T3_ETIMEOUT and the recorded code if a bounded device
    wait gave up since the last call; synchronizes the stream."""
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    detail = ctypes.c_int32(0)
    rc = load().t3_last_device_error(ctypes.c_void_p(s.cuda_stream), ctypes.byref(detail))
    return rc, detail.value


def t3_set_small_product_limit(macs: int) -> int:
    """Products of at most `macs` multiply-adds (macs / 8 when every operand's
    rows are 4-byte aligned) run on the CUDA cores, larger ones on the tensor
    cores (default 2**29; 0: always the tensor cores).  Returns the previous
    limit."""
    return int(load().t3_set_small_product_limit(int(macs)))


def t3_selftest_wait_timeout(limit_ns: int, stream=None):
    """Launches the bounded-wait self-test: one CTA waits on a barrier that
    nothing completes and gives up after limit_ns of device time, recording
    its code for t3_last_device_error."""
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(load().t3_selftest_wait_timeout(int(limit_ns), ctypes.c_void_p(s.cuda_stream)),
           "t3_selftest_wait_timeout")


def t3_selftest_scan_wait_timeout(limit_ns: int, stream=None):
    """The same for the recurrence's wait on the other CTAs of a cluster."""
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    _check(load().t3_selftest_scan_wait_timeout(int(limit_ns), ctypes.c_void_p(s.cuda_stream)),
           "t3_selftest_scan_wait_timeout")


def t3_version() -> int:
    return load().t3_version()
