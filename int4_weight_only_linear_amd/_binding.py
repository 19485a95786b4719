"""ctypes binding of libw4a16 (include/w4a16.h).

Argument marshalling only: shapes, dtypes and pointers are read off torch
tensors (device memory) or numpy arrays (host memory) and handed to the C
entry points of the same names; every step of the computation runs in the
library.  There is no fallback: if libw4a16.so is missing or fails to load,
importing this module raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libw4a16.so")

W4A16_OK = 0
W4A16_F16 = 0
W4A16_BF16 = 1
W4A16_F32 = 2
W4A16_E4M3 = 3
W4A16_E8M0 = 4
SCORES = {"softmax": 0, "sigmoid": 1}
PATH_AUTO, PATH_GEMV, PATH_GEMM = 0, 1, 2
GEMV_MAX_M = 16
ABI_VERSION = 4

STATUS_NAMES = {
    0: "W4A16_OK", 1: "W4A16_ERR_INVALID_ARG", 2: "W4A16_ERR_UNSUPPORTED",
    3: "W4A16_ERR_ALIGNMENT", 4: "W4A16_ERR_DEVICE", 5: "W4A16_ERR_LAUNCH",
    6: "W4A16_ERR_WORKSPACE",
}

# the exported symbols of include/w4a16.h: name -> (restype, argtypes)
_c_int, _c_i32, _c_i64, _c_sz, _vp = ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p
SIGNATURES = {
    "w4a16_abi_version": (_c_int, []),
    "w4a16_reload_tuning": (None, []),
    "w4a16_last_error": (ctypes.c_char_p, []),
    "w4a16_pack_weights": (_c_int, [_vp, _c_i64, _c_i64, _vp]),
    "w4a16_unpack_weights": (_c_int, [_vp, _c_i64, _c_i64, _vp]),
    "w4a16_pack_zeros": (_c_int, [_vp, _c_i64, _c_i64, _vp]),
    "w4a16_unpack_zeros": (_c_int, [_vp, _c_i64, _c_i64, _vp]),
    "w4a16_check_args": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32]),
    "w4a16_select_path": (_c_int, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32]),
    "w4a16_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32]),
    "w4a16_linear": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32,
                              _vp, _c_sz, _vp]),
    "w4a16_linear_path": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32,
                                   _c_i32, _vp, _c_sz, _vp, _c_i32]),
    "w4a16_linear_noalloc": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32,
                                      _c_i32, _vp]),
    "w4a16_dequant": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i32, _c_i32, _vp]),
    "w4a16_unpack_device": (_c_int, [_vp, _vp, _c_i64, _c_i64, _vp]),
    "w4a16_linear_dense": (_c_int, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _vp, _c_sz,
                                    _vp]),
    "w4a16_dense_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32]),
    "w4a16_lora_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i64, _c_i32]),
    "w4a16_lora_linear": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64,
                                   _c_i64, _c_i32, _c_i64, _c_i64, _c_i32, _vp, _c_sz, _vp]),
    "w4a16_lora_backward_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i64, _c_i64, _c_i32]),
    "w4a16_lora_backward": (_c_int, [_vp] * 13 + [_c_i64, _c_i64, _c_i64, _c_i32, _c_i64, _c_i64, _c_i32, _vp, _c_sz, _vp]),
    "w4a16_moe_linear": (_c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64,
                                  _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _vp]),
}


class PlanInfo(ctypes.Structure):
    """w4a16_plan_info (include/w4a16.h)."""
    _fields_ = [("path", ctypes.c_int32), ("tile_features", ctypes.c_int32),
                ("tile_tokens", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("tiles", ctypes.c_int64), ("counter_tiles", ctypes.c_int64),
                ("launches", ctypes.c_int32), ("waves", ctypes.c_int32),
                ("two_pass", ctypes.c_int32), ("kernel", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_uint64), ("tail_tile_tokens", ctypes.c_int32),
                ("tail_tile_features", ctypes.c_int32), ("tail_tiles", ctypes.c_int64)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


SIGNATURES["w4a16_plan"] = (_c_int, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32,
                                     ctypes.POINTER(PlanInfo)])


class AdamwTensor(ctypes.Structure):
    """w4a16_adamw_tensor (include/w4a16.h)."""
    _fields_ = [("param", _vp), ("grad", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp),
                ("copy", _vp), ("n", _c_i64)]


class AdamwPlanInfo(ctypes.Structure):
    """w4a16_adamw_plan (include/w4a16.h)."""
    _fields_ = [("tensors", _c_i64), ("chunks", _c_i64), ("blocks", _c_i64), ("state_bits", _c_i32),
                ("param_dtype", _c_i32), ("grad_dtype", _c_i32), ("reserved", _c_i32)]


_c_dbl = ctypes.c_double
SIGNATURES["w4a16_adamw_table_size"] = (_c_sz, [ctypes.POINTER(AdamwTensor), _c_i64])
SIGNATURES["w4a16_adamw_table"] = (_c_int, [ctypes.POINTER(AdamwTensor), _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _vp,
                                            _c_sz, ctypes.POINTER(AdamwPlanInfo)])
SIGNATURES["w4a16_adamw_step"] = (_c_int, [_vp, ctypes.POINTER(AdamwPlanInfo), _c_dbl, _c_dbl, _c_dbl, _c_dbl, _c_dbl,
                                           _c_i64, _c_dbl, ctypes.c_uint32, _vp])
SIGNATURES["w4a16_adamw_moments"] = (_c_int, [_vp, ctypes.POINTER(AdamwPlanInfo), _vp, _vp, _vp])


SIGNATURES["w4a16_route"] = (_c_int, [_vp] * 4 + [_c_i64] * 6 + [_c_i32, _c_i32, _c_i32, _c_dbl, _vp])
SIGNATURES["w4a16_route_backward"] = (_c_int, [_vp] * 4 + [_c_i64] * 3 + [_c_i32, _c_i32, _c_i32, _c_dbl, _vp])
SIGNATURES["w4a16_minifloat_quantize"] = (_c_int, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i32, _vp])
SIGNATURES["w4a16_minifloat_linear_workspace_size"] = (_c_sz, [_c_i64, _c_i64, _c_i64, _c_i32, _c_i32])
SIGNATURES["w4a16_minifloat_linear"] = (_c_int, [_vp] * 6 + [_c_i64] * 3 + [_c_i32] * 4 + [_vp, _c_sz, _vp])
SIGNATURES["w4a16_minifloat_moe_workspace_size"] = (_c_sz, [_c_i64] * 5 + [_c_i32] * 3)
SIGNATURES["w4a16_minifloat_moe_linear"] = (_c_int, [_vp] * 8 + [_c_i64] * 5 + [_c_i32] * 5 + [_vp, _c_sz, _vp])


class W4A16Error(RuntimeError):
    """A libw4a16 call returned a non-zero status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{message} [{STATUS_NAMES.get(status, status)}]")
        self.status = status
        self.message = message


def _load():
    # One HIP runtime per process: when PyTorch is present, let it load its
    # own libamdhip64 first so that libw4a16's dependency (same soname)
    # resolves to that copy instead of a second runtime from /opt/rocm.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run int4_weight_only_linear_amd.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.w4a16_abi_version() != ABI_VERSION:
        raise ImportError(f"libw4a16 ABI {lib.w4a16_abi_version()} != binding ABI {ABI_VERSION}")
    return lib


lib = _load()


def _check(status: int):
    if status != W4A16_OK:
        raise W4A16Error(status, lib.w4a16_last_error().decode())


def w4a16_abi_version() -> int:
    return lib.w4a16_abi_version()


def w4a16_last_error() -> str:
    return lib.w4a16_last_error().decode()


def w4a16_reload_tuning() -> None:
    """Re-read the tuning environment variables (the library reads them once)."""
    lib.w4a16_reload_tuning()
    _sizes.clear()


# ------------------------------------------------------------------ host ---

def _host(a, dtype) -> np.ndarray:
    a = np.ascontiguousarray(a)
    if a.dtype != dtype:
        raise TypeError(f"expected {np.dtype(dtype)}, got {a.dtype}")
    return a


def w4a16_pack_weights(q: np.ndarray) -> np.ndarray:
    """uint8 [N, K] codes (0..15) -> int32 [N, K/8] words."""
    q = _host(q, np.uint8)
    N, K = q.shape
    out = np.empty((N, K // 8 if K % 8 == 0 else 0), dtype=np.int32)
    _check(lib.w4a16_pack_weights(q.ctypes.data, N, K, out.ctypes.data))
    return out


def w4a16_unpack_weights(wq: np.ndarray, K: int | None = None) -> np.ndarray:
    """int32/uint32 [N, K/8] words -> uint8 [N, K] codes."""
    wq = np.ascontiguousarray(wq)
    if wq.dtype not in (np.int32, np.uint32):
        raise TypeError(f"weights must be int32 or uint32, got {wq.dtype}")
    N = wq.shape[0]
    K = wq.shape[1] * 8 if K is None else K
    out = np.empty((N, K), dtype=np.uint8)
    _check(lib.w4a16_unpack_weights(wq.ctypes.data, N, K, out.ctypes.data))
    return out


def w4a16_pack_zeros(z: np.ndarray) -> np.ndarray:
    """uint8 [N, G] zero points -> int32 [N/8, G] words."""
    z = _host(z, np.uint8)
    N, G = z.shape
    out = np.empty((N // 8 if N % 8 == 0 else 0, G), dtype=np.int32)
    _check(lib.w4a16_pack_zeros(z.ctypes.data, N, G, out.ctypes.data))
    return out


def w4a16_unpack_zeros(zpk: np.ndarray, N: int | None = None) -> np.ndarray:
    """int32/uint32 [N/8, G] words -> uint8 [N, G] zero points."""
    zpk = np.ascontiguousarray(zpk)
    if zpk.dtype not in (np.int32, np.uint32):
        raise TypeError(f"zero points must be int32 or uint32, got {zpk.dtype}")
    N = zpk.shape[0] * 8 if N is None else N
    G = zpk.shape[1]
    out = np.empty((N, G), dtype=np.uint8)
    _check(lib.w4a16_unpack_zeros(zpk.ctypes.data, N, G, out.ctypes.data))
    return out


def w4a16_select_path(M, N, K, group_size, dtype, has_zp) -> int:
    return int(lib.w4a16_select_path(M, N, K, group_size, dtype, int(bool(has_zp))))


def w4a16_workspace_size(M, N, K, group_size, dtype, has_zp, path=PATH_AUTO) -> int:
    return int(lib.w4a16_workspace_size(M, N, K, group_size, dtype, int(bool(has_zp)), path))


def w4a16_plan(M, N, K, group_size, dtype, has_zp, path=PATH_AUTO) -> dict:
    """How the library would run this problem (host only): path, tile shape,
    output tiles, K splits, launches, waves, workspace bytes."""
    info = PlanInfo()
    _check(lib.w4a16_plan(M, N, K, group_size, dtype, int(bool(has_zp)), path, ctypes.byref(info)))
    return info.as_dict()


def w4a16_check_args(x_ptr, wq_ptr, s_ptr, zp_ptr, bias_ptr, y_ptr, M, N, K, group_size, dtype):
    """Raw-pointer argument check (no device access); raises W4A16Error."""
    _check(lib.w4a16_check_args(x_ptr, wq_ptr, s_ptr, zp_ptr, bias_ptr, y_ptr, M, N, K,
                                group_size, dtype))


# ---------------------------------------------------------------- device ---

_ZP_MSG = "Zero points must be int32 or uint32 (packed 8x uint4 along dim 0), got {}"


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _act_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float16:
        return W4A16_F16
    if t.dtype == torch.bfloat16:
        return W4A16_BF16
    raise TypeError(f"activations must be float16 or bfloat16, got {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _require_device(t, name, device):
    if t is None:
        return
    if not t.is_cuda or t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _require_all(device, *named):
    """_require_device for (tensor, name) pairs: one pass over those that pass."""
    index = device.index
    for t, name in named:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            _require_device(t, name, device)


def _invoke(device, fn, *args):
    """Call a device entry point with `device` current (it mostly is already:
    the check costs a tenth of a device guard) and raise on its error."""
    torch = _torch()
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    if status != W4A16_OK:
        _check(status)


def _raw_stream(device) -> int:
    """The current stream's handle, without building a Stream object."""
    return _torch()._C._cuda_getCurrentRawStream(device.index)


# workspace sizes by (entry point, device, sizes): the plan behind one is the
# same for every call of these sizes until the tuning variables are read again.
# A serving process meets many token counts: started afresh at this many.
_SIZES_MAX = 4096
_sizes: dict = {}


def _size_of(device, fn, *args) -> int:
    key = (fn.__name__, device.index, args)
    n = _sizes.get(key)
    if n is None:
        torch = _torch()
        with torch.cuda.device(device):
            n = int(fn(*args))
        if len(_sizes) >= _SIZES_MAX:
            _sizes.clear()
        _sizes[key] = n
    return n


_ws_lock = threading.Lock()
_ws_cache: dict = {}


def _workspace(device, stream_ptr: int, nbytes: int):
    """A zero-filled buffer of at least nbytes, reused per (device, stream).

    Calls on one stream run in order, and every call leaves the buffer's
    counters zero again, so reuse across calls on the same stream is safe.
    """
    if nbytes == 0:
        return None
    torch = _torch()
    key = (device.index, stream_ptr)
    with _ws_lock:
        buf = _ws_cache.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
            _ws_cache[key] = buf
        return buf


def _given_workspace(device, workspace):
    """(the pointer, the bytes) of a caller's workspace, which must lie on `device`: its pointer
    goes to kernels; contiguous, since an expanded tensor has fewer bytes than elements."""
    _require_device(workspace, "workspace", device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _own_workspace(device, stream_ptr: int, nbytes: int):
    """(the pointer, the bytes) of the workspace kept for the device and stream."""
    workspace = _workspace(device, stream_ptr, nbytes)
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())


def _linear_args(x, wq, scales, zp, bias, group_size, out):
    torch = _torch()
    dtype = x.dtype
    dt = _act_code(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    words = (torch.int32, getattr(torch, "uint32", torch.int32))
    if wq.dim() != 2 or wq.dtype not in words:
        raise TypeError(f"wq must be a 2-D int32 or uint32 tensor, got {wq.dtype}")
    N, J = wq.shape
    if J * 8 != K:
        raise ValueError(f"wq is {tuple(wq.shape)}, expected [N, K/8] with K={K}")
    if scales.dtype != dtype:
        raise TypeError(f"scales must be {dtype}, got {scales.dtype}")
    if group_size <= 0 or K % group_size:
        raise ValueError(f"K={K} is not a multiple of group_size={group_size}")
    G = K // group_size
    if scales.shape != (N, G):
        raise ValueError(f"scales are {tuple(scales.shape)}, expected {(N, G)}")
    if zp is not None:
        if zp.dtype not in words:
            raise RuntimeError(_ZP_MSG.format(zp.dtype))
        if zp.shape != (N // 8, G) or N % 8:
            raise ValueError(f"zp is {tuple(zp.shape)}, expected {(N // 8, G)} (N % 8 == 0)")
    if bias is not None:
        if bias.dtype != dtype or bias.shape != (N,):
            raise ValueError(f"bias must be {dtype} [{N}]")
    device = x.device
    _require_device(x, "x", device)
    _require_all(device, (wq, "wq"), (scales, "scales"), (zp, "zp"), (bias, "bias"))
    if out is None:
        out = x.new_empty((M, N))
    else:
        if out.dtype != dtype or out.shape != (M, N):
            raise ValueError(f"out must be {dtype} [{M}, {N}]")
        _require_device(out, "out", device)
    return dt, M, N, K, out


def w4a16_linear_path(x, wq, scales, zp=None, bias=None, *, group_size: int, path: int = PATH_AUTO,
                      out=None, workspace=None):
    """y = x . dequant(wq, scales, zp)^T (+ bias) on x's device and current stream."""
    torch = _torch()
    dt, M, N, K, out = _linear_args(x, wq, scales, zp, bias, group_size, out)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        need = w4a16_workspace_size(M, N, K, group_size, dt, zp is not None, path)
        ws_ptr, ws_bytes = (_own_workspace(x.device, stream, need) if workspace is None
                            else _given_workspace(x.device, workspace))
        _check(lib.w4a16_linear_path(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), _ptr(zp),
                                     _ptr(bias), out.data_ptr(), M, N, K, group_size, dt, ws_ptr,
                                     ws_bytes, stream, path))
    return out


def w4a16_linear(x, wq, scales, zp=None, bias=None, *, group_size: int, out=None, workspace=None):
    """w4a16_linear_path with the library's own choice of kernel."""
    return w4a16_linear_path(x, wq, scales, zp, bias, group_size=group_size, path=PATH_AUTO,
                             out=out, workspace=workspace)


NOALLOC_SCRATCH_BYTES = 64 << 20


def w4a16_linear_noalloc(x, wq, scales, zp=None, bias=None, *, group_size: int, out):
    """w4a16_linear without a workspace: a K split uses the library's own
    per-GPU scratch (calls that overlap on one GPU race).  `out` is required,
    so that the call allocates nothing."""
    torch = _torch()
    dt, M, N, K, out = _linear_args(x, wq, scales, zp, bias, group_size, out)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        _check(lib.w4a16_linear_noalloc(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), _ptr(zp),
                                        _ptr(bias), out.data_ptr(), M, N, K, group_size, dt, stream))
    return out


def w4a16_dequant(wq, scales, zp=None, *, group_size: int, out=None):
    """Dequantised weights [N, K] in the scales' dtype, rounded once to nearest-even."""
    torch = _torch()
    dt = _act_code(scales)
    N, K = wq.shape[0], wq.shape[1] * 8
    if zp is not None and zp.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32)):
        raise RuntimeError(_ZP_MSG.format(zp.dtype))
    for t, name in ((wq, "wq"), (scales, "scales"), (zp, "zp")):
        _require_device(t, name, wq.device)
    if out is None:
        out = torch.empty((N, K), dtype=scales.dtype, device=wq.device)
    stream = torch.cuda.current_stream(wq.device).cuda_stream
    with torch.cuda.device(wq.device):
        _check(lib.w4a16_dequant(wq.data_ptr(), scales.data_ptr(), _ptr(zp), out.data_ptr(), N, K,
                                 group_size, dt, stream))
    return out


def w4a16_unpack_device(wq, out=None):
    """uint8 codes [N, K] unpacked on the device."""
    torch = _torch()
    N, K = wq.shape[0], wq.shape[1] * 8
    _require_device(wq, "wq", wq.device)
    if out is None:
        out = torch.empty((N, K), dtype=torch.uint8, device=wq.device)
    stream = torch.cuda.current_stream(wq.device).cuda_stream
    with torch.cuda.device(wq.device):
        _check(lib.w4a16_unpack_device(wq.data_ptr(), out.data_ptr(), N, K, stream))
    return out


def w4a16_dense_workspace_size(M, N, K, dtype, has_bias) -> int:
    return int(lib.w4a16_dense_workspace_size(M, N, K, dtype, int(bool(has_bias))))


def w4a16_linear_dense(x, w, bias=None, *, out=None, workspace=None):
    """y = x . w^T (+ bias) with w the dequantised weights [N, K] (w4a16_dequant),
    on x's device and current stream."""
    torch = _torch()
    dt = _act_code(x)
    if x.dim() != 2 or w.dim() != 2 or w.shape[1] != x.shape[1]:
        raise ValueError(f"x must be [M, K] and w [N, K], got {tuple(x.shape)} and {tuple(w.shape)}")
    if w.dtype != x.dtype or (bias is not None and bias.dtype != x.dtype):
        raise TypeError("x, w and bias must share one dtype")
    M, K = x.shape
    N = w.shape[0]
    if bias is not None and tuple(bias.shape) != (N,):
        raise ValueError(f"bias must be [{N}]")
    for t, name in ((x, "x"), (w, "w"), (bias, "bias")):
        _require_device(t, name, x.device)
    if out is None:
        out = torch.empty((M, N), dtype=x.dtype, device=x.device)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        need = w4a16_dense_workspace_size(M, N, K, dt, bias is not None)
        ws_ptr, ws_bytes = (_own_workspace(x.device, stream, need) if workspace is None
                            else _given_workspace(x.device, workspace))
        _check(lib.w4a16_linear_dense(x.data_ptr(), w.data_ptr(), _ptr(bias), out.data_ptr(), M, N, K,
                                      dt, ws_ptr, ws_bytes, stream))
    return out


def w4a16_moe_linear(x, wq, scales, topk_ids, zp=None, bias=None, topk_weights=None, *,
                     group_size: int, x_per_slot: bool = False, out=None):
    """Expert-indexed decode: y[m*topk + j] = topk_weights[m, j] * (x_row . W_e^T + b_e),
    e = topk_ids[m, j], with stacks wq [E, N, K/8], scales [E, N, G], zp [E, N/8, G],
    bias [E, N]; x is [M, K] (or [M*topk, K] with x_per_slot).  Returns [M*topk, N]."""
    torch = _torch()
    dt = _act_code(x)
    if wq.dim() != 3:
        raise ValueError("wq must be [E, N, K/8]")
    E, N, K = wq.shape[0], wq.shape[1], wq.shape[2] * 8
    if topk_ids.dim() != 2 or topk_ids.dtype != torch.int32:
        raise TypeError("topk_ids must be int32 [M, topk]")
    M, topk = topk_ids.shape
    if x.dim() != 2 or x.shape[1] != K or x.shape[0] != (M * topk if x_per_slot else M):
        raise ValueError(f"x is {tuple(x.shape)}, expected [{M * topk if x_per_slot else M}, {K}]")
    if group_size <= 0 or K % group_size:
        raise ValueError(f"K={K} is not a multiple of group_size={group_size}")
    G = K // group_size
    if scales.dtype != x.dtype or tuple(scales.shape) != (E, N, G):
        raise ValueError(f"scales must be {x.dtype} {(E, N, G)}")
    if zp is not None and (zp.dtype not in (torch.int32, getattr(torch, "uint32", torch.int32))
                           or tuple(zp.shape) != (E, N // 8, G)):
        raise ValueError(f"zp must be int32 {(E, N // 8, G)}")
    if bias is not None and (bias.dtype != x.dtype or tuple(bias.shape) != (E, N)):
        raise ValueError(f"bias must be {x.dtype} {(E, N)}")
    if topk_weights is not None and (topk_weights.dtype != torch.float32
                                     or tuple(topk_weights.shape) != (M, topk)):
        raise ValueError(f"topk_weights must be float32 {(M, topk)}")
    for t, name in ((x, "x"), (wq, "wq"), (scales, "scales"), (zp, "zp"), (bias, "bias"),
                    (topk_ids, "topk_ids"), (topk_weights, "topk_weights")):
        _require_device(t, name, x.device)
    if out is None:
        out = torch.empty((M * topk, N), dtype=x.dtype, device=x.device)
    stream = torch.cuda.current_stream(x.device).cuda_stream
    with torch.cuda.device(x.device):
        _check(lib.w4a16_moe_linear(x.data_ptr(), wq.data_ptr(), scales.data_ptr(), _ptr(zp), _ptr(bias),
                                    topk_ids.data_ptr(), _ptr(topk_weights), out.data_ptr(), M, topk, E,
                                    N, K, group_size, dt, int(bool(x_per_slot)), stream))
    return out


# ------------------------------------------------------ low-rank adapters ---

def w4a16_lora_workspace_size(M, N, K, group_size, dtype, has_zp, R, save_u=False) -> int:
    return int(lib.w4a16_lora_workspace_size(M, N, K, group_size, dtype, int(bool(has_zp)), R, int(bool(save_u))))


def _adapter_args(x, la, lb, ids, alpha, M, N, K):
    torch = _torch()
    if la.dim() != 3 or la.shape[2] != K:
        raise ValueError(f"la is {tuple(la.shape)}, expected [S, R, {K}]")
    S, R, _ = la.shape
    if lb.shape != (S, N, R):
        raise ValueError(f"lb is {tuple(lb.shape)}, expected {(S, N, R)}")
    if la.dtype != x.dtype or lb.dtype != x.dtype:
        raise TypeError(f"la and lb must be {x.dtype}, got {la.dtype} and {lb.dtype}")
    if ids.dtype != torch.int32 or ids.shape != (M,):
        raise TypeError(f"ids must be int32 [{M}], got {ids.dtype} {tuple(ids.shape)}")
    if alpha is not None and (alpha.dtype != torch.float32 or alpha.shape != (S,)):
        raise TypeError(f"alpha must be float32 [{S}]")
    _require_all(x.device, (la, "la"), (lb, "lb"), (ids, "ids"), (alpha, "alpha"))
    return S, R


def w4a16_lora_linear(x, wq, scales, la, lb, ids, zp=None, bias=None, alpha=None, *, group_size: int,
                      save_u: bool = False, out=None, workspace=None):
    """y = x . dequant(wq, scales, zp)^T (+ bias) + alpha_a * (x . A_a^T) . B_a^T with token
    m's adapter a = ids[m] out of the stacks la [S, R, K] and lb [S, N, R] (an id outside
    [0, S): no adapter).  With save_u returns (y, u), u = x . A_a^T in float32 [M, R] for
    w4a16_lora_backward.  Not recorded by autograd: y requires no gradient, whatever la, lb
    and x do; a training step calls w4a16_lora_backward itself.  workspace: zero-filled uint8 of
    w4a16_lora_workspace_size; without one a buffer kept per stream is used, which a later, larger
    call replaces, so calls captured in a graph bring their own."""
    torch = _torch()
    dt, M, N, K, out = _linear_args(x, wq, scales, zp, bias, group_size, out)
    S, R = _adapter_args(x, la, lb, ids, alpha, M, N, K)
    device = x.device
    u = torch.empty((M, R), dtype=torch.float32, device=device) if save_u else None
    stream = _raw_stream(device)
    ws_ptr, ws_bytes = (_own_workspace(device, stream, _size_of(device, lib.w4a16_lora_workspace_size, M, N, K, group_size, dt,
                                                                int(zp is not None), R, int(save_u)))
                        if workspace is None else _given_workspace(device, workspace))
    _invoke(device, lib.w4a16_lora_linear, x.data_ptr(), wq.data_ptr(), scales.data_ptr(), _ptr(zp), _ptr(bias),
            la.data_ptr(), lb.data_ptr(), ids.data_ptr(), _ptr(alpha), out.data_ptr(), _ptr(u), M, N, K, group_size, S, R,
            dt, ws_ptr, ws_bytes, stream)
    return (out, u) if save_u else out


def w4a16_lora_backward_workspace_size(M, N, K, group_size, S, R, dtype) -> int:
    return int(lib.w4a16_lora_backward_workspace_size(M, N, K, group_size, S, R, dtype))


def w4a16_lora_backward(dy, x, u, wq, scales, la, lb, ids, zp=None, alpha=None, *, group_size: int,
                        need_dx: bool = True, out=None, workspace=None):
    """Gradients of w4a16_lora_linear: (dx, dla, dlb) for dy [M, N], with x and the u that the
    forward call kept (save_u).  dx is None where need_dx is false.  out: (dx or None, dla, dlb)
    to write into: overwritten, not added to.  workspace: as for w4a16_lora_linear, of
    w4a16_lora_backward_workspace_size."""
    torch = _torch()
    if dy.dim() != 2 or x.dim() != 2 or dy.shape[0] != x.shape[0] or dy.shape[1] != wq.shape[0]:
        raise ValueError(f"dy is {tuple(dy.shape)}, expected {(x.shape[0], wq.shape[0])}")
    if dy.dtype != x.dtype:
        raise TypeError(f"dy must be {x.dtype}, got {dy.dtype}")
    # the projection's own checks (dy stands where its output would)
    dt, M, N, K, _ = _linear_args(x, wq, scales, zp, None, group_size, dy)
    S, R = _adapter_args(x, la, lb, ids, alpha, M, N, K)
    device = x.device
    if u.dtype != torch.float32 or u.shape != (M, R):
        raise TypeError(f"u must be float32 {(M, R)}, got {u.dtype} {tuple(u.shape)}")
    _require_device(u, "u", device)
    if out is None:
        dx, dla, dlb = torch.empty_like(x) if need_dx else None, torch.empty_like(la), torch.empty_like(lb)
    else:
        dx, dla, dlb = out
        if dla is None or dlb is None:
            raise ValueError("dla and dlb must be given")
        for t, like, name in ((dx, x, "dx"), (dla, la, "dla"), (dlb, lb, "dlb")):
            if t is not None and (t.dtype != x.dtype or t.shape != like.shape):
                raise ValueError(f"{name} must be {x.dtype} {tuple(like.shape)}")
            _require_device(t, name, device)
    stream = _raw_stream(device)
    ws_ptr, ws_bytes = (_own_workspace(device, stream, _size_of(device, lib.w4a16_lora_backward_workspace_size, M, N, K, group_size,
                                                                S, R, dt))
                        if workspace is None else _given_workspace(device, workspace))
    _invoke(device, lib.w4a16_lora_backward, dy.data_ptr(), x.data_ptr(), u.data_ptr(), wq.data_ptr(), scales.data_ptr(),
            _ptr(zp), la.data_ptr(), lb.data_ptr(), ids.data_ptr(), _ptr(alpha), _ptr(dx), dla.data_ptr(), dlb.data_ptr(),
            M, N, K, group_size, S, R, dt, ws_ptr, ws_bytes, stream)
    return dx, dla, dlb


# ---------------------------------------------------------------- AdamW ---

class AdamwPlan:
    """The table of a list of tensors on their device, with the tensors it names."""

    def __init__(self, info, table, tensors, device):
        self.info, self.table, self.tensors, self.device = info, table, tensors, device
        self.info_ref = ctypes.byref(info)

    @property
    def state_bits(self) -> int:
        return self.info.state_bits

    @property
    def blocks(self) -> int:
        """256-element blocks over all tensors."""
        return self.info.blocks


def _float_code(t, name) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return W4A16_F32
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be float16, bfloat16 or float32, got {t.dtype}")
    return _act_code(t)


def w4a16_adamw_plan(params, grads, exp_avgs, exp_avg_sqs, *, m_scales=None, v_scales=None, copies=None) -> AdamwPlan:
    """Lays out the table for w4a16_adamw_step over lists of tensors of equal length.

    exp_avgs / exp_avg_sqs are float32 (moments in 32 bits), or int8 / uint8 with
    m_scales / v_scales float32 [ceil(n / 256)] (moments in 8 bits; zeros to begin
    with).  copies: float16 or bfloat16 copies of the parameters, written by every
    step (None for a parameter that has none).  The plan keeps the tensors, and every
    step reads and writes them where they are now: gradients that are allocated anew
    (set to None between steps) need a new plan, or are copied into the plan's."""
    torch = _torch()
    params, grads, ms, vs = list(params), list(grads), list(exp_avgs), list(exp_avg_sqs)
    count = len(params)
    if count == 0:
        raise ValueError("need at least one tensor")
    eight = m_scales is not None or v_scales is not None
    if eight and (m_scales is None or v_scales is None):
        raise ValueError("moments in 8 bits need both m_scales and v_scales")
    msc, vsc = (list(m_scales), list(v_scales)) if eight else ([None] * count, [None] * count)
    cps = [None] * count if copies is None else list(copies)
    for name, got in (("grads", grads), ("exp_avgs", ms), ("exp_avg_sqs", vs), ("m_scales", msc), ("v_scales", vsc),
                      ("copies", cps)):
        if len(got) != count:
            raise ValueError(f"{len(got)} {name} for {count} params")
    device = params[0].device
    copy_type = next((c.dtype for c in cps if c is not None), None)  # any of them may be None
    want_m, want_v = (torch.int8, torch.uint8) if eight else (torch.float32, torch.float32)
    rows = (AdamwTensor * count)()
    for i, (p, g, m, v, a, b, c) in enumerate(zip(params, grads, ms, vs, msc, vsc, cps)):
        n = p.numel()
        if p.dtype != params[0].dtype or g.dtype != grads[0].dtype or (c is not None and c.dtype != copy_type):
            raise TypeError(f"tensor {i}: all tensors of a plan share their types")
        if m.dtype != want_m or v.dtype != want_v:
            raise TypeError(f"tensor {i}: moments must be {want_m} and {want_v}, got {m.dtype} and {v.dtype}")
        if g.numel() != n or m.numel() != n or v.numel() != n or (c is not None and c.numel() != n):
            raise ValueError(f"tensor {i}: sizes differ")
        if eight and (a.dtype != torch.float32 or b.dtype != torch.float32 or a.numel() != (n + 255) // 256
                      or b.numel() != (n + 255) // 256):
            raise ValueError(f"tensor {i}: scales must be float32 [{(n + 255) // 256}]")
        for t, name in ((p, "param"), (g, "grad"), (m, "exp_avg"), (v, "exp_avg_sq"), (a, "m_scale"), (b, "v_scale"),
                        (c, "copy")):
            _require_device(t, f"tensor {i}: {name}", device)
        rows[i] = AdamwTensor(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(), _ptr(a), _ptr(b), _ptr(c), n)
    copy_dtype = W4A16_BF16 if copy_type is None else _act_code(next(c for c in cps if c is not None))
    size = int(lib.w4a16_adamw_table_size(rows, count))
    host = np.zeros((size + 7) // 8, dtype=np.int64)
    info = AdamwPlanInfo()
    _check(lib.w4a16_adamw_table(rows, count, 8 if eight else 32, _float_code(params[0], "params"),
                                 _float_code(grads[0], "grads"), copy_dtype, host.ctypes.data, size, ctypes.byref(info)))
    table = torch.from_numpy(host).to(device)
    return AdamwPlan(info, table, (params, grads, ms, vs, msc, vsc, cps), device)


def w4a16_adamw_step(plan: AdamwPlan, *, lr: float, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 0.0,
                     step: int, grad_scale: float = 1.0, seed: int = 0) -> None:
    """One AdamW step (number `step`, from 1) over the plan's tensors, on the current stream.
    Moments in 8 bits are rounded with a dither that seed chooses: give every step another.
    A captured graph repeats the numbers it was captured with."""
    _invoke(plan.device, lib.w4a16_adamw_step, plan.table.data_ptr(), plan.info_ref, lr, betas[0], betas[1], eps,
            weight_decay, step, grad_scale, seed & 0xFFFFFFFF, _raw_stream(plan.device))


def w4a16_adamw_moments(plan: AdamwPlan, m=None, v=None):
    """The moments that a plan's 8-bit codes stand for: two float32 tensors [blocks * 256], the
    tensors' blocks one after another, zeros past each tensor's last element."""
    torch = _torch()
    if m is None:
        m = torch.empty(plan.blocks * 256, dtype=torch.float32, device=plan.device)
    if v is None:
        v = torch.empty(plan.blocks * 256, dtype=torch.float32, device=plan.device)
    for t, name in ((m, "m"), (v, "v")):
        if t.dtype != torch.float32 or t.shape != (plan.blocks * 256,):
            raise ValueError(f"{name} must be float32 [{plan.blocks * 256}]")
        _require_device(t, name, plan.device)
    _invoke(plan.device, lib.w4a16_adamw_moments, plan.table.data_ptr(), plan.info_ref, m.data_ptr(), v.data_ptr(),
            _raw_stream(plan.device))
    return m, v


# --------------------------------------------------- routing to experts ---

def _score_code(score) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid', got {score!r}")
    return SCORES[score]


def w4a16_route(logits, topk: int, bias=None, *, score: str = "softmax", groups: int = 1, topk_groups: int = 1,
                group_top: int = 1, renormalize: bool = False, scale: float = 1.0, out=None):
    """(weights float32 [M, topk], ids int32 [M, topk]) of the topk experts of each token, from
    the router's logits [M, E] (float16, bfloat16 or float32): the largest softmax or sigmoid
    scores, plus bias (float32 [E], moves the choice only), of the topk_groups of `groups` groups
    of experts whose group_top (1 or 2) largest sum highest; ties to the lower index.  weights:
    the scores without the bias, divided by their sum with renormalize, times scale.  Experts of
    logit -inf are never chosen: id -1, weight 0 where none is left.  Not recorded by autograd:
    a training step calls w4a16_route_backward.  out: (weights, ids) to write into."""
    torch = _torch()
    code = _float_code(logits, "logits")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [M, E]")
    M, E = logits.shape
    if bias is not None and (bias.dtype != torch.float32 or bias.shape != (E,)):
        raise TypeError(f"bias must be float32 [{E}]")
    device = logits.device
    _require_device(logits, "logits", device)
    if out is None:
        weights, ids = logits.new_empty((M, topk), dtype=torch.float32), logits.new_empty((M, topk), dtype=torch.int32)
        _require_all(device, (bias, "bias"))
    else:
        weights, ids = out
        if weights.dtype != torch.float32 or ids.dtype != torch.int32 or weights.shape != (M, topk) or ids.shape != (M, topk):
            raise ValueError(f"out must be float32 and int32 {(M, topk)}")
        _require_all(device, (bias, "bias"), (weights, "weights"), (ids, "ids"))
    _invoke(device, lib.w4a16_route, logits.data_ptr(), _ptr(bias), weights.data_ptr(), ids.data_ptr(), M, E, topk, groups,
            topk_groups, group_top, code, _score_code(score), int(bool(renormalize)), scale, _raw_stream(device))
    return weights, ids


def w4a16_route_backward(dweights, logits, ids, *, score: str = "softmax", renormalize: bool = False, scale: float = 1.0,
                         out=None):
    """dlogits [M, E], in the logits' dtype: the gradient of w4a16_route's weights for dweights
    float32 [M, topk], with its logits and the ids that it chose.  score, renormalize and scale as
    given there."""
    torch = _torch()
    code = _float_code(logits, "logits")
    if logits.dim() != 2 or ids.dim() != 2 or ids.shape[0] != logits.shape[0]:
        raise ValueError(f"logits must be [M, E] and ids [M, topk], got {tuple(logits.shape)} and {tuple(ids.shape)}")
    (M, E), topk = logits.shape, ids.shape[1]
    if ids.dtype != torch.int32 or dweights.dtype != torch.float32 or dweights.shape != ids.shape:
        raise TypeError(f"dweights must be float32 and ids int32 {(M, topk)}")
    device = logits.device
    if out is None:
        out = torch.empty_like(logits)
    elif out.dtype != logits.dtype or out.shape != logits.shape:
        raise ValueError(f"out must be {logits.dtype} {tuple(logits.shape)}")
    _require_device(logits, "logits", device)
    _require_all(device, (dweights, "dweights"), (ids, "ids"), (out, "out"))
    _invoke(device, lib.w4a16_route_backward, dweights.data_ptr(), logits.data_ptr(), ids.data_ptr(), out.data_ptr(), M, E,
            topk, code, _score_code(score), int(bool(renormalize)), scale, _raw_stream(device))
    return out


# --------------------------------------- 8-bit floating-point weights ---

def _blocks(n: int) -> int:
    return (n + 127) // 128


def w4a16_minifloat_quantize(x, *, out=None):
    """(codes float8_e4m3fn [M, K'], scales float8_e8m0fnu [M, B]) of x [M, K] (float16 or
    bfloat16): one power-of-two scale for each token and 128 k; K' is K rounded up to 128 (zeros
    behind K), B = ceil(K / 512) * 4.  out: (codes, scales) to write into."""
    torch = _torch()
    code = _act_code(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    device = x.device
    _require_device(x, "x", device)
    shapes = (M, _blocks(K) * 128), (M, (K + 511) // 512 * 4)
    if out is None:
        codes = x.new_empty(shapes[0], dtype=torch.float8_e4m3fn)
        scales = x.new_empty(shapes[1], dtype=torch.float8_e8m0fnu)
    else:
        codes, scales = out
        if codes.dtype != torch.float8_e4m3fn or scales.dtype != torch.float8_e8m0fnu or (codes.shape, scales.shape) != shapes:
            raise ValueError(f"out must be float8_e4m3fn {shapes[0]} and float8_e8m0fnu {shapes[1]}")
        _require_all(device, (codes, "codes"), (scales, "scales"))
    _invoke(device, lib.w4a16_minifloat_quantize, x.data_ptr(), codes.data_ptr(), scales.data_ptr(), M, K, code, _raw_stream(device))
    return codes, scales


def _fp8_args(x, w, scales, bias, transpose, x_scales, dtype, rows, lead):
    """Checks of both products; lead: () or (E,).  Returns (device, output dtype, its code, x's
    code, the scales' code, x's rows, N, K)."""
    torch = _torch()
    shape, s_dtype, x_dtype, x_shape = w.shape, scales.dtype, x.dtype, x.shape
    if len(shape) != 2 + len(lead) or w.dtype != torch.float8_e4m3fn:
        raise TypeError(f"w must be float8_e4m3fn with {2 + len(lead)} dimensions, got {w.dtype} {tuple(shape)}")
    if s_dtype == torch.float32:
        s_code = W4A16_F32
    elif s_dtype == torch.float8_e8m0fnu:
        s_code = W4A16_E8M0
    else:
        raise TypeError(f"scales must be float32 or float8_e8m0fnu, got {s_dtype}")
    R, C = shape[-2:]
    K, N = (R, C) if transpose else (C, R)
    expected = (*lead, (R + 127) // 128, (C + 127) // 128)
    if scales.shape != expected:
        raise ValueError(f"scales are {tuple(scales.shape)}, expected {expected}")
    if len(x_shape) != 2 or (rows is not None and x_shape[0] != rows):
        raise ValueError(f"x must be 2-D [{'M' if rows is None else rows}, K], got {tuple(x_shape)}")
    if x_dtype == torch.float8_e4m3fn:
        x_code, dtype = W4A16_E4M3, torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError(f"dtype must be float16 or bfloat16, got {dtype}")
        if x_shape[1] != _blocks(K) * 128:
            raise ValueError(f"codes are {tuple(x_shape)}, expected {_blocks(K) * 128} columns for K={K}")
        if x_scales is None or x_scales.dtype != torch.float8_e8m0fnu or x_scales.shape != (x_shape[0], (K + 511) // 512 * 4):
            raise ValueError(f"codes need x_scales, float8_e8m0fnu {(x_shape[0], (K + 511) // 512 * 4)}")
        dt = W4A16_F16 if dtype == torch.float16 else W4A16_BF16
    else:
        dt = x_code = _act_code(x)
        if x_scales is not None or (dtype is not None and dtype != x_dtype):
            raise ValueError("x_scales and another dtype go with float8_e4m3fn codes")
        dtype = x_dtype
        if x_shape[1] != K:
            raise ValueError(f"x is {tuple(x_shape)}, expected {K} columns")
    if bias is not None and (bias.dtype != dtype or bias.shape != (*lead, N)):
        raise ValueError(f"bias must be {dtype} {(*lead, N)}")
    device = x.device
    _require_device(x, "x", device)
    _require_all(device, (w, "w"), (scales, "scales"), (bias, "bias"), (x_scales, "x_scales"))
    return device, dtype, dt, x_code, s_code, x_shape[0], N, K


def _fp8_workspace(device, stream, workspace, fn, *sizes):
    """(its pointer, its bytes): the caller's, or the one of the device and stream."""
    if workspace is not None:
        return _given_workspace(device, workspace)
    return _own_workspace(device, stream, _size_of(device, fn, *sizes))


def _fp8_out(x, out, dtype, shape):
    if out is None:
        return x.new_empty(shape, dtype=dtype)
    if out.dtype != dtype or out.shape != shape:
        raise ValueError(f"out must be {dtype} {shape}")
    _require_device(out, "out", x.device)
    return out


def w4a16_minifloat_linear_workspace_size(M, N, K, x_dtype, transpose=False) -> int:
    return int(lib.w4a16_minifloat_linear_workspace_size(M, N, K, x_dtype, int(bool(transpose))))


def w4a16_minifloat_linear(x, w, scales, bias=None, *, transpose: bool = False, x_scales=None, dtype=None, out=None,
                     workspace=None):
    """y = x . (w * scales)^T (+ bias): w float8_e4m3fn [N, K] with scales float32 or float8_e8m0fnu
    [ceil(N / 128), ceil(K / 128)]; x float16 or bfloat16 [M, K], quantised as by
    w4a16_minifloat_quantize, or its codes with x_scales (y then of dtype, bfloat16 by default).  With
    transpose w is [K, N], y = x . (w * scales): w4a16_minifloat_linear(dy, w, scales, transpose=True) is
    the gradient of a layer's input.  Of eight products of neighbouring k the matrix unit drops what
    lies more than 13 bits below the largest; sums beyond are in float32.  Not recorded by autograd.
    workspace: as for w4a16_lora_linear, of w4a16_minifloat_linear_workspace_size."""
    device, dtype, dt, x_code, s_code, M, N, K = _fp8_args(x, w, scales, bias, transpose, x_scales, dtype, None, ())
    out = _fp8_out(x, out, dtype, (M, N))
    stream, transpose = _raw_stream(device), int(bool(transpose))
    ws_ptr, ws_bytes = _fp8_workspace(device, stream, workspace, lib.w4a16_minifloat_linear_workspace_size, M, N, K, x_code, transpose)
    _invoke(device, lib.w4a16_minifloat_linear, x.data_ptr(), _ptr(x_scales), w.data_ptr(), scales.data_ptr(), _ptr(bias),
            out.data_ptr(), M, N, K, x_code, s_code, dt, transpose, ws_ptr, ws_bytes, stream)
    return out


def w4a16_minifloat_moe_workspace_size(M, topk, E, N, K, x_dtype, transpose=False, x_per_slot=False) -> int:
    return int(lib.w4a16_minifloat_moe_workspace_size(M, topk, E, N, K, x_dtype, int(bool(transpose)), int(bool(x_per_slot))))


def w4a16_minifloat_moe_linear(x, w, scales, topk_ids, topk_weights=None, bias=None, *, transpose: bool = False,
                         x_per_slot: bool = False, x_scales=None, dtype=None, out=None, workspace=None):
    """w4a16_minifloat_linear with each slot's expert: y[m * topk + j] = topk_weights[m, j] * (x_row .
    (w_e * scales_e)^T + bias_e), e = topk_ids[m, j] (outside [0, E): a zero row), from stacks
    w [E, N, K], scales [E, ceil(N / 128), ceil(K / 128)] and bias [E, N]; x is [M, K], or
    [M * topk, K] with x_per_slot.  topk_ids int32 and topk_weights float32 [M, topk] as w4a16_route
    gives them.  With transpose w is [E, K, N].  Returns [M * topk, N]."""
    torch = _torch()
    if topk_ids.dim() != 2 or topk_ids.dtype != torch.int32:
        raise TypeError("topk_ids must be int32 [M, topk]")
    M, topk = topk_ids.shape
    E = w.shape[0]
    device, dtype, dt, x_code, s_code, _, N, K = _fp8_args(x, w, scales, bias, transpose, x_scales, dtype,
                                                           M * topk if x_per_slot else M, (E,))
    if topk_weights is not None and (topk_weights.dtype != torch.float32 or topk_weights.shape != (M, topk)):
        raise ValueError(f"topk_weights must be float32 {(M, topk)}")
    _require_all(device, (topk_ids, "topk_ids"), (topk_weights, "topk_weights"))
    out = _fp8_out(x, out, dtype, (M * topk, N))
    stream, transpose, x_per_slot = _raw_stream(device), int(bool(transpose)), int(bool(x_per_slot))
    ws_ptr, ws_bytes = _fp8_workspace(device, stream, workspace, lib.w4a16_minifloat_moe_workspace_size, M, topk, E, N, K, x_code,
                                      transpose, x_per_slot)
    _invoke(device, lib.w4a16_minifloat_moe_linear, x.data_ptr(), _ptr(x_scales), w.data_ptr(), scales.data_ptr(), _ptr(bias),
            topk_ids.data_ptr(), _ptr(topk_weights), out.data_ptr(), M, topk, E, N, K, x_code, s_code, dt, transpose, x_per_slot,
            ws_ptr, ws_bytes, stream)
    return out
