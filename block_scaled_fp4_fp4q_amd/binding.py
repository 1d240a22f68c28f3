"""Thin ctypes binding of libfp4q.so (include/fp4q.h).

Argument marshalling only: tensors are torch tensors on a ROCm device, whose
data pointers and current HIP stream are handed to the C ABI unchanged.  All
arithmetic happens in the library's HIP kernels.  There is no fallback: if the
library is missing, or a call is rejected, this module raises.
"""
import ctypes as C
import operator
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4q.so")

FP4Q_NVFP4, FP4Q_MXFP4, FP4Q_IF4, FP4Q_IF3, FP4Q_IF6 = 0, 1, 2, 3, 4
FP4Q_F32, FP4Q_BF16 = 0, 1
FP4Q_SCALE_ABSMAX, FP4Q_SCALE_SWEEP, FP4Q_SCALE_FOUR_OVER_SIX = 0, 1, 2
FP4Q_OBJ_MSE, FP4Q_OBJ_WMSE = 0, 1

STATUS = {0: "FP4Q_OK", -1: "FP4Q_E_NULL", -2: "FP4Q_E_ARG", -3: "FP4Q_E_SHAPE",
          -4: "FP4Q_E_UNSUPPORTED", -5: "FP4Q_E_HIP", -6: "FP4Q_E_ALIGN", -7: "FP4Q_E_SCRATCH"}

# every symbol include/fp4q.h declares
EXPORTS = ("fp4q_workspace_bytes", "fp4q_quantize", "fp4q_quantize_noalloc",
           "fp4q_quantize_relaxed", "fp4q_dequantize", "fp4q_error", "fp4q_status_string",
           "fp4q_abi_version", "fp4q_kv_write", "fp4q_kv_read", "fp4q_attend",
           "fp4q_attend_workspace_bytes")


class fp4q_spec(C.Structure):
    _fields_ = [("format", C.c_int32), ("block", C.c_int32), ("scale_rule", C.c_int32),
                ("objective", C.c_int32), ("sweep_lo", C.c_int32), ("sweep_hi", C.c_int32),
                ("rotate", C.c_int32), ("global_scale_given", C.c_int32)]


class fp4q_kv_cache(C.Structure):
    _fields_ = [("k_codes", C.c_void_p), ("k_scales", C.c_void_p), ("k_global", C.c_void_p),
                ("v_codes", C.c_void_p), ("v_scales", C.c_void_p), ("v_global", C.c_void_p),
                ("num_pages", C.c_int64), ("kv_heads", C.c_int32), ("page_size", C.c_int32),
                ("head_dim", C.c_int32), ("reserved", C.c_int32),
                ("code_page", C.c_int64), ("code_head", C.c_int64), ("code_token", C.c_int64),
                ("scale_page", C.c_int64), ("scale_head", C.c_int64), ("scale_token", C.c_int64)]


class fp4q_attention(C.Structure):
    _fields_ = [("q", C.c_void_p), ("q_row_stride", C.c_int64), ("q_head_stride", C.c_int64),
                ("out", C.c_void_p), ("out_row_stride", C.c_int64), ("out_head_stride", C.c_int64),
                ("lse", C.c_void_p), ("q_starts", C.c_void_p), ("kv_lens", C.c_void_p),
                ("block_table", C.c_void_p), ("table_stride", C.c_int64), ("total_q", C.c_int64),
                ("table_len", C.c_int32), ("batch", C.c_int32), ("max_q", C.c_int32),
                ("max_kv", C.c_int32), ("q_heads", C.c_int32), ("dtype", C.c_int32),
                ("causal", C.c_int32), ("window", C.c_int32), ("scale", C.c_float),
                ("reserved", C.c_int32)]


class Fp4qError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        msg = _lib_handle().fp4q_status_string(status).decode() if _LIB is not None else ""
        super().__init__(f"{fn} returned {STATUS.get(status, status)}: {msg}")


_LIB = None


def _lib_handle():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                              "or python block_scaled_fp4_fp4q_amd/build.py")
        L = C.CDLL(LIB_PATH)
        vp, i32, i64, sz = C.c_void_p, C.c_int32, C.c_int64, C.c_size_t
        sp = C.POINTER(fp4q_spec)
        L.fp4q_workspace_bytes.restype = sz
        L.fp4q_workspace_bytes.argtypes = [sp, i64, i64]
        L.fp4q_quantize.restype = C.c_int
        L.fp4q_quantize.argtypes = [sp, vp, i32, i64, i64, vp, vp, vp, vp, vp, sz, vp]
        L.fp4q_quantize_noalloc.restype = C.c_int
        L.fp4q_quantize_noalloc.argtypes = [sp, vp, i32, i64, i64, vp, vp, vp, vp, vp]
        L.fp4q_quantize_relaxed.restype = C.c_int
        L.fp4q_quantize_relaxed.argtypes = [sp, vp, i32, i64, i64, vp, i32, i32, vp, vp, vp, vp,
                                            sz, vp]
        L.fp4q_dequantize.restype = C.c_int
        L.fp4q_dequantize.argtypes = [sp, vp, vp, vp, i64, i64, i32, vp, i32, vp]
        L.fp4q_error.restype = C.c_int
        L.fp4q_error.argtypes = [sp, vp, i32, i64, i64, vp, vp, vp, vp, vp, sz,
                                 C.POINTER(C.c_double), vp]
        kp, ap = C.POINTER(fp4q_kv_cache), C.POINTER(fp4q_attention)
        L.fp4q_kv_write.restype = C.c_int
        L.fp4q_kv_write.argtypes = [sp, kp, vp, vp, i32, i64, i64, i64, i64, i64, vp, vp]
        L.fp4q_kv_read.restype = C.c_int
        L.fp4q_kv_read.argtypes = [sp, kp, vp, i64, vp, vp, i32, vp]
        L.fp4q_attend_workspace_bytes.restype = sz
        L.fp4q_attend_workspace_bytes.argtypes = [sp, kp, ap]
        L.fp4q_attend.restype = C.c_int
        L.fp4q_attend.argtypes = [sp, kp, ap, vp, sz, vp]
        L.fp4q_status_string.restype = C.c_char_p
        L.fp4q_status_string.argtypes = [C.c_int]
        L.fp4q_abi_version.restype = C.c_int
        L.fp4q_abi_version.argtypes = []
        _LIB = L
    return _LIB


def lib():
    return _lib_handle()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return FP4Q_F32
    if t.dtype == torch.bfloat16:
        return FP4Q_BF16
    raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _check(fn, st):
    if st != 0:
        raise Fp4qError(fn, st)


def make_spec(format=FP4Q_NVFP4, scale_rule=FP4Q_SCALE_ABSMAX, objective=FP4Q_OBJ_MSE,
              window=None, rotate=0, global_scale_given=False):
    block = 32 if format == FP4Q_MXFP4 else 16
    if window is None:
        # E8M0: the OCP exponent and the next one up; E4M3: the pages' windows
        window = (0, 1) if format == FP4Q_MXFP4 else \
            ((-8, 7) if objective == FP4Q_OBJ_WMSE else (-3, 7))
    lo, hi = window
    return fp4q_spec(format, block, scale_rule, objective, lo, hi, rotate, int(global_scale_given))


def _as_2d(x):
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch tensor")
    if x.dim() < 2:
        raise ValueError("x must have at least 2 dimensions (rows, cols)")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    return x.reshape(-1, x.shape[-1])


# The C ABI receives bare device pointers and cannot see a buffer's size,
# device or type: a host tensor or a short buffer would be read or written
# out of bounds by a kernel.  Every tensor argument is therefore checked here,
# before the library is called.  `require_cuda` is only turned off by the
# host-side tests of these checks.

def _check_device(name, t, device, require_cuda):
    if require_cuda and t.device.type != "cuda":
        raise ValueError(f"{name} must be a tensor on a ROCm device, not {t.device}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, but x is on {device}")


def _check_tensor(name, t, dtypes, min_numel, device, require_cuda=True, optional=False):
    """A device tensor argument: on x's device, one of `dtypes`, contiguous,
    at least `min_numel` elements.  None passes only when `optional`."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    _check_device(name, t, device, require_cuda)
    if t.dtype not in dtypes:
        want = " or ".join(str(d) for d in dtypes)
        raise ValueError(f"{name} has dtype {t.dtype}; expected {want}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < min_numel:
        raise ValueError(f"{name} has {t.numel()} elements; at least {min_numel} are needed")


_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_X = (torch.float32, torch.bfloat16)


ADAPTIVE = (FP4Q_IF4, FP4Q_IF3, FP4Q_IF6)


def code_bytes(format, n):
    """Bytes of the code stream of n elements: n-bit codes for IF3 (3) and
    IF6 (6), 4-bit codes otherwise."""
    return n * {FP4Q_IF3: 3, FP4Q_IF6: 6}.get(format, 4) // 8


def _needs_importance(spec):
    return spec.objective == FP4Q_OBJ_WMSE and (spec.scale_rule != FP4Q_SCALE_ABSMAX
                                                or spec.format in ADAPTIVE)


def _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda):
    n = rows * cols
    _check_tensor("codes", codes, _U8, code_bytes(spec.format, n), dev, require_cuda)
    _check_tensor("scales", scales, _U8, n // spec.block, dev, require_cuda)
    _check_tensor("global_scale", global_scale, _F32, 1, dev, require_cuda,
                  optional=spec.format == FP4Q_MXFP4)


def _check_workspace(spec, rows, cols, workspace, dev, require_cuda):
    need = fp4q_workspace_bytes(spec, rows, cols)
    _check_tensor("workspace", workspace, _U8, need, dev, require_cuda)


def check_quantize_args(spec, x, importance, codes, scales, global_scale, workspace,
                        require_cuda=True):
    """Host-side checks of fp4q_quantize's tensor arguments; raises
    ValueError/TypeError.  Returns x as a [rows, cols] view."""
    x2 = _as_2d(x)
    _check_device("x", x2, None, require_cuda)
    _dtype_code(x2)
    rows, cols = x2.shape
    dev = x2.device
    _check_tensor("importance", importance, _F32, cols, dev, require_cuda,
                  optional=not _needs_importance(spec))
    _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda)
    _check_workspace(spec, rows, cols, workspace, dev, require_cuda)
    return x2


def check_quantize_noalloc_args(spec, x, importance, codes, scales, global_scale,
                                require_cuda=True):
    """fp4q_quantize's checks without the workspace (the library's own
    static scratch serves instead)."""
    x2 = _as_2d(x)
    _check_device("x", x2, None, require_cuda)
    _dtype_code(x2)
    rows, cols = x2.shape
    dev = x2.device
    _check_tensor("importance", importance, _F32, cols, dev, require_cuda,
                  optional=not _needs_importance(spec))
    _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda)
    return x2


def check_relaxed_args(spec, x, coef, coef_group, codes, scales, global_scale, workspace,
                       require_cuda=True):
    x2 = _as_2d(x)
    _check_device("x", x2, None, require_cuda)
    _dtype_code(x2)
    rows, cols = x2.shape
    dev = x2.device
    if coef_group <= 0:
        raise ValueError("coef_group must be positive")
    _check_tensor("coef", coef, _F32, rows * (cols // coef_group), dev, require_cuda)
    _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda)
    _check_workspace(spec, rows, cols, workspace, dev, require_cuda)
    return x2


def check_dequantize_args(spec, codes, scales, global_scale, rows, cols, y, require_cuda=True):
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a torch tensor")
    _check_device("y", y, None, require_cuda)
    dev = y.device
    _check_tensor("y", y, _X, rows * cols, dev, require_cuda)
    _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda)


def check_error_args(spec, x, importance, codes, scales, global_scale, workspace,
                     require_cuda=True):
    x2 = _as_2d(x)
    _check_device("x", x2, None, require_cuda)
    _dtype_code(x2)
    rows, cols = x2.shape
    dev = x2.device
    _check_tensor("importance", importance, _F32, cols, dev, require_cuda, optional=True)
    _check_outputs(spec, rows, cols, codes, scales, global_scale, dev, require_cuda)
    _check_workspace(spec, rows, cols, workspace, dev, require_cuda)
    return x2


# ---------------------------------------------------------------------------
# the C ABI, one Python function per entry point
# ---------------------------------------------------------------------------

def fp4q_workspace_bytes(spec, rows, cols):
    return int(_lib_handle().fp4q_workspace_bytes(C.byref(spec), rows, cols))


def fp4q_quantize(spec, x, importance, codes, scales, global_scale, workspace, stream=None):
    x2 = check_quantize_args(spec, x, importance, codes, scales, global_scale, workspace)
    rows, cols = x2.shape
    st = _lib_handle().fp4q_quantize(C.byref(spec), _ptr(x2), _dtype_code(x2), rows, cols,
                                     _ptr(importance), _ptr(codes), _ptr(scales),
                                     _ptr(global_scale), _ptr(workspace), workspace.numel(),
                                     _stream(stream))
    _check("fp4q_quantize", st)


def fp4q_quantize_noalloc(spec, x, importance, codes, scales, global_scale, stream=None):
    """fp4q_quantize without a workspace: the library's static per-GPU
    scratch serves instead.  Calls that overlap on one GPU race on it."""
    x2 = check_quantize_noalloc_args(spec, x, importance, codes, scales, global_scale)
    rows, cols = x2.shape
    st = _lib_handle().fp4q_quantize_noalloc(C.byref(spec), _ptr(x2), _dtype_code(x2), rows, cols,
                                             _ptr(importance), _ptr(codes), _ptr(scales),
                                             _ptr(global_scale), _stream(stream))
    _check("fp4q_quantize_noalloc", st)


def fp4q_quantize_relaxed(spec, x, coef, coef_group, scales_given, codes, scales, global_scale,
                          workspace, stream=None):
    x2 = check_relaxed_args(spec, x, coef, coef_group, codes, scales, global_scale, workspace)
    rows, cols = x2.shape
    st = _lib_handle().fp4q_quantize_relaxed(C.byref(spec), _ptr(x2), _dtype_code(x2), rows, cols,
                                             _ptr(coef), coef_group, int(scales_given), _ptr(codes),
                                             _ptr(scales), _ptr(global_scale), _ptr(workspace),
                                             workspace.numel(), _stream(stream))
    _check("fp4q_quantize_relaxed", st)


def fp4q_dequantize(spec, codes, scales, global_scale, rows, cols, unrotate, y, stream=None):
    check_dequantize_args(spec, codes, scales, global_scale, rows, cols, y)
    st = _lib_handle().fp4q_dequantize(C.byref(spec), _ptr(codes), _ptr(scales),
                                       _ptr(global_scale), rows, cols, unrotate, _ptr(y),
                                       _dtype_code(y), _stream(stream))
    _check("fp4q_dequantize", st)


def fp4q_error(spec, x, importance, codes, scales, global_scale, workspace, stream=None):
    x2 = check_error_args(spec, x, importance, codes, scales, global_scale, workspace)
    rows, cols = x2.shape
    out = (C.c_double * 2)()
    st = _lib_handle().fp4q_error(C.byref(spec), _ptr(x2), _dtype_code(x2), rows, cols,
                                  _ptr(importance), _ptr(codes), _ptr(scales),
                                  _ptr(global_scale), _ptr(workspace), workspace.numel(),
                                  out, _stream(stream))
    _check("fp4q_error", st)
    return out[0], out[1]


# ---------------------------------------------------------------------------
# convenience: allocate outputs with torch, then call the entry points
# ---------------------------------------------------------------------------

def alloc_workspace(spec, rows, cols, device):
    n = fp4q_workspace_bytes(spec, rows, cols)
    if n == 0:
        raise ValueError("invalid spec or shape")
    return torch.empty(n, dtype=torch.uint8, device=device)


def quantize(x, format=FP4Q_NVFP4, scale_rule=FP4Q_SCALE_ABSMAX, objective=FP4Q_OBJ_MSE,
             window=None, rotate=0, importance=None, global_scale=None, workspace=None,
             stream=None):
    """Returns (codes uint8 [code_bytes(format, rows*cols)], scales uint8
    [rows*cols/block], global_scale float32 [1])."""
    spec = make_spec(format, scale_rule, objective, window, rotate, global_scale is not None)
    x2 = _as_2d(x)
    rows, cols = x2.shape
    dev = x.device
    codes = torch.empty(code_bytes(format, rows * cols), dtype=torch.uint8, device=dev)
    scales = torch.empty(rows * cols // spec.block, dtype=torch.uint8, device=dev)
    if global_scale is None:
        gs = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        gs = torch.as_tensor(global_scale, dtype=torch.float32, device=dev).reshape(1).clone()
    ws = workspace if workspace is not None else alloc_workspace(spec, rows, cols, dev)
    fp4q_quantize(spec, x2, importance, codes, scales, gs, ws, stream)
    return codes, scales, gs


def quantize_relaxed(x, coef, coef_group, format=FP4Q_NVFP4, scales=None, global_scale=None,
                     workspace=None, stream=None):
    """FOCUS deploy encode.  coef: float32 [rows, cols/coef_group] on the
    device; scales: given S_dq bytes, or None to compute the AbsMax ones.
    Returns (codes, scales, global_scale)."""
    spec = make_spec(format, global_scale_given=global_scale is not None)
    x2 = _as_2d(x)
    rows, cols = x2.shape
    dev = x.device
    codes = torch.empty(rows * cols // 2, dtype=torch.uint8, device=dev)
    given = scales is not None
    sc = scales if given else torch.empty(rows * cols // spec.block, dtype=torch.uint8, device=dev)
    if global_scale is None:
        gs = torch.empty(1, dtype=torch.float32, device=dev)
    else:
        gs = torch.as_tensor(global_scale, dtype=torch.float32, device=dev).reshape(1).clone()
    ws = workspace if workspace is not None else alloc_workspace(spec, rows, cols, dev)
    fp4q_quantize_relaxed(spec, x2, coef, coef_group, given, codes, sc, gs, ws, stream)
    return codes, sc, gs


def dequantize(codes, scales, global_scale, rows, cols, format=FP4Q_NVFP4, unrotate=0,
               dtype=torch.float32, stream=None):
    spec = make_spec(format)
    y = torch.empty(rows, cols, dtype=dtype, device=codes.device)
    fp4q_dequantize(spec, codes, scales, global_scale, rows, cols, unrotate, y, stream)
    return y


def error(x, codes, scales, global_scale, format=FP4Q_NVFP4, rotate=0, importance=None,
          workspace=None, stream=None):
    spec = make_spec(format, rotate=rotate)
    x2 = _as_2d(x)
    rows, cols = x2.shape
    ws = workspace if workspace is not None else alloc_workspace(spec, rows, cols, x.device)
    return fp4q_error(spec, x2, importance, codes, scales, global_scale, ws, stream)


# ---------------------------------------------------------------------------
# the 4-bit KV cache
# ---------------------------------------------------------------------------

def _cache_tensor(name, t, shape, device, require_cuda):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    _check_device(name, t, device, require_cuda)
    if t.dtype != torch.uint8:
        raise ValueError(f"{name} has dtype {t.dtype}; expected torch.uint8")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected {shape}")
    if t.stride(3) != 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")


class KvCache:
    """A 4-bit KV cache: K and V as codes uint8 [pages, kv_heads, page_size,
    head_dim / 2] and scales uint8 [pages, kv_heads, page_size, head_dim /
    block] (any strides, the last dimension contiguous, K's and V's alike) and
    one global scale float32 [1] each (None for MXFP4).  The tensors are the
    caller's; this handle checks them once, keeps references to them and passes
    their addresses on.  A contiguous cache [B, H, T, D] is one of B pages of T
    tokens.  Expanded dimensions can be read, not written.  `scale_rule`,
    `window` and `rotate` say how rows are written (and `rotate` how they are
    read).

    The calls run on torch's current stream of the cache's device, or on
    `stream`, one of that device; tensors that they are given must be ready
    there, and stay as they are until it has passed the call."""

    def __init__(self, k_codes, k_scales, k_global, v_codes, v_scales, v_global,
                 format=FP4Q_NVFP4, scale_rule=FP4Q_SCALE_ABSMAX, window=None, rotate=0,
                 require_cuda=True):
        if format not in (FP4Q_NVFP4, FP4Q_MXFP4):
            raise ValueError("a KV cache is NVFP4 or MXFP4")
        self.spec = make_spec(format, scale_rule, FP4Q_OBJ_MSE, window, rotate,
                              global_scale_given=format != FP4Q_MXFP4)
        if not isinstance(k_codes, torch.Tensor):
            raise TypeError("k_codes must be a torch tensor")
        if k_codes.dim() != 4:
            raise ValueError("k_codes must be [pages, kv_heads, page_size, head_dim / 2]")
        pages, heads, page, half = k_codes.shape
        self.pages, self.heads, self.page_size, self.head_dim = pages, heads, page, 2 * half
        if self.head_dim not in (64, 128, 256):
            raise ValueError(f"head_dim {self.head_dim} is not supported; use 64, 128 or 256")
        if heads < 1 or page < 1:
            raise ValueError("a KV cache needs at least one head and one token per page")
        self.device = k_codes.device
        _check_device("k_codes", k_codes, None, require_cuda)
        small = (pages, heads, page, self.head_dim // self.spec.block)
        for name, t, shape in (("k_codes", k_codes, (pages, heads, page, half)),
                               ("v_codes", v_codes, (pages, heads, page, half)),
                               ("k_scales", k_scales, small), ("v_scales", v_scales, small)):
            _cache_tensor(name, t, shape, self.device, require_cuda)
        for name, t in (("k_global", k_global), ("v_global", v_global)):
            _check_tensor(name, t, _F32, 1, self.device, require_cuda,
                          optional=format == FP4Q_MXFP4)
        if k_codes.stride() != v_codes.stride() or k_scales.stride() != v_scales.stride():
            raise ValueError("K and V of a cache must have the same strides")
        self.tensors = (k_codes, k_scales, k_global, v_codes, v_scales, v_global)
        ptr = [None if t is None else t.data_ptr() for t in self.tensors]
        self.struct = fp4q_kv_cache(*ptr, pages, heads, page, self.head_dim, 0,
                                    *k_codes.stride()[:3], *k_scales.stride()[:3])
        self._spec, self._struct = C.byref(self.spec), C.byref(self.struct)
        self._calls = {}  # attend's checked argument shapes


def alloc_kv_cache(pages, kv_heads, page_size, head_dim, k_global=None, v_global=None,
                   format=FP4Q_NVFP4, scale_rule=FP4Q_SCALE_ABSMAX, window=None, rotate=0,
                   device="cuda"):
    """A zeroed cache.  The global scales (numbers or tensors, NVFP4 only) are
    those of the tensors that will be written, max|x| / 1536 for instance."""
    block = 32 if format == FP4Q_MXFP4 else 16
    t = []
    for g in (k_global, v_global):
        if format == FP4Q_MXFP4:
            g = None
        elif g is None:
            raise ValueError("an NVFP4 cache needs both global scales")
        else:
            g = torch.as_tensor(g, dtype=torch.float32, device=device).reshape(1).clone()
        t += [torch.zeros(pages, kv_heads, page_size, head_dim // 2, dtype=torch.uint8, device=device),
              torch.zeros(pages, kv_heads, page_size, head_dim // block, dtype=torch.uint8, device=device),
              g]
    return KvCache(*t, format=format, scale_rule=scale_rule, window=window, rotate=rotate)


def _rows(name, t, rows, heads, dim, device, dtypes=_X):
    """A [rows, heads, dim] tensor whose last dimension is contiguous; returns
    its strides."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, but the cache is on {device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}; expected " + " or ".join(map(str, dtypes)))
    if tuple(t.shape) != (rows, heads, dim):
        raise ValueError(f"{name} has shape {tuple(t.shape)}; expected [{rows}, {heads}, {dim}]")
    st = t.stride()
    if st[2] != 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return st


def _ints(name, t, dtype, device, dim=1):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, but the cache is on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}; expected {dtype}")
    if t.dim() != dim or (t.numel() > 0 and t.stride()[-1] != 1):
        raise ValueError(f"{name} must have {dim} dimension(s), the last one contiguous")


def _here(device, stream):
    """Whether a call on `device` runs as it is: no stream given, and the
    device current."""
    return stream is None and (device.type != "cuda" or device.index == _current_device())


class _on:
    """The device as the current one, and a given stream as torch's current
    one there, so that what a call allocates belongs to its stream."""

    def __init__(self, device, stream):
        self.inner = [torch.cuda.device(device)]
        if stream is not None:
            # entered, it would make its own device the current one
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, but the cache is on {device}")
            self.inner.append(torch.cuda.stream(stream))

    def __enter__(self):
        for c in self.inner:
            c.__enter__()

    def __exit__(self, *exc):
        for c in reversed(self.inner):
            c.__exit__(*exc)


# the current device's index and a device's current stream as an integer,
# without the objects that the public functions make (these calls take a few
# microseconds in all)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def kv_write(cache, k, v, slots, stream=None):
    """Quantize k and v, float32 or bfloat16 [tokens, kv_heads, head_dim] (last
    dimension contiguous), into the cache at `slots` (int64 [tokens]; a
    negative or too large slot skips its token)."""
    dev = cache.device
    if not _here(dev, stream):
        with _on(dev, stream):
            return kv_write(cache, k, v, slots)
    _ints("slots", slots, torch.int64, dev)
    n = slots.shape[0]
    ks = _rows("k", k, n, cache.heads, cache.head_dim, dev)
    vs = _rows("v", v, n, cache.heads, cache.head_dim, dev)
    if k.dtype != v.dtype:
        raise ValueError("k and v must have the same dtype")
    _check("fp4q_kv_write", _lib_handle().fp4q_kv_write(
        cache._spec, cache._struct, k.data_ptr(), v.data_ptr(), _dtype_code(k), n, ks[0], ks[1],
        vs[0], vs[1], slots.data_ptr(), _current_stream(dev.index)))


def kv_read(cache, slots, dtype=torch.float32, stream=None):
    """The values of the rows at `slots` (int64 [tokens]): (k, v), each
    [tokens, kv_heads, head_dim] of `dtype`, un-rotated."""
    dev = cache.device
    if not _here(dev, stream):
        with _on(dev, stream):
            return kv_read(cache, slots, dtype)
    _ints("slots", slots, torch.int64, dev)
    if dtype not in _X:
        raise TypeError(f"unsupported dtype {dtype}; use float32 or bfloat16")
    n = slots.shape[0]
    k = torch.empty((n, cache.heads, cache.head_dim), dtype=dtype, device=dev)
    v = torch.empty_like(k)
    _check("fp4q_kv_read", _lib_handle().fp4q_kv_read(
        cache._spec, cache._struct, slots.data_ptr(), n, k.data_ptr(), v.data_ptr(),
        _dtype_code(k), _current_stream(dev.index)))
    return k, v


def _numbers(max_kv, max_q, causal, window, scale):
    """The numbers of an attention call as Python's own: what counts is an
    argument's value now (a 0-dimensional tensor may change in place)."""
    if type(max_kv) is not int and max_kv is not None:
        max_kv = operator.index(max_kv)
    if type(max_q) is not int and max_q is not None:
        max_q = operator.index(max_q)
    if type(causal) is not bool:
        causal = int(causal)
    if type(window) is not int:
        window = operator.index(window)
    if type(scale) is not float and scale is not None:
        scale = C.c_float(scale).value
    return max_kv, max_q, causal, window, scale


def _attention(cache, q, kv_lens, max_kv, block_table, q_starts, max_q, causal, window, scale, out):
    """The call's fp4q_attention without its pointers, from checked tensors and
    _numbers."""
    dev = cache.device
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a torch tensor [total_q, q_heads, head_dim]")
    total, heads = q.shape[0], q.shape[1]
    if heads < 1 or heads % cache.heads:
        raise ValueError(f"q has {heads} heads; expected a multiple of the cache's {cache.heads}")
    qs = _rows("q", q, total, heads, cache.head_dim, dev)
    _ints("kv_lens", kv_lens, torch.int32, dev)
    batch = kv_lens.shape[0]
    if q_starts is not None:
        _ints("q_starts", q_starts, torch.int32, dev)
        if q_starts.shape[0] != batch + 1:
            raise ValueError(f"q_starts has {q_starts.shape[0]} entries; expected batch + 1 = {batch + 1}")
        if max_q is None:
            max_q = total
    else:
        each = total // batch if batch else 0
        if each * batch != total or (max_q is not None and max_q != each):
            raise ValueError("without q_starts, q must hold max_q rows for each sequence")
        max_q = each
    stride, entries = 0, 0
    if block_table is not None:
        _ints("block_table", block_table, torch.int32, dev, 2)
        if block_table.shape[0] != batch:
            raise ValueError(f"block_table has {block_table.shape[0]} rows; expected {batch}")
        if cache.page_size % 16:
            raise ValueError("with a block_table the page size must be a multiple of 16")
        stride, entries = block_table.stride(0), block_table.shape[1]
    if max_kv is None:
        max_kv = cache.page_size * (entries if block_table is not None else 1)
    # ctypes would drop the upper bits of these
    for name, n in (("batch", batch), ("max_q", max_q), ("max_kv", max_kv), ("window", window),
                    ("block_table's entries", entries)):
        if not 0 <= n < 1 << 31:
            raise ValueError(f"{name} is {n}; expected 31 bits")
    os = _rows("out", out, total, heads, cache.head_dim, dev, (q.dtype,))
    if scale is None:
        scale = cache.head_dim ** -0.5
    return fp4q_attention(None, qs[0], qs[1], None, os[0], os[1], None, None, None, None, stride,
                          total, entries, batch, max_q, max_kv, heads, _dtype_code(q), causal,
                          window, scale, 0)


def _point(call, q, out, lse, kv_lens, block_table, q_starts):
    call.q, call.out, call.kv_lens = q.data_ptr(), out.data_ptr(), kv_lens.data_ptr()
    if lse is not None:
        call.lse = lse.data_ptr()
    if block_table is not None:
        call.block_table = block_table.data_ptr()
    if q_starts is not None:
        call.q_starts = q_starts.data_ptr()


def _same(t):
    """What the checks of a tensor depend on."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _workspace_bytes(cache, call):
    return int(_lib_handle().fp4q_attend_workspace_bytes(cache._spec, cache._struct, C.byref(call)))


def attend_workspace_bytes(cache, q, kv_lens, max_kv=None, block_table=None, q_starts=None,
                           max_q=None, causal=True, window=0):
    """Bytes that `attend` of these arguments needs as its workspace (only
    their shapes and types matter)."""
    max_kv, max_q, causal, window, _ = _numbers(max_kv, max_q, causal, window, None)
    call = _attention(cache, q, kv_lens, max_kv, block_table, q_starts, max_q, causal, window, None, q)
    call.out_row_stride, call.out_head_stride = q.shape[1] * q.shape[2], q.shape[2]  # of any output
    _point(call, q, q, None, kv_lens, block_table, q_starts)
    return _workspace_bytes(cache, call)


def attend(cache, q, kv_lens, max_kv=None, block_table=None, q_starts=None, max_q=None,
           causal=True, window=0, scale=None, return_lse=False, out=None, workspace=None, stream=None):
    """Attention of the queries q, float32 or bfloat16 [total_q, q_heads,
    head_dim], over the cache; query head h reads KV head h // (q_heads //
    kv_heads).  Returns out like q, or (out, lse float32 [total_q, q_heads])
    with return_lse.

    kv_lens      int32 [batch]: keys of each sequence, its new ones among them.
    max_kv       a bound on kv_lens (default: what a sequence's pages hold).
                 Calls of the same shapes and numbers share their checks: a
                 bound that stays costs less than one that follows the lengths.
    block_table  int32 [batch, entries]: the pages of each sequence; None:
                 sequence b is page b (a contiguous cache).
    q_starts     int32 [batch + 1]: the queries of sequence b are the rows
                 q_starts[b] : q_starts[b+1]; None: the same number for each.
    max_q        a bound on the queries of a sequence.
    causal       the last query of a sequence sees all of its keys, each one
                 before it one less; False: every query sees all.
    window       with causal, only the last `window` of those (0: all).
    scale        of the logits (default head_dim ** -0.5).
    out          like q, of any strides without expanded dimensions.
    A query without keys gives zeros and lse -inf.  Rows of no sequence are not
    written: they stay what they are in `out`, unspecified where it is
    allocated here.  A given workspace (uint8, attend_workspace_bytes) must
    not be shared by calls that may run at the same time."""
    dev = cache.device
    if not _here(dev, stream):
        with _on(dev, stream):
            return attend(cache, q, kv_lens, max_kv, block_table, q_starts, max_q, causal, window,
                          scale, return_lse, out, workspace)
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch tensor [total_q, q_heads, head_dim]")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    lse = torch.empty(q.shape[:2], dtype=torch.float32, device=dev) if return_lse else None
    max_kv, max_q, causal, window, scale = _numbers(max_kv, max_q, causal, window, scale)
    # calls that differ in addresses alone share their checks
    key = (_same(q), _same(kv_lens), _same(block_table), _same(q_starts), _same(out), max_kv, max_q,
           causal, window, scale)
    known = cache._calls.get(key)
    if known is None:
        call = _attention(cache, q, kv_lens, max_kv, block_table, q_starts, max_q, causal, window, scale, out)
        _point(call, q, out, lse, kv_lens, block_table, q_starts)
        if len(cache._calls) >= 64:
            cache._calls.clear()
        need = _workspace_bytes(cache, call)
        cache._calls[key] = (bytes(call), need)
    else:
        call, need = fp4q_attention.from_buffer_copy(known[0]), known[1]
        call.lse = None
        _point(call, q, out, lse, kv_lens, block_table, q_starts)
    if not need:
        space = None
    elif workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        space = workspace.data_ptr()
    else:
        _check_tensor("workspace", workspace, _U8, need, dev, require_cuda=False)
        space = workspace.data_ptr()
    st = _lib_handle().fp4q_attend(cache._spec, cache._struct, C.byref(call), space, need,
                                   _current_stream(dev.index))
    if st:
        cache._calls.pop(key, None)
        _check("fp4q_attend", st)
    return (out, lse) if return_lse else out
