"""ctypes binding of libfa.so: the C ABI of include/fa.h under the same names,
plus ``forward``/``backward`` helpers that marshal torch CUDA tensors.

Every computation runs in the library's kernels. There is no fallback: if
libfa.so is missing, or a tensor is not a CUDA tensor, the call raises.
torch is used only to allocate device memory and to name the stream. The
helpers check every buffer against the shapes that q and k imply (the C ABI
receives only pointers and those sizes) and launch on q's device.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfa.so")
# The same library built with device-side index and bounds checks (FA_CHECK=1;
# see fa_last_device_status in include/fa.h). Selected with use_library().
LIB_CHECK_PATH = os.path.join(_HERE, "libfa_check.so")

FA_FP16, FA_BF16 = 0, 1
FA_OK = 0
FA_ERR_MISALIGNED = -3
FA_ERR_WORKSPACE = -7
STATUS = {
    0: "FA_OK", -1: "FA_ERR_INVALID_ARG", -2: "FA_ERR_UNSUPPORTED", -3: "FA_ERR_MISALIGNED",
    -4: "FA_ERR_CUDA", -5: "FA_ERR_TIMEOUT", -6: "FA_ERR_NOT_IMPLEMENTED", -7: "FA_ERR_WORKSPACE",
    -8: "FA_ERR_SCRATCH_LIMIT", -9: "FA_ERR_BOUNDS",
}
FA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
EXPORTED = ("fa_fwd", "fa_fwd_ex", "fa_fwd_fp8", "fa_fwd_fp8_ex", "fa_bwd", "fa_bwd_ex", "fa_bwd_noalloc",
            "fa_fwd_workspace_size", "fa_fwd_workspace_size_ex", "fa_fwd_split_plan",
            "fa_bwd_workspace_size", "fa_bwd_workspace_size_ex", "fa_selftest_wait_timeout",
            "fa_diff_fwd", "fa_diff_fwd_workspace_size", "fa_diff_bwd", "fa_diff_bwd_workspace_size", "fa_rotary",
            "fa_last_device_status", "fa_strerror", "fa_version")
FA_LAMBDA_FP32 = 2
FA_ROTARY_MAX_AXES = 8


class FaTensor(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64),
                ("stride_s", ctypes.c_int64), ("stride_h", ctypes.c_int64)]


class FwdParams(ctypes.Structure):
    _fields_ = [("q", FaTensor), ("k", FaTensor), ("v", FaTensor), ("o", FaTensor),
                ("lse", ctypes.c_void_p),
                ("B", ctypes.c_int), ("H", ctypes.c_int), ("Sq", ctypes.c_int), ("Sk", ctypes.c_int),
                ("D", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("dtype", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("split_ranks", ctypes.c_int)]


class FwdFp8Params(ctypes.Structure):
    _fields_ = [("q", FaTensor), ("k", FaTensor), ("v", FaTensor), ("o", FaTensor),
                ("lse", ctypes.c_void_p),
                ("B", ctypes.c_int), ("H", ctypes.c_int), ("Sq", ctypes.c_int), ("Sk", ctypes.c_int),
                ("D", ctypes.c_int), ("scale", ctypes.c_float),
                ("q_descale", ctypes.c_float), ("k_descale", ctypes.c_float), ("v_descale", ctypes.c_float),
                ("causal", ctypes.c_int), ("o_dtype", ctypes.c_int)]


class BwdParams(ctypes.Structure):
    _fields_ = [("q", FaTensor), ("k", FaTensor), ("v", FaTensor), ("o", FaTensor), ("dO", FaTensor),
                ("lse", ctypes.c_void_p),
                ("dq", FaTensor), ("dk", FaTensor), ("dv", FaTensor),
                ("B", ctypes.c_int), ("H", ctypes.c_int), ("Sq", ctypes.c_int), ("Sk", ctypes.c_int),
                ("D", ctypes.c_int), ("scale", ctypes.c_float), ("causal", ctypes.c_int),
                ("dtype", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("deterministic", ctypes.c_int)]


class DiffLambda(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("stride_h", ctypes.c_int64), ("extent_b", ctypes.c_int), ("extent_s", ctypes.c_int),
                ("extent_h", ctypes.c_int), ("dtype", ctypes.c_int)]


class DiffFwdParams(ctypes.Structure):
    _fields_ = [("q", FaTensor * 2), ("k", FaTensor * 2), ("v", FaTensor), ("lam", DiffLambda),
                ("k_lens", ctypes.c_void_p), ("o", FaTensor), ("o2", FaTensor), ("lse", ctypes.c_void_p),
                ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("Sq", ctypes.c_int),
                ("Sk", ctypes.c_int), ("D", ctypes.c_int), ("Dv", ctypes.c_int), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t)]


class DiffBwdParams(ctypes.Structure):
    _fields_ = [("q", FaTensor * 2), ("k", FaTensor * 2), ("v", FaTensor), ("o", FaTensor), ("o2", FaTensor),
                ("dO", FaTensor), ("lse", ctypes.c_void_p), ("lam", DiffLambda),
                ("dq", FaTensor * 2), ("dk", FaTensor * 2), ("dv", FaTensor), ("dlam", ctypes.c_void_p),
                ("B", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int), ("Sq", ctypes.c_int),
                ("Sk", ctypes.c_int), ("D", ctypes.c_int), ("Dv", ctypes.c_int), ("scale", ctypes.c_float),
                ("causal", ctypes.c_int), ("dtype", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
                ("deterministic", ctypes.c_int)]


class RotaryParams(ctypes.Structure):
    _fields_ = [("q", FaTensor), ("k", FaTensor), ("q_out", FaTensor), ("k_out", FaTensor),
                ("positions", ctypes.c_void_p), ("pos_stride_axis", ctypes.c_int64),
                ("pos_stride_b", ctypes.c_int64), ("pos_stride_s", ctypes.c_int64), ("pos_int64", ctypes.c_int),
                ("inv_freq", ctypes.c_void_p), ("inv_freq_fp64", ctypes.c_int), ("axes", ctypes.c_int),
                ("sections", ctypes.c_int * FA_ROTARY_MAX_AXES),
                ("B", ctypes.c_int), ("S", ctypes.c_int), ("H", ctypes.c_int), ("Hk", ctypes.c_int),
                ("D", ctypes.c_int), ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int),
                ("dtype", ctypes.c_int)]


class FaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({fa_strerror(status)})")


_lib = None


def use_library(path: str) -> None:
    """Route every call of this module through the library at `path` from now
    on (LIB_PATH, or LIB_CHECK_PATH for the check build). The library is
    loaded at the next call."""
    global _lib, LIB_PATH
    LIB_PATH = path
    _lib = None
    _packed_fns.clear()


def lib():
    """Load libfa.so (once). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m exact_io_aware_96_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        L.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
        L.fa_fwd.restype = i
        L.fa_fwd_ex.argtypes = [ctypes.POINTER(FwdParams), vp]
        L.fa_fwd_ex.restype = i
        L.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, f, f, f, i, i, vp]
        L.fa_fwd_fp8.restype = i
        L.fa_fwd_fp8_ex.argtypes = [ctypes.POINTER(FwdFp8Params), vp]
        L.fa_fwd_fp8_ex.restype = i
        L.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, vp]
        L.fa_bwd.restype = i
        L.fa_bwd_ex.argtypes = [ctypes.POINTER(BwdParams), vp]
        L.fa_bwd_ex.restype = i
        L.fa_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
        L.fa_bwd_noalloc.restype = i
        L.fa_fwd_workspace_size.argtypes = [i, i, i, i, i, i]
        L.fa_fwd_workspace_size.restype = sz
        L.fa_fwd_workspace_size_ex.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int)]
        L.fa_fwd_workspace_size_ex.restype = sz
        L.fa_fwd_split_plan.argtypes = [i, i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_int), ctypes.c_void_p, i]
        L.fa_fwd_split_plan.restype = i
        L.fa_bwd_workspace_size.argtypes = [i, i, i, i]
        L.fa_bwd_workspace_size.restype = sz
        L.fa_bwd_workspace_size_ex.argtypes = [i, i, i, i, i, i]
        L.fa_bwd_workspace_size_ex.restype = sz
        L.fa_diff_fwd.argtypes = [ctypes.POINTER(DiffFwdParams), vp]
        L.fa_diff_fwd.restype = i
        L.fa_diff_fwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i]
        L.fa_diff_fwd_workspace_size.restype = sz
        L.fa_diff_bwd.argtypes = [ctypes.POINTER(DiffBwdParams), vp]
        L.fa_diff_bwd.restype = i
        L.fa_diff_bwd_workspace_size.argtypes = [i, i, i, i, i, i, i, i, i]
        L.fa_diff_bwd_workspace_size.restype = sz
        L.fa_rotary.argtypes = [ctypes.POINTER(RotaryParams), vp]
        L.fa_rotary.restype = i
        L.fa_selftest_wait_timeout.argtypes = [ctypes.c_uint, vp]
        L.fa_selftest_wait_timeout.restype = i
        L.fa_last_device_status.argtypes = [ctypes.POINTER(ctypes.c_int)]
        L.fa_last_device_status.restype = i
        L.fa_strerror.argtypes = [i]
        L.fa_strerror.restype = ctypes.c_char_p
        L.fa_version.argtypes = []
        L.fa_version.restype = i
        _lib = L
    return _lib


_packed_fns = {}


def _packed(name: str):
    """The entry point `name` taking its params struct as packed bytes."""
    f = _packed_fns.get(name)
    if f is None:
        f = lib()[name]  # a function object of its own
        f.argtypes, f.restype = [ctypes.c_char_p, ctypes.c_void_p], ctypes.c_int
        _packed_fns[name] = f
    return f


# ---------------------------------------------------------------- raw C ABI
def fa_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale, causal, dtype, stream=0) -> int:
    return lib().fa_fwd(q, k, v, o, lse, B, H, Sq, Sk, D, scale, causal, dtype, stream)


def fa_fwd_ex(params: FwdParams, stream=0) -> int:
    return lib().fa_fwd_ex(ctypes.byref(params), stream)


def fa_fwd_fp8(q, k, v, o, lse, B, H, Sq, Sk, D, scale, q_descale, k_descale, v_descale, causal, o_dtype,
               stream=0) -> int:
    return lib().fa_fwd_fp8(q, k, v, o, lse, B, H, Sq, Sk, D, scale, q_descale, k_descale, v_descale, causal,
                            o_dtype, stream)


def fa_fwd_fp8_ex(params: FwdFp8Params, stream=0) -> int:
    return lib().fa_fwd_fp8_ex(ctypes.byref(params), stream)


def fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, dtype,
           workspace, workspace_bytes, stream=0) -> int:
    return lib().fa_bwd(q, k, v, o, lse, dO, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, dtype,
                        workspace, workspace_bytes, stream)


def fa_bwd_ex(params: BwdParams, stream=0) -> int:
    return lib().fa_bwd_ex(ctypes.byref(params), stream)


def fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, dtype, stream=0) -> int:
    """Backward with the library's built-in scratch instead of a workspace
    (for callers that cannot allocate device memory; see include/fa.h)."""
    return lib().fa_bwd_noalloc(q, k, v, o, lse, dO, dq, dk, dv, B, H, Sq, Sk, D, scale, causal, dtype, stream)


def fa_bwd_workspace_size(B, H, Sq, D) -> int:
    return lib().fa_bwd_workspace_size(B, H, Sq, D)


def fa_bwd_workspace_size_ex(B, H, Sq, Sk, D, deterministic) -> int:
    return lib().fa_bwd_workspace_size_ex(B, H, Sq, Sk, D, deterministic)


def fa_diff_fwd(params: DiffFwdParams, stream=0) -> int:
    return lib().fa_diff_fwd(ctypes.byref(params), stream)


def fa_diff_fwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal) -> int:
    return lib().fa_diff_fwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal)


def fa_diff_bwd(params: DiffBwdParams, stream=0) -> int:
    return lib().fa_diff_bwd(ctypes.byref(params), stream)


def fa_diff_bwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal, deterministic) -> int:
    return lib().fa_diff_bwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal, deterministic)


def fa_rotary(params: RotaryParams, stream=0) -> int:
    return lib().fa_rotary(ctypes.byref(params), stream)


def fa_selftest_wait_timeout(limit_us, stream=0) -> int:
    """Launch the failure-path self-test (see include/fa.h)."""
    return lib().fa_selftest_wait_timeout(limit_us, stream)


def fa_last_device_status():
    """(status, [code, block, role, iteration]) — synchronises the device."""
    d = (ctypes.c_int * 4)()
    st = lib().fa_last_device_status(d)
    return st, list(d)


def fa_strerror(status: int) -> str:
    return lib().fa_strerror(status).decode()


def fa_version() -> int:
    return lib().fa_version()


# ------------------------------------------------------------ torch helpers
_DT = {torch.float16: FA_FP16, torch.bfloat16: FA_BF16}


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"fp16/bf16 tensors only, got {t.dtype}")
    return _DT[t.dtype]


def _view(t: torch.Tensor) -> FaTensor:
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
    if t.dim() != 4 or t.stride(3) != 1:
        raise ValueError("expected a [B, S, H, D] view with a contiguous last axis")
    return FaTensor(t.data_ptr(), t.stride(0), t.stride(1), t.stride(2))


def _expect(name: str, t: torch.Tensor, shape, dtype, device) -> None:
    """The C ABI takes raw pointers and the sizes of q and k only, so every
    other buffer must have exactly the shape, dtype and device they imply
    (a smaller one would be read or written past its end)."""
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, q on {device}")


def _expect_lse(lse: torch.Tensor, B: int, H: int, Sq: int, device) -> None:
    _expect("lse", lse, (B, H, Sq), torch.float32, device)
    if not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [B, H, Sq] tensor")


def _dims(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, S, H, D] tensors")
    B, Sq, H, D = q.shape
    if (k.shape[0], k.shape[2], k.shape[3]) != (B, H, D):
        raise ValueError(f"k: expected [B={B}, Sk, H={H}, D={D}], got {tuple(k.shape)}")
    return B, Sq, H, D, k.shape[1]


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def fwd_workspace_size(B, H, Sq, Sk, D, causal, split_ranks=0, device=None):
    """(bytes, split ranks) of the forward's key-range split on `device`
    (default: the current one); (0, 0) when no split is chosen."""
    ns = ctypes.c_int(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        n = lib().fa_fwd_workspace_size_ex(B, H, Sq, Sk, D, int(bool(causal)), int(split_ranks), ctypes.byref(ns))
    return int(n), ns.value


def fwd_split_plan(B, H, Sq, Sk, D, causal, split_ranks=0, sms=0):
    """(n_split, [(rank, kind), ...]) of the forward's key-range split for
    `sms` SMs (0: the current device); kind 0 whole rank, 1/2 its key halves."""
    ns = ctypes.c_int(0)
    buf = (ctypes.c_ubyte * 256)()
    n = lib().fa_fwd_split_plan(B, H, Sq, Sk, D, int(bool(causal)), int(split_ranks), int(sms), ctypes.byref(ns),
                                buf, 256)
    if n < 0:
        raise FaError(n, "fa_fwd_split_plan")
    return ns.value, [(buf[i] // 3, buf[i] % 3) for i in range(n)]


def fwd_workspace_for(B, H, Sq, Sk, D, causal, device, split_ranks=0):
    """A workspace for forward(..., workspace=...), or None when no split is chosen."""
    n, _ = fwd_workspace_size(B, H, Sq, Sk, D, causal, split_ranks, device)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def forward(q, k, v, causal=False, scale=None, out=None, lse=None, stream=None, workspace=None, split_ranks=0):
    """O, LSE = attention(q, k, v) on [B, S, H, D] CUDA tensors (strided views allowed).

    split_ranks: 0 lets the library choose a key-range split of the heaviest
    query blocks (it then needs a workspace, taken from torch's allocator
    unless one is given), k > 0 splits the first k query-block ranks, -1
    never splits."""
    B, Sq, H, D, Sk = _dims(q, k)
    dt = _dtype_code(q)
    dev = q.device
    _expect("k", k, (B, Sk, H, D), q.dtype, dev)
    _expect("v", v, (B, Sk, H, D), q.dtype, dev)
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Sq, H, D), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev)
    _expect("out", out, (B, Sq, H, D), q.dtype, dev)
    _expect_lse(lse, B, H, Sq, dev)
    views = (_view(q), _view(k), _view(v), _view(out))  # refuses non-CUDA tensors first
    if workspace is None and split_ranks >= 0:
        workspace = fwd_workspace_for(B, H, Sq, Sk, D, causal, dev, split_ranks)
    if workspace is not None:
        if workspace.device != dev or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("workspace: expected a contiguous uint8 tensor on q's device")
    p = FwdParams(*views, lse.data_ptr(),
                  B, H, Sq, Sk, D, float(scale), int(bool(causal)), dt,
                  workspace.data_ptr() if workspace is not None else None,
                  workspace.numel() if workspace is not None else 0, int(split_ranks))
    with torch.cuda.device(dev):
        st = fa_fwd_ex(p, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_ex")
    return out, lse


def forward_fp8(q, k, v, q_descale, k_descale, v_descale, causal=False, scale=None,
                out_dtype=torch.bfloat16, out=None, lse=None, stream=None):
    """O, LSE from e4m3 tensors: the values attended over are q * q_descale,
    k * k_descale, v * v_descale. q, k, v are torch.float8_e4m3fn (or uint8
    holding E4M3 bytes) [B, S, H, D] CUDA views; O is ``out_dtype``."""
    B, Sq, H, D, Sk = _dims(q, k)
    if q.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise TypeError(f"e4m3 tensors (torch.float8_e4m3fn or uint8 bytes) only, got {q.dtype}")
    dev = q.device
    _expect("k", k, (B, Sk, H, D), q.dtype, dev)
    _expect("v", v, (B, Sk, H, D), q.dtype, dev)
    od = _DT.get(out_dtype)
    if od is None:
        raise TypeError(f"out_dtype must be fp16 or bf16, got {out_dtype}")
    if scale is None:
        scale = D ** -0.5
    if out is None:
        out = torch.empty((B, Sq, H, D), dtype=out_dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, H, Sq), dtype=torch.float32, device=dev)
    _expect("out", out, (B, Sq, H, D), out_dtype, dev)
    _expect_lse(lse, B, H, Sq, dev)
    p = FwdFp8Params(_view(q), _view(k), _view(v), _view(out), lse.data_ptr(),
                     B, H, Sq, Sk, D, float(scale), float(q_descale), float(k_descale), float(v_descale),
                     int(bool(causal)), od)
    with torch.cuda.device(dev):
        st = fa_fwd_fp8_ex(p, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_fwd_fp8_ex")
    return out, lse


def backward_noalloc(q, k, v, o, lse, do, causal=False, scale=None, dq=None, dk=None, dv=None, stream=None):
    """dQ, dK, dV through fa_bwd_noalloc: the backward that takes no workspace
    and uses the library's built-in device scratch (64 MiB per device;
    larger problems raise with FA_ERR_SCRATCH_LIMIT). The tensors must be
    dense [B, S, H, D] (the entry point takes no strides). Calls that overlap
    on the GPU share that scratch and race: see include/fa.h."""
    B, Sq, H, D, Sk = _dims(q, k)
    dt = _dtype_code(q)
    dev = q.device
    if not q.is_cuda:
        raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
    for name, t, S in (("q", q, Sq), ("k", k, Sk), ("v", v, Sk), ("o", o, Sq), ("do", do, Sq)):
        _expect(name, t, (B, S, H, D), q.dtype, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be a dense [B, S, H, D] tensor for fa_bwd_noalloc")
    _expect_lse(lse, B, H, Sq, dev)
    if scale is None:
        scale = D ** -0.5
    dq = torch.empty((B, Sq, H, D), dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty((B, Sk, H, D), dtype=q.dtype, device=dev) if dk is None else dk
    dv = torch.empty((B, Sk, H, D), dtype=q.dtype, device=dev) if dv is None else dv
    for name, t, S in (("dq", dq, Sq), ("dk", dk, Sk), ("dv", dv, Sk)):
        _expect(name, t, (B, S, H, D), q.dtype, dev)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be a dense [B, S, H, D] tensor for fa_bwd_noalloc")
    with torch.cuda.device(dev):
        st = fa_bwd_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
                            dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Sq, Sk, D, float(scale),
                            int(bool(causal)), dt, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_noalloc")
    return dq, dk, dv


def workspace_for(B, H, Sq, D, device, Sk=None, deterministic=False) -> torch.Tensor:
    if deterministic:
        n = fa_bwd_workspace_size_ex(B, H, Sq, Sq if Sk is None else Sk, D, 1)
    else:
        n = fa_bwd_workspace_size(B, H, Sq, D)
    return torch.empty(n, dtype=torch.uint8, device=device)


def backward(q, k, v, o, lse, do, causal=False, scale=None, dq=None, dk=None, dv=None,
             workspace=None, stream=None, deterministic=False):
    """dQ, dK, dV of L = sum(dO * O) for O = attention(q, k, v).
    ``deterministic=True`` sums dQ in a fixed order (bit-identical runs; more
    workspace and time)."""
    B, Sq, H, D, Sk = _dims(q, k)
    dt = _dtype_code(q)
    dev = q.device
    _expect("k", k, (B, Sk, H, D), q.dtype, dev)
    _expect("v", v, (B, Sk, H, D), q.dtype, dev)
    _expect("o", o, (B, Sq, H, D), q.dtype, dev)
    _expect("do", do, (B, Sq, H, D), q.dtype, dev)
    _expect_lse(lse, B, H, Sq, dev)
    if scale is None:
        scale = D ** -0.5
    dq = torch.empty((B, Sq, H, D), dtype=q.dtype, device=dev) if dq is None else dq
    dk = torch.empty((B, Sk, H, D), dtype=q.dtype, device=dev) if dk is None else dk
    dv = torch.empty((B, Sk, H, D), dtype=q.dtype, device=dev) if dv is None else dv
    _expect("dq", dq, (B, Sq, H, D), q.dtype, dev)
    _expect("dk", dk, (B, Sk, H, D), q.dtype, dev)
    _expect("dv", dv, (B, Sk, H, D), q.dtype, dev)
    if workspace is None:
        workspace = workspace_for(B, H, Sq, D, dev, Sk=Sk, deterministic=deterministic)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous buffer on {dev}")
    ws_bytes = workspace.numel() * workspace.element_size()
    p = BwdParams(_view(q), _view(k), _view(v), _view(o), _view(do), lse.data_ptr(),
                  _view(dq), _view(dk), _view(dv), B, H, Sq, Sk, D, float(scale),
                  int(bool(causal)), dt, workspace.data_ptr(), ws_bytes, int(bool(deterministic)))
    with torch.cuda.device(dev):
        st = fa_bwd_ex(p, _stream(stream))
    if st != FA_OK:
        raise FaError(st, "fa_bwd_ex")
    return dq, dk, dv


# ------------------------------------- differential attention, rotary positions
# These helpers are called on single tokens, where the GPU's part is a few
# microseconds, so they spend little on the host: parameter structs are packed
# in one step (the layouts of DiffFwdParams, DiffBwdParams and RotaryParams;
# "@" pads as the C compiler does), tensors are asked for their shape and
# strides once, and the detailed checks run only where a quick one fails.
_T = "Pqqq"  # fa_tensor
_LAM = "Pqqqiiii"  # fa_diff_lambda
_DIFF_FWD = struct.Struct("@" + 5 * _T + _LAM + "P" + 2 * _T + "P7ifiiPN")
_DIFF_BWD = struct.Struct("@" + 8 * _T + "P" + _LAM + 5 * _T + "P7ifiiPNi0P")
_ROTARY = struct.Struct("@" + 4 * _T + f"PqqqiPii{FA_ROTARY_MAX_AXES}i8i0P")
_NO_TENSOR = (0, 0, 0, 0)


@contextlib.contextmanager
def _on(dev, stream):
    """Makes `dev` current, and the caller's stream (if any) torch's current
    one, so that what the helper allocates belongs to the stream that uses it."""
    with torch.cuda.device(dev):
        if stream is None:
            yield
            return
        if not isinstance(stream, torch.cuda.Stream):
            raw = _stream(stream)
            stream = torch.cuda.ExternalStream(raw, device=dev) if raw else torch.cuda.default_stream(dev)
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, q on {dev}")
        with torch.cuda.stream(stream):
            yield


def _elsewhere(dev, stream) -> bool:
    """Whether a call has to change the current device or stream first."""
    if dev.type != "cuda":
        raise ValueError("tensors must live on a CUDA device (the library has no CPU path)")
    return stream is not None or dev.index != torch.cuda.current_device()


try:  # the handle alone, without a Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:  # a torch without CUDA, or without this function
    def _raw_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


def _flat(name: str, t: torch.Tensor):
    """fa_tensor of a [B, S, H, D] view."""
    sb, ss, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    return t.data_ptr(), sb, ss, sh


def _pair(name: str, t: torch.Tensor):
    """The two maps' fa_tensors of a [B, S, H, 2, D] view of 16-bit values."""
    sb, ss, sh, sc, sd = t.stride()
    if sd != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")
    at = t.data_ptr()
    return at, sb, ss, sh, at + 2 * sc, sb, ss, sh


def _need(name: str, t: torch.Tensor, shape, dtype, dev) -> None:
    if t.shape != shape or t.dtype is not dtype or t.device != dev:
        _expect(name, t, shape, dtype, dev)


def _diff_dims(q, k, v):
    if q.dim() != 5 or k.dim() != 5 or v.dim() != 4 or q.shape[3] != 2 or k.shape[3] != 2:
        raise ValueError("expected q [B, Sq, H, 2, D], k [B, Sk, Hk, 2, D] and v [B, Sk, Hk, Dv]")
    B, Sq, H, _, D = q.shape
    _, Sk, Hk, Dv = v.shape
    dt, dev = _dtype_code(q), q.device
    _need("k", k, (B, Sk, Hk, 2, D), q.dtype, dev)
    _need("v", v, (B, Sk, Hk, Dv), q.dtype, dev)
    if Hk < 1 or H % Hk:
        raise ValueError(f"{H} query heads cannot share {Hk} key heads evenly")
    return B, Sq, H, D, Sk, Hk, Dv, dt, dev


def _lambda(lam, B, Sq, H, dtype, dev):
    if not isinstance(lam, torch.Tensor) or lam.dim() > 3:
        raise ValueError("lam must be a tensor that broadcasts to [B, Sq, H]")
    none = 3 - lam.dim()
    eb, es, eh = (1,) * none + tuple(lam.shape)
    if (eb != 1 and eb != B) or (es != 1 and es != Sq) or (eh != 1 and eh != H):
        raise ValueError(f"lam: {tuple(lam.shape)} does not broadcast to [{B}, {Sq}, {H}]")
    if lam.dtype is not torch.float32 and lam.dtype is not dtype:
        raise TypeError(f"lam: expected float32 or {dtype}, got {lam.dtype}")
    if lam.device != dev:
        raise ValueError(f"lam is on {lam.device}, q on {dev}")
    code = FA_LAMBDA_FP32 if lam.dtype is torch.float32 else _DT[lam.dtype]
    return (lam.data_ptr(), *((0,) * none + lam.stride()), eb, es, eh, code)


def _diff_lse(lse, B, H, Sq, dev):
    _need("lse", lse, (2, B, H, Sq), torch.float32, dev)
    if not lse.is_contiguous():
        raise ValueError("lse must be a contiguous fp32 [2, B, H, Sq] tensor")


def _ws(workspace, dev):
    """(address, bytes) of a workspace, or of none."""
    if workspace is None:
        return 0, 0
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous buffer on {dev}")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def diff_forward(q, k, v, lam, causal=False, scale=None, k_lens=None, need_o2=False, out=None, out2=None, lse=None,
                 workspace=None, stream=None):
    """(O, LSE, O2) of differential attention,
    O = (softmax(scale q_1 k_1^T) - lam softmax(scale q_2 k_2^T)) v.

    q [B, Sq, H, 2, D], k [B, Sk, Hk, 2, D] and v [B, Sk, Hk, Dv] are CUDA
    tensors (strided views allowed), D <= 64, Dv <= 128; Hk divides H. lam
    (float32 or q's dtype) broadcasts to [B, Sq, H]. k_lens, int32 [B]: batch
    entry b attends to its first k_lens[b] keys, and the causal mask aligns to
    that end. LSE is fp32 [2, B, H, Sq]. O2 = softmax(scale q_2 k_2^T) v is
    written if need_o2 or out2 asks for it (diff_backward needs it), else None."""
    B, Sq, H, D, Sk, Hk, Dv, dt, dev = _diff_dims(q, k, v)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return diff_forward(q, k, v, lam, causal, scale, k_lens, need_o2, out, out2, lse, workspace)
    lp = _lambda(lam, B, Sq, H, q.dtype, dev)
    if k_lens is not None:
        _need("k_lens", k_lens, (B,), torch.int32, dev)
        if not k_lens.is_contiguous():
            raise ValueError("k_lens must be contiguous")
    shape, causal = (B, Sq, H, Dv), 1 if causal else 0
    if out is None:
        out = q.new_empty(shape)
    else:
        _need("out", out, shape, q.dtype, dev)
    if out2 is not None:
        _need("out2", out2, shape, q.dtype, dev)
    elif need_o2:
        out2 = q.new_empty(shape)
    if lse is None:
        lse = torch.empty((2, B, H, Sq), dtype=torch.float32, device=dev)
    else:
        _diff_lse(lse, B, H, Sq, dev)
    if workspace is None and Sq <= 16:  # calls of more rows need none
        n = fa_diff_fwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev) if n else None
    p = _DIFF_FWD.pack(*_pair("q", q), *_pair("k", k), *_flat("v", v), *lp,
                       0 if k_lens is None else k_lens.data_ptr(), *_flat("out", out),
                       *(_NO_TENSOR if out2 is None else _flat("out2", out2)), lse.data_ptr(),
                       B, H, Hk, Sq, Sk, D, Dv, D ** -0.5 if scale is None else float(scale), causal, dt,
                       *_ws(workspace, dev))
    st = _packed("fa_diff_fwd")(p, _raw_stream(dev.index))
    if st != FA_OK:
        raise FaError(st, "fa_diff_fwd")
    return out, lse, out2


def diff_backward(q, k, v, lam, o, o2, lse, do, causal=False, scale=None, dq=None, dk=None, dv=None, dlam=None,
                  workspace=None, stream=None, deterministic=False):
    """(dQ, dK, dV, dLam) of L = sum(dO * O) for O of diff_forward, whose o, o2
    and lse it takes. dLam has lam's shape and dtype: the gradient is summed
    over the axes lam is broadcast over. ``deterministic=True`` sums dQ in a
    fixed order (dK, dV and dLam always are)."""
    B, Sq, H, D, Sk, Hk, Dv, dt, dev = _diff_dims(q, k, v)
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return diff_backward(q, k, v, lam, o, o2, lse, do, causal, scale, dq, dk, dv, dlam, workspace, None,
                                 deterministic)
    lp = _lambda(lam, B, Sq, H, q.dtype, dev)
    shape, det = (B, Sq, H, Dv), 1 if deterministic else 0
    for name, t in (("o", o), ("o2", o2), ("do", do)):
        _need(name, t, shape, q.dtype, dev)
    _diff_lse(lse, B, H, Sq, dev)
    grads = []
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v), ("dlam", dlam, lam)):
        if t is None:
            t = like.new_empty(like.shape)
        else:
            _need(name, t, like.shape, like.dtype, dev)
        grads.append(t)
    dq, dk, dv, dlam = grads
    if not dlam.is_contiguous():
        raise ValueError("dlam must be contiguous")
    causal = 1 if causal else 0
    if workspace is None:
        n = fa_diff_bwd_workspace_size(B, H, Hk, Sq, Sk, D, Dv, causal, det)
        workspace = torch.empty(n, dtype=torch.uint8, device=dev)
    p = _DIFF_BWD.pack(*_pair("q", q), *_pair("k", k), *_flat("v", v), *_flat("o", o), *_flat("o2", o2),
                       *_flat("do", do), lse.data_ptr(), *lp, *_pair("dq", dq), *_pair("dk", dk), *_flat("dv", dv),
                       dlam.data_ptr(), B, H, Hk, Sq, Sk, D, Dv, D ** -0.5 if scale is None else float(scale),
                       causal, dt, *_ws(workspace, dev), det)
    st = _packed("fa_diff_bwd")(p, _raw_stream(dev.index))
    if st != FA_OK:
        raise FaError(st, "fa_diff_bwd")
    return dq, dk, dv, dlam


def rotary_inv_freq(sections, base=10000.0, per_axis=False, device="cuda") -> torch.Tensor:
    """fp64 [R] frequencies base^(-j / R) of R = sum(sections) pairs; with
    per_axis every axis has a ladder of its own, base^(-j / sections[axis])."""
    counts = list(sections) if per_axis else [sum(sections)]
    return torch.tensor([float(base) ** (-j / n) for n in counts for j in range(n)], dtype=torch.float64,
                        device=device)


def _heads(name: str, t: torch.Tensor, B, S, D, dtype, dev):
    """(heads, fa_tensor) of [B, S, heads, D], or of [B, S, H, 2, D] with the two maps as neighbouring heads."""
    if t.dim() == 5:
        try:
            t = t.view(t.shape[0], t.shape[1], -1, t.shape[4])
        except RuntimeError:
            raise ValueError(f"{name}: the head axes of [B, S, H, 2, D] must be one run of heads") from None
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, S, heads, D] or [B, S, H, 2, D]")
    n = t.shape[2]
    _need(name, t, (B, S, n, D), dtype, dev)
    return n, _flat(name, t)


def rotary(q, k, positions, inv_freq, sections=None, interleaved=False, inverse=False, out_q=None, out_k=None,
           stream=None):
    """(q, k) with rotary positions of one or more axes applied: R pairs of
    columns of every head turn by positions[axis] * inv_freq[pair].

    q and k (or None) are fp16/bf16 CUDA tensors [B, S, heads, D] (strided views
    allowed), or [B, S, H, 2, D] as differential attention takes them. positions
    is int32 or int64 [axes, B, S] ([B, S] for one axis; expanded axes allowed),
    inv_freq fp32 or fp64 [R]; sections gives the pairs of each axis (default:
    all on the only axis). Pairs are columns (j, j + R), or (2j, 2j + 1) if
    interleaved; columns from 2R on are copied. inverse turns back: it is also
    the gradient. out_q may be q and out_k may be k (in place)."""
    dt, dev, dtype = _dtype_code(q), q.device, q.dtype
    if _elsewhere(dev, stream):
        with _on(dev, stream):
            return rotary(q, k, positions, inv_freq, sections, interleaved, inverse, out_q, out_k)
    B, S, D = q.shape[0], q.shape[1], q.shape[-1]
    H, vq = _heads("q", q, B, S, D, dtype, dev)
    Hk, vk = _heads("k", k, B, S, D, dtype, dev) if k is not None else (0, _NO_TENSOR)
    if positions.dim() == 2:
        positions = positions[None]
    if positions.dim() != 3 or positions.shape[1:] != (B, S):
        raise ValueError(f"positions: expected [axes, {B}, {S}], got {tuple(positions.shape)}")
    if positions.dtype not in (torch.int32, torch.int64):
        raise TypeError(f"positions: expected int32 or int64, got {positions.dtype}")
    if inv_freq.dtype not in (torch.float32, torch.float64):
        raise TypeError(f"inv_freq: expected float32 or float64, got {inv_freq.dtype}")
    if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous [pairs] tensor")
    for name, t in (("positions", positions), ("inv_freq", inv_freq)):
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, q on {dev}")
    axes, pairs = positions.shape[0], inv_freq.shape[0]
    sections = (pairs,) if sections is None else tuple(sections)
    if len(sections) != axes or not 1 <= axes <= FA_ROTARY_MAX_AXES:
        raise ValueError(f"sections: expected one entry for each of 1 to {FA_ROTARY_MAX_AXES} axes, got "
                         f"{len(sections)} for {axes}")
    if sum(sections) != pairs or min(sections) < 0:
        raise ValueError(f"sections {sections} do not add up to inv_freq's {pairs} pairs")
    if 2 * pairs > D:
        raise ValueError(f"{pairs} pairs do not fit into {D} columns")
    if out_q is None:
        out_q = q.new_empty(q.shape)
    elif out_q.shape != q.shape:
        _expect("out_q", out_q, q.shape, dtype, dev)
    if k is None:
        if out_k is not None:
            raise ValueError("out_k without k")
        wk = _NO_TENSOR
    else:
        if out_k is None:
            out_k = k.new_empty(k.shape)
        elif out_k.shape != k.shape:
            _expect("out_k", out_k, k.shape, dtype, dev)
        wk = _heads("out_k", out_k, B, S, D, dtype, dev)[1]
    p = _ROTARY.pack(*vq, *vk, *_heads("out_q", out_q, B, S, D, dtype, dev)[1], *wk, positions.data_ptr(),
                     *positions.stride(), 1 if positions.dtype is torch.int64 else 0, inv_freq.data_ptr(),
                     1 if inv_freq.dtype is torch.float64 else 0, axes,
                     *sections, *(0,) * (FA_ROTARY_MAX_AXES - axes), B, S, H, Hk, D,
                     1 if interleaved else 0, 1 if inverse else 0, dt)
    st = _packed("fa_rotary")(p, _raw_stream(dev.index))
    if st != FA_OK:
        raise FaError(st, "fa_rotary")
    return out_q, out_k
