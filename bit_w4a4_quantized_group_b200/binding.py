"""Binding of libsvdq (argument marshalling only): ctypes, and a small CPython extension for the hot calls.

Every function keeps the name of the C entry point in ``include/svdq.h``.
The ``*_t`` helpers take torch tensors and pass their data pointers and the
current CUDA stream.  Those of the prologue and the GEMM check nothing the library does not
check itself; those of the row operators also compare types, shapes, devices and buffer sizes.
Loading fails loudly when the library is missing: there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libsvdq.so")
CALLS_PATH = os.path.join(_PKG, "_lib", "svdq_call.so")

SVDQ_OK, SVDQ_ERR_INVALID_ARG, SVDQ_ERR_UNSUPPORTED, SVDQ_ERR_CUDA, SVDQ_ERR_TIMEOUT = range(5)
SVDQ_FMT_NVFP4_G16 = 1
SVDQ_FMT_INT4_G64 = 2
SVDQ_FMT_MXFP4_G32 = 3
SVDQ_FMT_W8A8 = 4
SVDQ_FMT_FP8_G128 = 5
FORMATS = {"nvfp4": SVDQ_FMT_NVFP4_G16, "int4": SVDQ_FMT_INT4_G64, "mxfp4": SVDQ_FMT_MXFP4_G32,
           "w8a8": SVDQ_FMT_W8A8, "fp8": SVDQ_FMT_FP8_G128}
SVDQ_ACT_SILU, SVDQ_ACT_GELU_TANH = 1, 2
ACTIVATIONS = {"silu": SVDQ_ACT_SILU, "gelu": SVDQ_ACT_GELU_TANH}

EXPORTED = (
    "svdq_buffer_sizes", "svdq_pack_weight", "svdq_quantize_act_lowrank_down",
    "svdq_w4a4_gemm_lowrank_up", "svdq_rmsnorm_quantize_act", "svdq_glu_quantize_act", "svdq_status_string", "svdq_get_last_device_error",
    "svdq_last_launch_count", "svdq_last_variant", "svdq_last_cuda_error", "svdq_selftest_bounded_wait",
)


class svdq_sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("x", "a_codes", "a_scales", "z", "w_codes", "w_scales", "l1", "l2", "bias", "y")]


class SvdqError(RuntimeError):
    def __init__(self, status: int, what: str):
        detail = f" [{svdq_last_cuda_error()}]" if status == SVDQ_ERR_CUDA else ""
        super().__init__(f"{what}: {status_name(status)} ({status}){detail}")
        self.status = status


_lib = None
_calls = None     # what makes the hot calls, see _bind_calls


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libsvdq.so (raises if it has not been built)."""
    global _lib, _calls
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libsvdq.so not found at {path}; run python -m bit_w4a4_quantized_group_b200.build")
    lib = ctypes.CDLL(path)
    vp, i64, c_int, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    lib.svdq_buffer_sizes.argtypes = [c_int, i64, i64, i64, c_int, ctypes.POINTER(svdq_sizes)]
    lib.svdq_pack_weight.argtypes = [c_int, i64, i64, c_int, f32, vp, vp, vp, vp, vp,
                                     ctypes.POINTER(ctypes.c_float), vp, vp]
    lib.svdq_quantize_act_lowrank_down.argtypes = [c_int, i64, i64, c_int, vp, vp, f32, vp, vp, vp, vp, vp]
    lib.svdq_w4a4_gemm_lowrank_up.argtypes = [c_int, i64, i64, i64, c_int, vp, vp, f32, vp, vp, f32,
                                              vp, vp, vp, vp, vp]
    lib.svdq_rmsnorm_quantize_act.argtypes = [c_int, i64, i64, vp, i64, vp, i64, vp, f32, vp, i64, vp, vp, vp]
    lib.svdq_glu_quantize_act.argtypes = [c_int, c_int, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp]
    lib.svdq_status_string.argtypes = [c_int]
    lib.svdq_status_string.restype = ctypes.c_char_p
    lib.svdq_get_last_device_error.argtypes = [vp, ctypes.POINTER(c_int)]
    lib.svdq_last_launch_count.argtypes = []
    lib.svdq_last_variant.argtypes = []
    lib.svdq_last_cuda_error.argtypes = []
    lib.svdq_last_cuda_error.restype = ctypes.c_char_p
    lib.svdq_selftest_bounded_wait.argtypes = [i64, vp]
    for name in EXPORTED:
        if name not in ("svdq_status_string", "svdq_last_cuda_error"):
            getattr(lib, name).restype = c_int
    _lib = lib
    _calls = _bind_calls(lib)
    return lib


def _bind_calls(lib):
    """The four hot entry points (prologue, GEMM and the two row operators): through the extension
    svdq_call, which converts their arguments ten times as fast as ctypes, or, where that was not
    built, through ctypes.  The same functions with the same positional arguments either way."""
    if not os.path.exists(CALLS_PATH):
        return lib
    from importlib.machinery import ExtensionFileLoader
    from importlib.util import module_from_spec, spec_from_loader
    loader = ExtensionFileLoader("svdq_call", CALLS_PATH)
    try:
        mod = module_from_spec(spec_from_loader("svdq_call", loader))
        loader.exec_module(mod)
    except ImportError:              # built for another Python
        return lib
    mod.bind(*(ctypes.cast(getattr(lib, n), ctypes.c_void_p).value for n in
               ("svdq_quantize_act_lowrank_down", "svdq_w4a4_gemm_lowrank_up", "svdq_rmsnorm_quantize_act",
                "svdq_glu_quantize_act")))
    return mod


def _hot():
    load()
    return _calls


def status_name(status: int) -> str:
    return load().svdq_status_string(int(status)).decode()


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


# ----------------------------------------------------------------- raw entry points

def svdq_buffer_sizes(fmt, M: int, N: int, K: int, rank: int) -> svdq_sizes:
    out = svdq_sizes()
    st = load().svdq_buffer_sizes(_fmt(fmt), M, N, K, rank, ctypes.byref(out))
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_buffer_sizes")
    return out


def svdq_pack_weight(fmt, N, K, rank, act_gscale, R, L1, L2, w_codes, w_scales, w_gscale, L1_bf16, L2_bf16) -> int:
    return load().svdq_pack_weight(_fmt(fmt), N, K, rank, act_gscale, R, L1, L2, w_codes, w_scales,
                                   w_gscale, L1_bf16, L2_bf16)


def svdq_quantize_act_lowrank_down(fmt, M, K, rank, X, lam, act_gscale, L1, a_codes, a_scales, Z, stream) -> int:
    return load().svdq_quantize_act_lowrank_down(_fmt(fmt), M, K, rank, X, lam, act_gscale, L1, a_codes,
                                                 a_scales, Z, stream)


def svdq_w4a4_gemm_lowrank_up(fmt, M, N, K, rank, a_codes, a_scales, act_gscale, w_codes, w_scales, w_gscale,
                              Z, L2, bias, Y, stream) -> int:
    return load().svdq_w4a4_gemm_lowrank_up(_fmt(fmt), M, N, K, rank, a_codes, a_scales, act_gscale, w_codes,
                                            w_scales, w_gscale, Z, L2, bias, Y, stream)


def svdq_rmsnorm_quantize_act(fmt, M, K, X, ldx, residual, ldr, gamma, eps, H, ldh, a_codes, a_scales, stream) -> int:
    return load().svdq_rmsnorm_quantize_act(_fmt(fmt), M, K, X, ldx, residual, ldr, gamma, eps, H, ldh, a_codes,
                                            a_scales, stream)


def svdq_glu_quantize_act(fmt, act, M, K, gate, ldg, up, ldu, lam, a_codes, a_scales, stream) -> int:
    return load().svdq_glu_quantize_act(_fmt(fmt), ACTIVATIONS[act] if isinstance(act, str) else int(act), M, K,
                                        gate, ldg, up, ldu, lam, a_codes, a_scales, stream)


def svdq_get_last_device_error(stream=None):
    site = ctypes.c_int(0)
    st = load().svdq_get_last_device_error(stream, ctypes.byref(site))
    return st, site.value


def svdq_selftest_bounded_wait(limit_ns: int, stream=None) -> int:
    return load().svdq_selftest_bounded_wait(int(limit_ns), stream)


def svdq_last_launch_count() -> int:
    return load().svdq_last_launch_count()


def svdq_last_variant() -> int:
    return load().svdq_last_variant()


def svdq_last_cuda_error() -> str:
    return load().svdq_last_cuda_error().decode()


# ----------------------------------------------------------------- torch helpers

_C = None     # torch._C, once a helper has needed it


def _stream():
    """Raw handle of torch's current stream on the current device.  Read without building a
    torch.cuda.Stream object (3 us), which would cost as much as the launch of a small call."""
    global _C
    if _C is None:
        import torch
        torch.cuda.current_device()            # initialises CUDA on first use
        _C = torch._C
    return _C._cuda_getCurrentRawStream(_C._cuda_getDevice())


def _check(st: int, what: str):
    if st != SVDQ_OK:
        raise SvdqError(st, what)


def pack_weight_np(fmt, R_nk, L1_rk, L2_nr, act_gscale: float = 1.0):
    """Host pack from NumPy float32 arrays; returns NumPy outputs and g_w."""
    import numpy as np
    N, K = R_nk.shape
    rank = 0 if L1_rk is None else L1_rk.shape[0]
    sz = svdq_buffer_sizes(fmt, 128, N, K, rank)
    R = np.ascontiguousarray(R_nk, dtype=np.float32)
    L1 = None if rank == 0 else np.ascontiguousarray(L1_rk, dtype=np.float32)
    L2 = None if rank == 0 else np.ascontiguousarray(L2_nr, dtype=np.float32)
    w_codes = np.zeros(sz.w_codes, np.uint8)
    w_scales = np.zeros(sz.w_scales, np.uint8)
    l1b = np.zeros(max(rank * K, 1), np.uint16)
    l2b = np.zeros(max(N * rank, 1), np.uint16)
    gw = ctypes.c_float(0.0)
    st = svdq_pack_weight(fmt, N, K, rank, act_gscale, R.ctypes.data,
                          None if L1 is None else L1.ctypes.data,
                          None if L2 is None else L2.ctypes.data,
                          w_codes.ctypes.data, w_scales.ctypes.data, ctypes.byref(gw),
                          l1b.ctypes.data, l2b.ctypes.data)
    _check(st, "svdq_pack_weight")
    return {"w_codes": w_codes, "w_scales": w_scales, "w_gscale": gw.value,
            "L1_bf16": l1b[: rank * K].reshape(rank, K), "L2_bf16": l2b[: N * rank].reshape(N, rank)}


def quantize_act_lowrank_down_t(fmt, X, lam, act_gscale, L1, a_codes, a_scales, Z, stream=None):
    """Device prologue on torch tensors (X [M, K] bf16, L1 [r, K] bf16 viewed as any 2-byte dtype).
    `stream` is a raw cudaStream_t handle; None means torch's current stream."""
    M, K = X.shape
    st = (_calls or _hot()).svdq_quantize_act_lowrank_down(
        _fmt(fmt), M, K, 0 if L1 is None else L1.shape[0], X.data_ptr(), None if lam is None else lam.data_ptr(),
        act_gscale, None if L1 is None else L1.data_ptr(), a_codes.data_ptr(), a_scales.data_ptr(),
        None if Z is None else Z.data_ptr(), _stream() if stream is None else stream)
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_quantize_act_lowrank_down")


def w4a4_gemm_lowrank_up_t(fmt, M, N, K, rank, a_codes, a_scales, act_gscale, w_codes, w_scales, w_gscale,
                           Z, L2, bias, Y, stream=None):
    st = (_calls or _hot()).svdq_w4a4_gemm_lowrank_up(
        _fmt(fmt), M, N, K, rank, a_codes.data_ptr(), a_scales.data_ptr(), act_gscale, w_codes.data_ptr(),
        w_scales.data_ptr(), w_gscale, None if Z is None else Z.data_ptr(), None if L2 is None else L2.data_ptr(),
        None if bias is None else bias.data_ptr(), Y.data_ptr(), _stream() if stream is None else stream)
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_w4a4_gemm_lowrank_up")


def _current_device() -> int:
    global _C
    if _C is None:
        import torch
        _C = torch._C
    return _C._cuda_getDevice()


def _row_ld(t, shape, dtype, dev, name):
    """Row stride in elements of a matrix of a call: of that shape and type, on that device, its rows
    contiguous (a single row's stride is its length)."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on device {dev}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return ld if shape[0] > 1 else shape[1]


def _column_vector(t, K, dev, name):
    """Pointer of an fp32 [K] vector (gamma, lambda) on that device; None for None."""
    if t is None:
        return None
    if t.dtype is not (_f32 or _float32()) or t.numel() != K or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous float32 [{K}] on device {dev}, got {tuple(t.shape)} {t.dtype} "
                         f"on {t.device}")
    return t.data_ptr()


_f32 = None
_bf16 = None


def _float32():
    global _f32
    if _f32 is None:
        import torch
        _f32 = torch.float32
    return _f32


def _bfloat16():
    global _bf16
    if _bf16 is None:
        import torch
        _bf16 = torch.bfloat16
    return _bf16


def _fp8_outputs(codes, scales, M, K, dev):
    """Pointers of the buffers that a row operator writes: dense, of a one-byte type (uint8, or the float8 type
    that the bytes stand for), on that device, M K bytes for the codes and
    ceil(M / 128) * 128 * ceil(K / 512) * 4 for the scales, or more."""
    if (codes.element_size() != 1 or codes.nbytes < M * K or codes.get_device() != dev or not codes.is_contiguous()
            or scales.element_size() != 1 or scales.nbytes < (M + 127 >> 7) * (K + 511 >> 9) * 512
            or scales.get_device() != dev or not scales.is_contiguous()):
        raise ValueError(f"a_codes, a_scales: expected contiguous uint8 (or float8) of at least {M * K} and "
                         f"{(M + 127 >> 7) * (K + 511 >> 9) * 512} elements on device {dev}, got "
                         f"{tuple(codes.shape)} {codes.dtype} on {codes.device} and {tuple(scales.shape)} "
                         f"{scales.dtype} on {scales.device}")
    return codes.data_ptr(), scales.data_ptr()


def _first_matrix(t, name):
    """(shape, type, device, row stride) of a call's first matrix: bf16, the one type that the row
    operators read, and on the current CUDA device, where the library launches (checked by the caller)."""
    shape, dtype, dev = t.shape, t.dtype, t.get_device()
    if dtype is not (_bf16 or _bfloat16()) or len(shape) != 2:
        raise ValueError(f"{name}: expected bfloat16 [M, K], got {tuple(shape)} {dtype}")
    ld, step = t.stride()
    if step != 1 and shape[1] > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return shape, dtype, dev, ld if shape[0] > 1 else shape[1]


def rmsnorm_quantize_act_t(fmt, X, residual, gamma, eps, H, a_codes, a_scales, stream=None):
    """Residual addition + RMS norm + quantization on torch tensors: X, residual, H bf16 [M, K] (rows
    may be strided; residual and H may be None), gamma fp32 [K] or None.  a_codes and a_scales are dense
    uint8 (or float8), at least as long as svdq_buffer_sizes says."""
    shape, dtype, dev, ldx = _first_matrix(X, "X")
    r = h = None
    ldr = ldh = 0
    if residual is not None:
        ldr, r = _row_ld(residual, shape, dtype, dev, "residual"), residual.data_ptr()
    if H is not None:
        ldh, h = _row_ld(H, shape, dtype, dev, "H"), H.data_ptr()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"expected tensors on the current CUDA device, got one on {X.device}")
    M, K = shape
    codes, scales = _fp8_outputs(a_codes, a_scales, M, K, dev)
    st = (_calls or _hot()).svdq_rmsnorm_quantize_act(
        _fmt(fmt), M, K, X.data_ptr(), ldx, r, ldr, _column_vector(gamma, K, dev, "gamma"), eps, h, ldh, codes, scales,
        _stream() if stream is None else stream)
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_rmsnorm_quantize_act")


def glu_quantize_act_t(fmt, act, gate, up, lam, a_codes, a_scales, stream=None):
    """act(gate) [* up] [/ lam] + quantization on torch tensors: act "silu" or "gelu" (tanh form), gate
    and up bf16 [M, K] (column slices of a wider tensor will do; up may be None), lam fp32 [K] or None.
    a_codes and a_scales as in rmsnorm_quantize_act_t."""
    code = ACTIVATIONS[act]
    shape, dtype, dev, ldg = _first_matrix(gate, "gate")
    u, ldu = None, 0
    if up is not None:
        ldu, u = _row_ld(up, shape, dtype, dev, "up"), up.data_ptr()
    if dev < 0 or dev != _current_device():
        raise ValueError(f"expected tensors on the current CUDA device, got one on {gate.device}")
    M, K = shape
    codes, scales = _fp8_outputs(a_codes, a_scales, M, K, dev)
    st = (_calls or _hot()).svdq_glu_quantize_act(
        _fmt(fmt), code, M, K, gate.data_ptr(), ldg, u, ldu, _column_vector(lam, K, dev, "lam"), codes, scales,
        _stream() if stream is None else stream)
    if st != SVDQ_OK:
        raise SvdqError(st, "svdq_glu_quantize_act")
