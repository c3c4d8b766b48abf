"""Python binding of libpipegemm, the software-pipelined GEMM library for GB300.

Argument marshalling only: every function here forwards to the C ABI declared
in ``include/pgemm.h`` (same names), and all arithmetic runs in the library's
CUDA kernels.  There is no fallback: if ``libpipegemm.so`` has not been built,
``lib()`` raises.

Operands may be given as torch tensors (CUDA, contiguous, row-major) or as raw
device pointers (ints).  ``stream`` defaults to torch's current stream when
torch is importable, else the legacy default stream.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "PgemmError", "lib", "library_path", "gemm_f32", "gemm_bf16", "gemm_i8", "gemm_f32_ex",
    "gemm_bf16_ex", "gemm_i8_ex", "pgemm_default_config", "pgemm_list_configs",
    "pgemm_kernel_attrs", "pgemm_get_device_status", "pgemm_selftest_wait_timeout",
    "pgemm_status_string", "pgemm_version", "gemm_i8_noalloc", "NOALLOC_SCRATCH_BYTES",
    "pgemm_stage_reuse_demo", "pgemm_schedule", "pgemm_stream_k_plan", "pgemm_trim_scratch",
    "DTYPES", "STATUS", "EXPORTED", "PRODUCERS", "ENGINES", "ACTIVATIONS",
    "linear_bf16", "linear_bf16_backward", "gated_bf16", "gated_bf16_backward", "xent_bf16",
    "xent_bf16_grad", "rmsnorm_bf16", "rmsnorm_i8", "rmsnorm_bf16_backward", "route_topk",
    "route_topk_backward", "expert_sort", "expert_gather_bf16", "expert_combine_bf16",
    "expert_combine_bf16_backward", "experts_linear_bf16", "experts_linear_bf16_backward",
    "experts_gated_bf16", "experts_gated_bf16_backward",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libpipegemm.so")

STATUS = {
    0: "PGEMM_OK", 1: "PGEMM_ERR_INVALID_VALUE", 2: "PGEMM_ERR_MISALIGNED",
    3: "PGEMM_ERR_UNSUPPORTED_DEVICE", 4: "PGEMM_ERR_CUDA", 5: "PGEMM_ERR_TIMEOUT",
    6: "PGEMM_ERR_UNSUPPORTED_CONFIG", 7: "PGEMM_ERR_TOO_LARGE",
}
# Size of the fixed device array gemm_i8_noalloc widens its operands into.
NOALLOC_SCRATCH_BYTES = 32 << 20
DTYPES = {"f32": 0, "bf16": 1, "i8": 2}
# pgemm_producer: who fills the shared-memory stages
PRODUCERS = {"tma": 0, "registers": 1, "staged": 2, "widen_in_kernel": 3}
# pgemm_engine: which multiply-accumulate consumes the stages
ENGINES = {"default": 0, "mma_sync": 1}
# pgemm_act: the activations of the operators
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
# Every function include/pgemm.h declares.
EXPORTED = [
    "gemm_f32", "gemm_bf16", "gemm_i8", "gemm_f32_ex", "gemm_bf16_ex", "gemm_i8_ex",
    "pgemm_default_config", "pgemm_list_configs", "pgemm_kernel_attrs",
    "pgemm_get_device_status", "pgemm_selftest_wait_timeout", "pgemm_status_string",
    "pgemm_version", "gemm_i8_noalloc", "pgemm_stage_reuse_demo", "pgemm_schedule",
    "pgemm_stream_k_plan", "pgemm_trim_scratch",
    "linear_bf16", "linear_bf16_backward", "gated_bf16", "gated_bf16_backward", "xent_bf16",
    "xent_bf16_grad", "rmsnorm_bf16", "rmsnorm_i8", "rmsnorm_bf16_backward", "route_topk",
    "route_topk_backward", "expert_sort", "expert_gather_bf16", "expert_combine_bf16",
    "expert_combine_bf16_backward", "experts_linear_bf16", "experts_linear_bf16_backward",
    "experts_gated_bf16", "experts_gated_bf16_backward",
]


class PgemmError(RuntimeError):
    """A non-OK pgemm_status."""

    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class Config(ctypes.Structure):
    """pgemm_config.  A tuple (bm, bn, bk, stages[, max_k_parts[, producer[,
    engine[, group_m]]]]) converts to it."""
    _fields_ = [("bm", ctypes.c_int), ("bn", ctypes.c_int), ("bk", ctypes.c_int),
                ("stages", ctypes.c_int), ("max_k_parts", ctypes.c_int),
                ("producer", ctypes.c_int), ("engine", ctypes.c_int), ("group_m", ctypes.c_int)]

    def as_tuple(self):
        """The kernel the configuration names: (bm, bn, bk, stages), with
        (..., max_k_parts, producer, engine) appended when the producer or
        the engine is not the default, and group_m after them when set."""
        if self.group_m:
            return (self.bm, self.bn, self.bk, self.stages, self.max_k_parts, self.producer,
                    self.engine, self.group_m)
        if self.producer or self.engine:
            return (self.bm, self.bn, self.bk, self.stages, self.max_k_parts, self.producer,
                    self.engine)
        return (self.bm, self.bn, self.bk, self.stages)


_lock = threading.Lock()
_lib = None


def _declare(L: ctypes.CDLL) -> ctypes.CDLL:
    i, f, vp, i32 = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_int32
    ll = ctypes.c_longlong
    cfgp = ctypes.POINTER(Config)
    ip = ctypes.POINTER(ctypes.c_int)
    llp = ctypes.POINTER(ctypes.c_longlong)
    sig = {
        "gemm_f32": [i, i, i, f, vp, vp, f, vp, vp],
        "gemm_bf16": [i, i, i, f, vp, vp, f, vp, vp],
        "gemm_i8": [i, i, i, i32, vp, vp, i32, vp, vp],
        "gemm_i8_noalloc": [i, i, i, i32, vp, vp, i32, vp, vp],
        "gemm_f32_ex": [i, i, i, f, vp, vp, f, vp, cfgp, vp],
        "gemm_bf16_ex": [i, i, i, f, vp, vp, f, vp, cfgp, vp],
        "gemm_i8_ex": [i, i, i, i32, vp, vp, i32, vp, cfgp, vp],
        "pgemm_default_config": [i, i, i, i, cfgp],
        "pgemm_list_configs": [i, cfgp, i],
        "pgemm_kernel_attrs": [i, cfgp, ip, ip, ip, ip],
        "pgemm_get_device_status": [vp],
        "pgemm_selftest_wait_timeout": [i, vp],
        "pgemm_status_string": [i],
        "pgemm_version": [],
        "pgemm_stage_reuse_demo": [vp, i, i, vp, vp, i, i, ctypes.c_uint, vp, i, vp],
        "pgemm_schedule": [i, cfgp, i, i, i, llp, ip, llp, ip, llp],
        "pgemm_stream_k_plan": [ll, i, i, i, llp, ip, ip, llp],
        "pgemm_trim_scratch": [],
        "linear_bf16": [i, i, i, vp, vp, vp, i, vp, vp, vp, vp],
        "linear_bf16_backward": [i, i, i, vp, vp, vp, i, vp, vp, vp, vp, vp, vp],
        "gated_bf16": [i, i, i, vp, vp, vp, i, vp, vp, vp],
        "gated_bf16_backward": [i, i, i, vp, vp, vp, i, vp, vp, vp, vp, vp, vp],
        "xent_bf16": [i, i, i, vp, vp, vp, vp, vp, vp],
        "xent_bf16_grad": [i, i, i, vp, vp, vp, vp, vp, vp, vp, vp, ll, vp],
        "rmsnorm_bf16": [i, i, vp, vp, vp, f, vp, vp, vp],
        "rmsnorm_i8": [i, i, vp, vp, vp, f, vp, vp, vp, vp],
        "rmsnorm_bf16_backward": [i, i, vp, vp, f, vp, vp, vp, vp, vp],
        "route_topk": [i, i, i, vp, i, vp, vp, vp],
        "route_topk_backward": [i, i, i, vp, i, vp, vp, vp, vp],
        "expert_sort": [i, i, i, vp, vp, vp, vp],
        "expert_gather_bf16": [i, i, i, vp, vp, vp, vp],
        "expert_combine_bf16": [i, i, i, vp, vp, vp, vp, vp, vp],
        "expert_combine_bf16_backward": [i, i, i, vp, vp, vp, vp, vp, vp, vp],
        "experts_linear_bf16": [i, i, i, i, vp, vp, vp, vp, vp],
        "experts_linear_bf16_backward": [i, i, i, i, vp, vp, vp, vp, vp, vp, vp],
        "experts_gated_bf16": [i, i, i, i, vp, vp, vp, vp, i, vp, vp, vp],
        "experts_gated_bf16_backward": [i, i, i, i, vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp],
    }
    for name, args in sig.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    L.pgemm_status_string.restype = ctypes.c_char_p
    return L


def lib() -> ctypes.CDLL:
    """The loaded library.  Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(library_path):
                raise RuntimeError(
                    f"{library_path} is missing: build it with "
                    "`python -m software_pipelined_tiled_loop_gb300.build` (needs nvcc)")
            _lib = _declare(ctypes.CDLL(library_path))
        return _lib


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if not x.is_cuda:
            raise ValueError("operands must be CUDA tensors (or raw device pointers)")
        if not x.is_contiguous():
            raise ValueError("operands must be contiguous row-major tensors")
        return int(x.data_ptr())
    raise TypeError(f"cannot take a device pointer from {type(x).__name__}")


_current_raw_stream = None  # torch's current stream of the current device, once CUDA is up


def _stream(s) -> int:
    if s is None:
        if _current_raw_stream is not None:
            return _current_raw_stream()
        return _find_current_stream()
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _find_current_stream() -> int:
    """torch's current stream (0 without torch or a GPU).  The first call that
    finds torch's CUDA state initialised keeps the direct lookup, which takes
    0.3 us a call instead of 3.8 through a Stream object."""
    global _current_raw_stream
    try:
        import torch
        if not torch.cuda.is_available():
            return 0
    except ImportError:
        return 0
    found = int(torch.cuda.current_stream().cuda_stream)
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    if torch.cuda.is_initialized() and raw is not None and device is not None:
        _current_raw_stream = lambda: raw(device())  # noqa: E731
    return found


def _check(code: int, where: str) -> None:
    if code != 0:
        raise PgemmError(code, where)


def _cfg(config):
    if config is None:
        return None
    if isinstance(config, Config):
        return ctypes.byref(config)
    return ctypes.byref(Config(*config))


def gemm_f32(M, N, K, alpha, A, B, beta, C, stream=None):
    """C <- alpha*A@B + beta*C, fp32 (FFMA).  Asynchronous on ``stream``."""
    _check(lib().gemm_f32(M, N, K, alpha, _ptr(A), _ptr(B), beta, _ptr(C), _stream(stream)),
           "gemm_f32")


def gemm_bf16(M, N, K, alpha, A, B, beta, C, stream=None):
    """C (fp32) <- alpha*A@B + beta*C with bf16 A, B (tcgen05).  Asynchronous."""
    _check(lib().gemm_bf16(M, N, K, alpha, _ptr(A), _ptr(B), beta, _ptr(C), _stream(stream)),
           "gemm_bf16")


def gemm_i8(M, N, K, alpha, A, B, beta, C, stream=None):
    """C (int32) <- alpha*A@B + beta*C with int8 A, B, exact modulo 2^32.  Asynchronous."""
    _check(lib().gemm_i8(M, N, K, int(alpha), _ptr(A), _ptr(B), int(beta), _ptr(C),
                         _stream(stream)), "gemm_i8")


def gemm_i8_noalloc(M, N, K, alpha, A, B, beta, C, stream=None):
    """gemm_i8 that allocates no device memory: for callers whose memory is
    owned by their own allocator or budget, or who may not call an allocator
    on this path.  Operands are widened into one fixed 32 MiB device array
    shared by all calls (calls overlapping on the GPU race); larger problems
    raise PgemmError(PGEMM_ERR_TOO_LARGE).  The first call on a device looks
    up that array's address and should come before any stream capture."""
    _check(lib().gemm_i8_noalloc(M, N, K, int(alpha), _ptr(A), _ptr(B), int(beta), _ptr(C),
                                 _stream(stream)), "gemm_i8_noalloc")


def gemm_f32_ex(M, N, K, alpha, A, B, beta, C, config=None, stream=None):
    _check(lib().gemm_f32_ex(M, N, K, alpha, _ptr(A), _ptr(B), beta, _ptr(C), _cfg(config),
                             _stream(stream)), "gemm_f32_ex")


def gemm_bf16_ex(M, N, K, alpha, A, B, beta, C, config=None, stream=None):
    _check(lib().gemm_bf16_ex(M, N, K, alpha, _ptr(A), _ptr(B), beta, _ptr(C), _cfg(config),
                              _stream(stream)), "gemm_bf16_ex")


def gemm_i8_ex(M, N, K, alpha, A, B, beta, C, config=None, stream=None):
    _check(lib().gemm_i8_ex(M, N, K, int(alpha), _ptr(A), _ptr(B), int(beta), _ptr(C),
                            _cfg(config), _stream(stream)), "gemm_i8_ex")


class _Kind:
    """An operand's element type: its size and the torch types that hold it."""

    def __init__(self, itemsize, *names):
        self.itemsize, self.names = itemsize, names
        self.seen = set()  # torch's own objects for them, once met


# (bf16 bit patterns also travel as 16-bit integers, as gemm_bf16 takes them)
_BF16 = _Kind(2, "torch.bfloat16", "torch.int16", "torch.uint16")
_F32 = _Kind(4, "torch.float32")
_I64 = _Kind(8, "torch.int64")
_I32 = _Kind(4, "torch.int32")
_I8 = _Kind(1, "torch.int8")


def _operand(x, name, count, kind) -> int:
    """_ptr of an operator's operand, which must hold at least ``count``
    elements of ``kind`` (checked for tensors; None and addresses pass)."""
    try:
        if (x.is_cuda and x.dtype in kind.seen and x.numel() >= count and x.is_contiguous()):
            return x.data_ptr()
    except AttributeError:
        pass  # None, a raw pointer, or nothing that has an address
    p = _ptr(x)
    if not hasattr(x, "element_size"):
        return p
    if x.element_size() != kind.itemsize:
        raise ValueError(f"{name}: elements of {x.element_size()} bytes, {kind.itemsize} wanted")
    dtype = getattr(x, "dtype", None)
    if dtype is not None and str(dtype) not in kind.names:
        raise ValueError(f"{name}: elements of type {dtype}, {kind.names[0]} wanted")
    if x.numel() < count:
        raise ValueError(f"{name}: {x.numel()} elements, at least {count} wanted")
    if dtype is not None:
        kind.seen.add(dtype)
    return p


_DIM_MAX = 2 ** 31 - 1  # the C interface's sizes are 32-bit


def _sizes(what, bits):
    """Refuse sizes, given as their bitwise or, of which ctypes would pass only the
    low 32 bits.  (Negative 32-bit sizes are left to the C function, which refuses
    them; what their or may hide has negative low bits itself or stands beside them.)"""
    if not -_DIM_MAX <= bits + 1 <= _DIM_MAX + 1:
        raise ValueError(f"{what}: sizes are at most {_DIM_MAX}")


def _act(act) -> int:
    if isinstance(act, str):
        if act not in ACTIVATIONS:
            raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
        return ACTIVATIONS[act]
    return int(act)


def linear_bf16(M, N, K, X, W, bias, act, residual, Y, preact=None, stream=None):
    """Y <- act(X @ W + bias) + residual, bf16 with fp32 arithmetic.  X: M x K,
    W: K x N; bias (N) and residual (M x N, may be Y) may be None; ``act`` is a
    name of ACTIVATIONS.  ``preact`` (M x N fp32) receives X @ W + bias for the
    backward call.  Asynchronous on ``stream``."""
    _sizes("linear_bf16", M | N | K)
    _check(lib().linear_bf16(
        M, N, K, _operand(X, "X", M * K, _BF16), _operand(W, "W", K * N, _BF16),
        _operand(bias, "bias", N, _BF16), _act(act), _operand(residual, "residual", M * N, _BF16),
        _operand(Y, "Y", M * N, _BF16), _operand(preact, "preact", M * N, _F32),
        _stream(stream)), "linear_bf16")


def linear_bf16_backward(M, N, K, X, W, bias, act, dY, dX, dW, dbias, preact=None, stream=None):
    """Gradients of linear_bf16 for dY (M x N) into dX (M x K), dW (K x N) and
    dbias (N), each skipped when None; X and W may be None where nothing wanted
    reads them.  ``preact``: what the forward call kept, or None to compute it
    again.  Asynchronous."""
    _sizes("linear_bf16_backward", M | N | K)
    _check(lib().linear_bf16_backward(
        M, N, K, _operand(X, "X", M * K, _BF16), _operand(W, "W", K * N, _BF16),
        _operand(bias, "bias", N, _BF16), _act(act), _operand(dY, "dY", M * N, _BF16),
        _operand(preact, "preact", M * N, _F32), _operand(dX, "dX", M * K, _BF16),
        _operand(dW, "dW", K * N, _BF16), _operand(dbias, "dbias", N, _BF16), _stream(stream)),
        "linear_bf16_backward")


def gated_bf16(M, F, K, X, Wg, Wu, act, H, preact=None, stream=None):
    """H <- act(X @ Wg) * (X @ Wu), bf16 with fp32 arithmetic.  X: M x K, Wg and
    Wu: K x F, H: M x F.  ``preact`` (2 x M x F fp32) receives both products
    for the backward call.  Asynchronous on ``stream``."""
    _sizes("gated_bf16", M | F | K)
    _check(lib().gated_bf16(
        M, F, K, _operand(X, "X", M * K, _BF16), _operand(Wg, "Wg", K * F, _BF16),
        _operand(Wu, "Wu", K * F, _BF16), _act(act), _operand(H, "H", M * F, _BF16),
        _operand(preact, "preact", 2 * M * F, _F32), _stream(stream)), "gated_bf16")


def gated_bf16_backward(M, F, K, X, Wg, Wu, act, dH, dX, dWg, dWu, preact=None, stream=None):
    """Gradients of gated_bf16 for dH (M x F) into dX (M x K), dWg and dWu
    (K x F); dX, or dWg and dWu together, may be None, and so may X, Wg and Wu
    where nothing wanted reads them.  ``preact``: what the forward call kept, or
    None to compute it again.  Asynchronous."""
    _sizes("gated_bf16_backward", M | F | K)
    _check(lib().gated_bf16_backward(
        M, F, K, _operand(X, "X", M * K, _BF16), _operand(Wg, "Wg", K * F, _BF16),
        _operand(Wu, "Wu", K * F, _BF16), _act(act), _operand(dH, "dH", M * F, _BF16),
        _operand(preact, "preact", 2 * M * F, _F32), _operand(dX, "dX", M * K, _BF16),
        _operand(dWg, "dWg", K * F, _BF16), _operand(dWu, "dWu", K * F, _BF16), _stream(stream)),
        "gated_bf16_backward")


def xent_bf16(T, V, D, X, W, target, loss, lse, stream=None):
    """Softmax cross entropy of logits X @ W.T over a vocabulary: X: T x D, W:
    V x D bf16, target: T int64 (outside [0, V): the row does not count, loss
    0); loss and lse: T fp32, either may be None.  Asynchronous."""
    _sizes("xent_bf16", T | V | D)
    _check(lib().xent_bf16(
        T, V, D, _operand(X, "X", T * D, _BF16), _operand(W, "W", V * D, _BF16),
        _operand(target, "target", T, _I64), _operand(loss, "loss", T, _F32),
        _operand(lse, "lse", T, _F32), _stream(stream)), "xent_bf16")


def xent_bf16_grad(T, V, D, X, W, target, dloss, loss, lse, dX, dW, workspace_bytes=0,
                   stream=None):
    """xent_bf16 with its gradients for dloss (T fp32; None: ones) into dX
    (T x D) and dW (V x D), either of which may be None.  ``workspace_bytes``
    bounds the scratch for the probabilities (0: the library's choice); larger
    ones go by in pieces of the vocabulary.  Asynchronous."""
    _sizes("xent_bf16_grad", T | V | D)
    _check(lib().xent_bf16_grad(
        T, V, D, _operand(X, "X", T * D, _BF16), _operand(W, "W", V * D, _BF16),
        _operand(target, "target", T, _I64), _operand(dloss, "dloss", T, _F32),
        _operand(loss, "loss", T, _F32), _operand(lse, "lse", T, _F32),
        _operand(dX, "dX", T * D, _BF16), _operand(dW, "dW", V * D, _BF16), int(workspace_bytes),
        _stream(stream)), "xent_bf16_grad")


def rmsnorm_bf16(T, D, X, residual, gain, eps, S, Y, stream=None):
    """S <- X + residual (bf16) and Y <- S * gain / sqrt(mean(S^2) + eps), row by row.
    X, residual, S and Y: T x D; gain: D.  residual, gain (ones) and S (not kept; may be
    X or residual) may be None.  Asynchronous on ``stream``."""
    _sizes("rmsnorm_bf16", T | D)
    _check(lib().rmsnorm_bf16(
        T, D, _operand(X, "X", T * D, _BF16), _operand(residual, "residual", T * D, _BF16),
        _operand(gain, "gain", D, _BF16), eps, _operand(S, "S", T * D, _BF16),
        _operand(Y, "Y", T * D, _BF16), _stream(stream)), "rmsnorm_bf16")


def rmsnorm_i8(T, D, X, residual, gain, eps, S, Q, scale, stream=None):
    """rmsnorm_bf16 with the result as int8 (Q: T x D) and a scale a row (T fp32):
    Q * scale is the result to within half a scale.  Asynchronous."""
    _sizes("rmsnorm_i8", T | D)
    _check(lib().rmsnorm_i8(
        T, D, _operand(X, "X", T * D, _BF16), _operand(residual, "residual", T * D, _BF16),
        _operand(gain, "gain", D, _BF16), eps, _operand(S, "S", T * D, _BF16),
        _operand(Q, "Q", T * D, _I8), _operand(scale, "scale", T, _F32), _stream(stream)),
        "rmsnorm_i8")


def rmsnorm_bf16_backward(T, D, S, gain, eps, dY, dS, dX, dgain, stream=None):
    """Gradients of rmsnorm_bf16 for dY (T x D) and, where S flows on, dS (or None) into
    dX (the gradient of X and of the residual; may be dS) and dgain (D), either of which
    may be None.  Asynchronous."""
    _sizes("rmsnorm_bf16_backward", T | D)
    _check(lib().rmsnorm_bf16_backward(
        T, D, _operand(S, "S", T * D, _BF16), _operand(gain, "gain", D, _BF16), eps,
        _operand(dY, "dY", T * D, _BF16), _operand(dS, "dS", T * D, _BF16),
        _operand(dX, "dX", T * D, _BF16), _operand(dgain, "dgain", D, _BF16), _stream(stream)),
        "rmsnorm_bf16_backward")


def route_topk(T, E, k, logits, normalise, experts, weights, stream=None):
    """The k largest of each token's E logits (T x E fp32) into experts (T x k int32, ties
    to the lowest index, -1 where fewer are above -inf) and their softmax over the chosen
    (``normalise``) or over all E into weights (T x k fp32).  Asynchronous."""
    _sizes("route_topk", T | E | k)
    _check(lib().route_topk(
        T, E, k, _operand(logits, "logits", T * E, _F32), int(bool(normalise)),
        _operand(experts, "experts", T * k, _I32), _operand(weights, "weights", T * k, _F32),
        _stream(stream)), "route_topk")


def route_topk_backward(T, E, k, logits, normalise, experts, dweights, dlogits, stream=None):
    """Gradient of route_topk's weights for dweights (T x k) into dlogits (T x E); experts
    as it left them.  Asynchronous."""
    _sizes("route_topk_backward", T | E | k)
    _check(lib().route_topk_backward(
        T, E, k, _operand(logits, "logits", T * E, _F32), int(bool(normalise)),
        _operand(experts, "experts", T * k, _I32), _operand(dweights, "dweights", T * k, _F32),
        _operand(dlogits, "dlogits", T * E, _F32), _stream(stream)), "route_topk_backward")


def expert_sort(T, E, k, experts, offsets, slot_row, stream=None):
    """Sort the slots of experts (T x k int32) by expert, stably: offsets (E + 1 int32)
    receives each expert's first row and the number of rows, slot_row (T x k int32) each
    slot's row (-1: an expert outside [0, E)).  Asynchronous."""
    _sizes("expert_sort", T | E | k)
    _check(lib().expert_sort(
        T, E, k, _operand(experts, "experts", T * k, _I32),
        _operand(offsets, "offsets", E + 1, _I32), _operand(slot_row, "slot_row", T * k, _I32),
        _stream(stream)), "expert_sort")


def expert_gather_bf16(T, k, D, X, slot_row, Xs, stream=None):
    """Xs[slot_row[t, j]] <- X[t].  X: T x D, Xs: T k x D (rows no slot has stay as they
    were).  The gradient is expert_combine_bf16 without weights and residual.
    Asynchronous."""
    _sizes("expert_gather_bf16", T | k | D)
    _check(lib().expert_gather_bf16(
        T, k, D, _operand(X, "X", T * D, _BF16), _operand(slot_row, "slot_row", T * k, _I32),
        _operand(Xs, "Xs", T * k * D, _BF16), _stream(stream)), "expert_gather_bf16")


def expert_combine_bf16(T, k, D, Ys, slot_row, weights, residual, Y, stream=None):
    """Y[t] <- residual[t] + sum over j of weights[t, j] * Ys[slot_row[t, j]].  Ys: T k x
    D, weights: T x k fp32 or None (ones), residual: T x D or None (may be Y).
    Asynchronous."""
    _sizes("expert_combine_bf16", T | k | D)
    _check(lib().expert_combine_bf16(
        T, k, D, _operand(Ys, "Ys", T * k * D, _BF16),
        _operand(slot_row, "slot_row", T * k, _I32), _operand(weights, "weights", T * k, _F32),
        _operand(residual, "residual", T * D, _BF16), _operand(Y, "Y", T * D, _BF16),
        _stream(stream)), "expert_combine_bf16")


def expert_combine_bf16_backward(T, k, D, Ys, slot_row, weights, dY, dYs, dweights, stream=None):
    """Gradients of expert_combine_bf16 for dY (T x D) into dYs (T k x D; rows no slot has
    stay as they were) and dweights (T x k fp32), either of which may be None; Ys may be
    None without dweights.  Asynchronous."""
    _sizes("expert_combine_bf16_backward", T | k | D)
    _check(lib().expert_combine_bf16_backward(
        T, k, D, _operand(Ys, "Ys", T * k * D, _BF16),
        _operand(slot_row, "slot_row", T * k, _I32), _operand(weights, "weights", T * k, _F32),
        _operand(dY, "dY", T * D, _BF16), _operand(dYs, "dYs", T * k * D, _BF16),
        _operand(dweights, "dweights", T * k, _F32), _stream(stream)),
        "expert_combine_bf16_backward")


def experts_linear_bf16(R, N, K, E, offsets, X, W, Y, stream=None):
    """Y[r] <- X[r] @ W[e] for the rows offsets[e] <= r < offsets[e + 1] of expert e.  X: R
    x K, W: E x K x N, Y: R x N (rows from offsets[E] on stay as they were), offsets: E + 1
    int32, as expert_sort leaves them.  A sum over columns (K; a dX's N, or 2 F) has 2^19
    of them at most.  Asynchronous, without a host synchronisation."""
    _sizes("experts_linear_bf16", R | N | K | E)
    _check(lib().experts_linear_bf16(
        R, N, K, E, _operand(offsets, "offsets", E + 1, _I32), _operand(X, "X", R * K, _BF16),
        _operand(W, "W", E * K * N, _BF16), _operand(Y, "Y", R * N, _BF16), _stream(stream)),
        "experts_linear_bf16")


def experts_linear_bf16_backward(R, N, K, E, offsets, X, W, dY, dX, dW, stream=None):
    """Gradients of experts_linear_bf16 for dY (R x N) into dX (R x K; rows from offsets[E]
    on stay as they were) and dW (E x K x N), either of which may be None, and so may X
    without dW and W without dX.  Asynchronous."""
    _sizes("experts_linear_bf16_backward", R | N | K | E)
    _check(lib().experts_linear_bf16_backward(
        R, N, K, E, _operand(offsets, "offsets", E + 1, _I32), _operand(X, "X", R * K, _BF16),
        _operand(W, "W", E * K * N, _BF16), _operand(dY, "dY", R * N, _BF16),
        _operand(dX, "dX", R * K, _BF16), _operand(dW, "dW", E * K * N, _BF16), _stream(stream)),
        "experts_linear_bf16_backward")


def experts_gated_bf16(R, F, K, E, offsets, X, Wg, Wu, act, H, preact=None, stream=None):
    """H[r] <- act(X[r] @ Wg[e]) * (X[r] @ Wu[e]) for the rows of each expert, as
    experts_linear_bf16.  Wg and Wu: E x K x F, H: R x F; ``act``: a name of ACTIVATIONS but
    relu.  ``preact`` (2 x R x F fp32) receives both products for the backward call.
    Asynchronous."""
    _sizes("experts_gated_bf16", R | F | K | E)
    _check(lib().experts_gated_bf16(
        R, F, K, E, _operand(offsets, "offsets", E + 1, _I32), _operand(X, "X", R * K, _BF16),
        _operand(Wg, "Wg", E * K * F, _BF16), _operand(Wu, "Wu", E * K * F, _BF16), _act(act),
        _operand(H, "H", R * F, _BF16), _operand(preact, "preact", 2 * R * F, _F32),
        _stream(stream)), "experts_gated_bf16")


def experts_gated_bf16_backward(R, F, K, E, offsets, X, Wg, Wu, act, dH, dX, dWg, dWu,
                                preact=None, stream=None):
    """Gradients of experts_gated_bf16 for dH (R x F) into dX (R x K), dWg and dWu (E x K x
    F); dX, or dWg and dWu together, may be None, and so may X, Wg and Wu where nothing
    wanted reads them.  ``preact``: what the forward call kept, or None to compute it
    again.  Asynchronous."""
    _sizes("experts_gated_bf16_backward", R | F | K | E)
    _check(lib().experts_gated_bf16_backward(
        R, F, K, E, _operand(offsets, "offsets", E + 1, _I32), _operand(X, "X", R * K, _BF16),
        _operand(Wg, "Wg", E * K * F, _BF16), _operand(Wu, "Wu", E * K * F, _BF16), _act(act),
        _operand(dH, "dH", R * F, _BF16), _operand(preact, "preact", 2 * R * F, _F32),
        _operand(dX, "dX", R * K, _BF16), _operand(dWg, "dWg", E * K * F, _BF16),
        _operand(dWu, "dWu", E * K * F, _BF16), _stream(stream)), "experts_gated_bf16_backward")


def pgemm_stage_reuse_demo(X, rows, cols, perm, out, check_reuse, delay_warp=-1, delay_ns=0,
                           trace=None, trace_cap=0, stream=None):
    """The two-stage copy-and-reduce hazard experiment (with or without the
    consume-before-reuse wait).  X: rows x cols fp32, perm: int32 row order,
    out: rows fp32 (zeroed by the caller); trace: optional uint64 buffer."""
    _check(lib().pgemm_stage_reuse_demo(_ptr(X), rows, cols, _ptr(perm), _ptr(out),
                                        int(check_reuse), int(delay_warp), int(delay_ns),
                                        _ptr(trace), int(trace_cap), _stream(stream)),
           "pgemm_stage_reuse_demo")


def pgemm_schedule(dtype: str, M: int, N: int, K: int, config=None):
    """The persistent schedule of a call on the current device: a dict with
    tiles, slots (units running at once), split_tiles and parts (split along
    K), and half_tiles (tiles run as two half-width units)."""
    t, sl, st, p = ctypes.c_longlong(), ctypes.c_int(), ctypes.c_longlong(), ctypes.c_int()
    ht = ctypes.c_longlong()
    _check(lib().pgemm_schedule(DTYPES[dtype], _cfg(config), M, N, K, ctypes.byref(t),
                                ctypes.byref(sl), ctypes.byref(st), ctypes.byref(p),
                                ctypes.byref(ht)),
           "pgemm_schedule")
    return {"tiles": t.value, "slots": sl.value, "split_tiles": st.value, "parts": p.value,
            "half_tiles": ht.value}


def pgemm_stream_k_plan(tiles: int, slots: int, k_tiles: int, max_parts: int = 0):
    """The stream-K rule (host only): a dict with sk_tiles, sk_slots,
    max_pieces and share (K-iterations per slot)."""
    st, gs, mp, sh = ctypes.c_longlong(), ctypes.c_int(), ctypes.c_int(), ctypes.c_longlong()
    _check(lib().pgemm_stream_k_plan(tiles, slots, k_tiles, max_parts, ctypes.byref(st),
                                     ctypes.byref(gs), ctypes.byref(mp), ctypes.byref(sh)),
           "pgemm_stream_k_plan")
    return {"sk_tiles": st.value, "sk_slots": gs.value, "max_pieces": mp.value,
            "share": sh.value}


def pgemm_default_config(dtype: str, M: int, N: int, K: int):
    c = Config()
    _check(lib().pgemm_default_config(DTYPES[dtype], M, N, K, ctypes.byref(c)),
           "pgemm_default_config")
    return c.as_tuple()


def pgemm_list_configs(dtype: str):
    n = lib().pgemm_list_configs(DTYPES[dtype], None, 0)
    arr = (Config * max(n, 1))()
    lib().pgemm_list_configs(DTYPES[dtype], arr, n)
    return [arr[i].as_tuple() for i in range(n)]


def pgemm_kernel_attrs(dtype: str, config):
    out = [ctypes.c_int(0) for _ in range(4)]
    _check(lib().pgemm_kernel_attrs(DTYPES[dtype], _cfg(config), *[ctypes.byref(o) for o in out]),
           "pgemm_kernel_attrs")
    return {"smem_bytes": out[0].value, "regs_per_thread": out[1].value,
            "threads_per_block": out[2].value, "blocks_per_sm": out[3].value}


def pgemm_get_device_status(stream=None) -> int:
    """Synchronise ``stream`` and return (and clear) the device status code."""
    return int(lib().pgemm_get_device_status(_stream(stream)))


def pgemm_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    return int(lib().pgemm_selftest_wait_timeout(int(limit_us), _stream(stream)))


def pgemm_status_string(code: int) -> str:
    return lib().pgemm_status_string(int(code)).decode()


def pgemm_version() -> int:
    return int(lib().pgemm_version())


def pgemm_trim_scratch() -> None:
    """Synchronise the current device and give the library's unused scratch
    memory back (the pool otherwise keeps it between calls)."""
    _check(lib().pgemm_trim_scratch(), "pgemm_trim_scratch")
