"""MX-FP8 and MX-FP4 casts of bf16 matrices, and operators that work on their outputs,
on sm_103a (GB300): Python binding.

Thin ctypes layer over the C ABI of ``libmxfp8_cast.so`` (declared in
``include/mxfp8_cast.h``).  Functions named like the C entry points take torch
tensors, check their shapes and that they share one CUDA device, make that
device current for the call, and pass raw device pointers plus its current
CUDA stream; every step of the cast runs in the library's CUDA kernels.  There
is no CPU fallback: if the library has not been built, importing the binding
raises.

Convenience wrappers (``cast_dim0_dim1``, ``cast_dim0``, ``cast_dim1``,
``cast_grouped_m``, ``cast_3d_dim1``, ``cast_3d_dim0``, ``cast_3d_dim0_dim1``,
``scales_to_blocked``, ``dequant_blocked``, ``cast_tensorwise``,
``cast_rowwise``, ``cast_fp4_dim0``, ``cast_fp4_dim1``, ``cast_fp4_dim0_dim1``,
``dequant_fp4``, ``matmul``, ``matmul_fp4``, ``matmul_swiglu``,
``matmul_swiglu_backward``, ``layer_norm``, ``layer_norm_backward``, ``swiglu``,
``swiglu_backward``) allocate outputs with torch and call the same entry points; the 2D
MX casts and all from ``dequant_fp4`` on in compiled code (``_torch_call.*.so``), which
hands every call it does not take as it stands to the checked functions here; without it
these take all calls.  ``feed_forward``
is a block of a network trained with them.

No function here takes part in autograd: results carry no graph, whatever their
inputs require.  ``feed_forward`` shows the ``autograd.Function`` that joins the
forward and backward operators.
"""
import ctypes
import functools
import importlib.util
import os
import sys
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxfp8_cast.so")
# The compiled wrappers use torch's classes as they lie in memory: each torch has its
# own file, and one of another torch is not found.
CALL_PATH = os.path.join(_PKG, "_torch_call.%s.torch-%s.so"
                         % (sys.implementation.cache_tag, torch.__version__.replace("+", "-")))

MX_OK = 0
MX_ERR_NULL = -1
MX_ERR_SHAPE = -2
MX_ERR_ALIGN = -3
MX_ERR_CUDA = -4
MX_ERR_GROUPS = -5
MX_ERR_DEVICE = -6
MX_ERR_TYPE = -7

# Every function the header declares, for load checks.
ABI_SYMBOLS = (
    "mx_cast_dim0_dim1", "mx_cast_dim0", "mx_cast_dim1", "mx_scales_to_blocked",
    "mx_cast_grouped_m", "mx_cast_3d_dim1", "mx_cast_3d_dim0", "mx_cast_3d_dim0_dim1",
    "mx_dequant_blocked", "mx_blocked_bytes", "mx_grouped_m_scale_bytes", "mx_3d_scale_bytes",
    "mx_3d_dim0_scale_bytes", "mx_cast_tensorwise", "mx_cast_rowwise", "mx_bounds_check",
    "mx_selftest_bounds",
    "mx_strerror", "mx_last_cuda_error", "mx_watchdog",
    "mx_selftest_watchdog", "mx_selftest_arm_stall", "mx_cast_dim0_dim1_noalloc",
    "mx_matmul", "mx_layer_norm", "mx_layer_norm_backward", "mx_layer_norm_backward_work_bytes",
    "mx_swiglu", "mx_swiglu_backward", "mx_cast_fp4_dim0", "mx_cast_fp4_dim1",
    "mx_cast_fp4_dim0_dim1", "mx_dequant_fp4", "mx_matmul_fp4", "mx_matmul_swiglu",
    "mx_matmul_swiglu_backward",
)


class MXError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        msg = "%s failed: %s (%d)" % (where, _lib().mx_strerror(code).decode(), code)
        if code == MX_ERR_CUDA:
            msg += " [cudaError %d]" % _lib().mx_last_cuda_error()
        super().__init__(msg)


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(
                "libmxfp8_cast.so is not built (expected at %s); build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` or "
                "`python -m mxfp8_block_scaled_dim0_gb300.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
        sig = {
            "mx_cast_dim0_dim1": ([P, I64, I64, P, P, P, P, P], ctypes.c_int),
            "mx_cast_dim0": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_dim1": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_scales_to_blocked": ([P, I64, I64, P, P], ctypes.c_int),
            "mx_cast_grouped_m": ([P, I64, I64, P, I32, P, P, P, P, P, P, P, P], ctypes.c_int),
            "mx_cast_3d_dim1": ([P, I64, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_3d_dim0": ([P, I64, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_3d_dim0_dim1": ([P, I64, I64, I64, P, P, P, P, P], ctypes.c_int),
            "mx_dequant_blocked": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_tensorwise": ([P, I64, P, P, P, P], ctypes.c_int),
            "mx_cast_rowwise": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_matmul": ([P, P, P, P, I64, I64, I64, I32, P, I32, P], ctypes.c_int),
            "mx_layer_norm": ([P, P, P, I32, I64, I64, ctypes.c_float, P, P, P, P, P, P],
                              ctypes.c_int),
            "mx_layer_norm_backward": ([P, P, P, P, P, I32, P, P, I64, I64, P, P, P, P, P],
                                       ctypes.c_int),
            "mx_layer_norm_backward_work_bytes": ([I64, I64], I64),
            "mx_swiglu": ([P, I64, I64, P, P, P, P], ctypes.c_int),
            "mx_swiglu_backward": ([P, P, P, P, I64, I64, P, P], ctypes.c_int),
            "mx_cast_fp4_dim0": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_fp4_dim1": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_cast_fp4_dim0_dim1": ([P, I64, I64, P, P, P, P, P], ctypes.c_int),
            "mx_dequant_fp4": ([P, I64, I64, P, P, P], ctypes.c_int),
            "mx_matmul_fp4": ([P, P, P, P, I64, I64, I64, P, I32, P], ctypes.c_int),
            "mx_matmul_swiglu": ([P, P, P, P, P, P, I64, I64, I64, I32, P, P, P, P], ctypes.c_int),
            "mx_matmul_swiglu_backward": ([P, P, P, P, I64, I64, I64, I32, P, P, P, P, P],
                                          ctypes.c_int),
            "mx_blocked_bytes": ([I64, I64], I64),
            "mx_grouped_m_scale_bytes": ([I64, I64, I32, I32], I64),
            "mx_3d_scale_bytes": ([I64, I64, I64], I64),
            "mx_3d_dim0_scale_bytes": ([I64, I64, I64], I64),
            "mx_strerror": ([ctypes.c_int], ctypes.c_char_p),
            "mx_last_cuda_error": ([], ctypes.c_int),
            "mx_watchdog": ([ctypes.c_int], ctypes.c_int),
            "mx_bounds_check": ([ctypes.c_int], ctypes.c_int),
            "mx_selftest_bounds": ([P, P], ctypes.c_int),
            "mx_selftest_watchdog": ([I64, P], ctypes.c_int),
            "mx_selftest_arm_stall": ([I64, I64], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        # Addresses that the compiled wrappers call.
        lib.addresses = {name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
                         for name in sig}
        _load_call()
        _LIB = lib               # last: another thread that sees it finds the wrappers too
    return _LIB


# The compiled wrappers (csrc/torch_call.cpp); None: not built.
_CALL = None


def _load_call():
    """Without the compiled wrappers the checked functions serve every call, some
    10 us of host time slower."""
    global _CALL
    if _CALL is not None:
        return
    try:
        spec = importlib.util.spec_from_file_location("_torch_call", CALL_PATH)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
    except (ImportError, OSError) as e:
        warnings.warn("the compiled wrappers (%s) do not load, calls go through Python: %s; build them "
                      "with `python -m mxfp8_block_scaled_dim0_gb300.build`" % (CALL_PATH, e),
                      RuntimeWarning, stacklevel=3)
        return
    _CALL = module


def library():
    """The loaded ctypes library (raises ImportError if it is not built)."""
    return _lib()


# ---- marshalling helpers ----------------------------------------------------

def _ptr(t):
    # ctypes converts a plain int (or None) for a c_void_p parameter.
    return t.data_ptr() if t is not None else None


# cudaStream_t (as an int) of a device's current stream; cheaper than
# building a torch.cuda.Stream object per call.  Builds of torch without the
# raw accessor take the public route.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _stream(stream, dev=None):
    """The call's cudaStream_t: `stream` (a torch.cuda.Stream or a raw
    handle), else the current stream of device index `dev` (default: the
    current device)."""
    if stream is None:
        return _raw_stream(torch.cuda.current_device() if dev is None else dev)
    if isinstance(stream, torch.cuda.Stream):
        if dev is not None and stream.device_index != dev:
            raise ValueError("stream is on cuda:%d, the tensors on cuda:%d"
                             % (stream.device_index, dev))
        return stream.cuda_stream
    return int(stream)


def _device(*tensors):
    """Index of the one CUDA device that all the call's tensors live on."""
    devs = {t.get_device() for t in tensors if t is not None}
    if any(d < 0 for d in devs):
        raise ValueError("every tensor of a call must be a CUDA tensor, got %s"
                         % ", ".join(sorted({str(t.device) for t in tensors if t is not None})))
    if len(devs) != 1:
        raise ValueError("all tensors of a call must be on one CUDA device, got %s"
                         % ", ".join("cuda:%d" % d for d in sorted(devs)))
    return devs.pop()


def _call(name, dev, stream, *args):
    """Call entry point `name` with device index `dev` current (the library
    launches on the current device) and the stream appended: by default the
    current stream of that device."""
    fn = getattr(_LIB or _lib(), name)
    if _current_device() == dev:
        rc = fn(*args, _raw_stream(dev) if stream is None else _stream(stream, dev))
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, _stream(stream, dev))
    if rc != MX_OK:
        raise MXError(rc, name)


# dtypes each kind of argument may have.  The C ABI sees only pointers, so
# this is the one place where a float16 tensor passed as bf16 input, or float
# offsets passed as int32 group ends, can be refused.
BF16 = (torch.bfloat16,)
BYTES = tuple(d for d in (torch.uint8, getattr(torch, "float8_e4m3fn", None),
                          getattr(torch, "float8_e8m0fnu", None)) if d is not None)
# Bytes of two e2m1 values.
BYTES4 = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())
I32 = (torch.int32,)
I64 = (torch.int64,)
F32 = (torch.float32,)
# Element types of arguments that may have either, as the C ABI numbers them.
TYPES = {torch.bfloat16: 0, torch.float32: 1}
# Formats of operands, by their elements' bits, as the C ABI numbers them.
FORMATS = {8: 0, 4: 1}


def _dev_tensor(t, name, nbytes=None, dtypes=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if dtypes is not None and t.dtype not in dtypes:
        raise TypeError("%s must have dtype %s, got %s"
                        % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if ndim is not None and t.dim() != ndim:
        raise ValueError("%s must have %d dimensions, got shape %s" % (name, ndim, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if nbytes is not None and t.nbytes < nbytes:
        raise ValueError("%s holds %d bytes, needs %d" % (name, t.nbytes, nbytes))
    return t


def _check(rc, where):
    if rc != MX_OK:
        raise MXError(rc, where)


# ---- sizes ------------------------------------------------------------------

# The size helpers are pure functions of their arguments; shapes repeat from
# call to call, so their results are cached on the Python side.
@functools.lru_cache(maxsize=4096)
def mx_blocked_bytes(R, C):
    return int(_lib().mx_blocked_bytes(R, C))


@functools.lru_cache(maxsize=4096)
def mx_grouped_m_scale_bytes(M, K, G, dim):
    return int(_lib().mx_grouped_m_scale_bytes(M, K, G, dim))


@functools.lru_cache(maxsize=4096)
def mx_3d_scale_bytes(E, N, K):
    return int(_lib().mx_3d_scale_bytes(E, N, K))


@functools.lru_cache(maxsize=4096)
def mx_3d_dim0_scale_bytes(E, N, K):
    return int(_lib().mx_3d_dim0_scale_bytes(E, N, K))


@functools.lru_cache(maxsize=4096)
def mx_layer_norm_backward_work_bytes(M, D):
    return int(_lib().mx_layer_norm_backward_work_bytes(M, D))


# ---- entry points (same names as the C ABI) ----------------------------------

def mx_cast_dim0_dim1(x, q0, s0_blk, q1, s1_blk, stream=None):
    """Fused dim0 + dim1 cast of bf16 x (M x K) into caller buffers."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q0, "q0", M * K, BYTES)
    _dev_tensor(q1, "q1", M * K, BYTES)
    _dev_tensor(s0_blk, "s0_blk", mx_blocked_bytes(M, K // 32), BYTES)
    _dev_tensor(s1_blk, "s1_blk", mx_blocked_bytes(K, M // 32), BYTES)
    dev = _device(x, q0, s0_blk, q1, s1_blk)
    _call("mx_cast_dim0_dim1", dev, stream, _ptr(x), M, K, _ptr(q0), _ptr(s0_blk), _ptr(q1),
          _ptr(s1_blk))


def mx_cast_dim0(x, q0, s0_blk, stream=None):
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q0, "q0", M * K, BYTES)
    _dev_tensor(s0_blk, "s0_blk", mx_blocked_bytes(M, K // 32), BYTES)
    _call("mx_cast_dim0", _device(x, q0, s0_blk), stream, _ptr(x), M, K, _ptr(q0), _ptr(s0_blk))


def mx_cast_dim1(x, q1, s1_blk, stream=None):
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q1, "q1", M * K, BYTES)
    _dev_tensor(s1_blk, "s1_blk", mx_blocked_bytes(K, M // 32), BYTES)
    _call("mx_cast_dim1", _device(x, q1, s1_blk), stream, _ptr(x), M, K, _ptr(q1), _ptr(s1_blk))


def mx_scales_to_blocked(s, out, stream=None):
    _dev_tensor(s, "s", dtypes=BYTES, ndim=2)
    R, C = s.shape
    _dev_tensor(out, "out", mx_blocked_bytes(R, C), BYTES)
    _call("mx_scales_to_blocked", _device(s, out), stream, _ptr(s), R, C, _ptr(out))


def mx_cast_grouped_m(x, offs, q0, s0_blk, s0_row_offs, q1, s1_blk, s1_col_offs, status,
                      stream=None):
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(offs, "offs", dtypes=I32, ndim=1)
    G = offs.numel()
    _dev_tensor(q0, "q0", M * K, BYTES)
    _dev_tensor(q1, "q1", M * K, BYTES)
    if G >= 1:
        _dev_tensor(s0_blk, "s0_blk", mx_grouped_m_scale_bytes(M, K, G, 0), BYTES)
        _dev_tensor(s1_blk, "s1_blk", mx_grouped_m_scale_bytes(M, K, G, 1), BYTES)
    _dev_tensor(s0_row_offs, "s0_row_offs", 8 * (G + 1), I64)
    _dev_tensor(s1_col_offs, "s1_col_offs", 8 * (G + 1), I64)
    _dev_tensor(status, "status", 4, I32)
    dev = _device(x, offs, q0, s0_blk, s0_row_offs, q1, s1_blk, s1_col_offs, status)
    _call("mx_cast_grouped_m", dev, stream, _ptr(x), M, K, _ptr(offs), G, _ptr(q0), _ptr(s0_blk),
          _ptr(s0_row_offs), _ptr(q1), _ptr(s1_blk), _ptr(s1_col_offs), _ptr(status))


def mx_cast_3d_dim1(w, q1, s1_blk, stream=None):
    _dev_tensor(w, "w", dtypes=BF16, ndim=3)
    E, N, K = w.shape
    _dev_tensor(q1, "q1", E * N * K, BYTES)
    _dev_tensor(s1_blk, "s1_blk", mx_3d_scale_bytes(E, N, K), BYTES)
    dev = _device(w, q1, s1_blk)
    _call("mx_cast_3d_dim1", dev, stream, _ptr(w), E, N, K, _ptr(q1), _ptr(s1_blk))


def mx_cast_3d_dim0(w, q0, s0_blk, stream=None):
    _dev_tensor(w, "w", dtypes=BF16, ndim=3)
    E, N, K = w.shape
    _dev_tensor(q0, "q0", E * N * K, BYTES)
    _dev_tensor(s0_blk, "s0_blk", mx_3d_dim0_scale_bytes(E, N, K), BYTES)
    dev = _device(w, q0, s0_blk)
    _call("mx_cast_3d_dim0", dev, stream, _ptr(w), E, N, K, _ptr(q0), _ptr(s0_blk))


def mx_cast_3d_dim0_dim1(w, q0, s0_blk, q1, s1_blk, stream=None):
    _dev_tensor(w, "w", dtypes=BF16, ndim=3)
    E, N, K = w.shape
    _dev_tensor(q0, "q0", E * N * K, BYTES)
    _dev_tensor(q1, "q1", E * N * K, BYTES)
    _dev_tensor(s0_blk, "s0_blk", mx_3d_dim0_scale_bytes(E, N, K), BYTES)
    _dev_tensor(s1_blk, "s1_blk", mx_3d_scale_bytes(E, N, K), BYTES)
    dev = _device(w, q0, s0_blk, q1, s1_blk)
    _call("mx_cast_3d_dim0_dim1", dev, stream, _ptr(w), E, N, K, _ptr(q0), _ptr(s0_blk), _ptr(q1),
          _ptr(s1_blk))


def mx_dequant_blocked(q, s_blk, out, stream=None):
    """bf16 out (R x C) = e4m3 q (R x C) times 2^(scale - 127), scales in
    blocked layout."""
    _dev_tensor(q, "q", dtypes=BYTES, ndim=2)
    R, C = q.shape
    _dev_tensor(s_blk, "s_blk", mx_blocked_bytes(R, C // 32), BYTES)
    _dev_tensor(out, "out", 2 * R * C, BF16)
    dev = _device(q, s_blk, out)
    _call("mx_dequant_blocked", dev, stream, _ptr(q), R, C, _ptr(s_blk), _ptr(out))


def mx_cast_tensorwise(x, q, scale, amax, stream=None):
    """Tensorwise fp8 of bf16 x (any shape): q (x.numel() bytes), scale and
    amax (one float32 each)."""
    _dev_tensor(x, "x", dtypes=BF16)
    n = x.numel()
    _dev_tensor(q, "q", n, BYTES)
    _dev_tensor(scale, "scale", 4, F32)
    _dev_tensor(amax, "amax", 4, F32)
    dev = _device(x, q, scale, amax)
    _call("mx_cast_tensorwise", dev, stream, _ptr(x), n, _ptr(q), _ptr(scale), _ptr(amax))


def mx_cast_rowwise(x, q, scale, stream=None):
    """Rowwise fp8 of bf16 x (M x K): q (M x K bytes), scale (M bf16)."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q, "q", M * K, BYTES)
    _dev_tensor(scale, "scale", 2 * M, BF16)
    _call("mx_cast_rowwise", _device(x, q, scale), stream, _ptr(x), M, K, _ptr(q), _ptr(scale))


def _operand(q, name):
    """A 2D byte operand that is contiguous, or the transpose of a contiguous
    matrix: (tensor, whether it is the latter)."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or q.is_contiguous():
        _dev_tensor(q, name, dtypes=BYTES, ndim=2)
        return False
    by_column = q.t().is_contiguous()
    _dev_tensor(q.t() if by_column else q, name, dtypes=BYTES, ndim=2)
    return by_column


def mx_matmul(qa, sa_blk, qb, sb_blk, out, stream=None):
    """out (M x N, bf16 or float32) = A B^T of MX operands: qa (M x K) and qb
    (N x K) bytes with their blocked scales; either may be the transposed view
    of a contiguous (K x M, K x N) matrix."""
    orders = (1 if _operand(qa, "qa") else 0) | (2 if _operand(qb, "qb") else 0)
    M, K = qa.shape
    N = qb.shape[0]
    if qb.shape[1] != K:
        raise ValueError("qa and qb must have equal rows, got %d and %d values" % (K, qb.shape[1]))
    _dev_tensor(sa_blk, "sa_blk", mx_blocked_bytes(M, K // 32), BYTES)
    _dev_tensor(sb_blk, "sb_blk", mx_blocked_bytes(N, K // 32), BYTES)
    _dev_tensor(out, "out", dtypes=tuple(TYPES), ndim=2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out must have shape %s, got %s" % ((M, N), tuple(out.shape)))
    dev = _device(qa, sa_blk, qb, sb_blk, out)
    _call("mx_matmul", dev, stream, _ptr(qa), _ptr(sa_blk), _ptr(qb), _ptr(sb_blk), M, N, K, orders,
          _ptr(out), TYPES[out.dtype])


def mx_cast_fp4_dim0(x, q0, s0_blk, stream=None):
    """MX-FP4 cast of bf16 x (M x K) along its rows: q0 (M x K/2 bytes)."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q0, "q0", M * K // 2, BYTES4)
    _dev_tensor(s0_blk, "s0_blk", mx_blocked_bytes(M, K // 32), BYTES)
    _call("mx_cast_fp4_dim0", _device(x, q0, s0_blk), stream, _ptr(x), M, K, _ptr(q0), _ptr(s0_blk))


def mx_cast_fp4_dim1(x, q1, s1_blk, stream=None):
    """MX-FP4 cast of bf16 x (M x K) along its columns: q1 (K x M/2 bytes)."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q1, "q1", M * K // 2, BYTES4)
    _dev_tensor(s1_blk, "s1_blk", mx_blocked_bytes(K, M // 32), BYTES)
    _call("mx_cast_fp4_dim1", _device(x, q1, s1_blk), stream, _ptr(x), M, K, _ptr(q1), _ptr(s1_blk))


def mx_cast_fp4_dim0_dim1(x, q0, s0_blk, q1, s1_blk, stream=None):
    """Both MX-FP4 casts of bf16 x (M x K) in one read."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, K = x.shape
    _dev_tensor(q0, "q0", M * K // 2, BYTES4)
    _dev_tensor(q1, "q1", M * K // 2, BYTES4)
    _dev_tensor(s0_blk, "s0_blk", mx_blocked_bytes(M, K // 32), BYTES)
    _dev_tensor(s1_blk, "s1_blk", mx_blocked_bytes(K, M // 32), BYTES)
    dev = _device(x, q0, s0_blk, q1, s1_blk)
    _call("mx_cast_fp4_dim0_dim1", dev, stream, _ptr(x), M, K, _ptr(q0), _ptr(s0_blk), _ptr(q1),
          _ptr(s1_blk))


def mx_dequant_fp4(q, s_blk, out, stream=None):
    """bf16 out (R x C) = e2m1 q (R x C/2 bytes) times 2^(scale - 127)."""
    _dev_tensor(q, "q", dtypes=BYTES4, ndim=2)
    R, C = q.shape[0], 2 * q.shape[1]
    _dev_tensor(s_blk, "s_blk", mx_blocked_bytes(R, C // 32), BYTES)
    _shaped(out, "out", (R, C), BF16)
    _call("mx_dequant_fp4", _device(q, s_blk, out), stream, _ptr(q), R, C, _ptr(s_blk), _ptr(out))


def _by_row(q, s_blk, name, bits):
    """Checks an MX operand of `bits` stored by row; its (rows, steps)."""
    if bits not in FORMATS:
        raise ValueError("bits must be 8 or 4, got %r" % (bits,))
    _dev_tensor(q, "q" + name, dtypes=BYTES if bits == 8 else BYTES4, ndim=2)
    R, K = q.shape[0], q.shape[1] * (8 // bits)
    _dev_tensor(s_blk, "s%s_blk" % name, mx_blocked_bytes(R, K // 32), BYTES)
    return R, K


def _same_steps(name_a, Ka, name_b, Kb):
    if Ka != Kb:
        raise ValueError("q%s and q%s must have equal rows, got %d and %d values"
                         % (name_a, name_b, Ka, Kb))


def mx_matmul_fp4(qa, sa_blk, qb, sb_blk, out, stream=None):
    """out (M x N, bf16 or float32) = A B^T of MX-FP4 operands: qa (M x K/2) and qb
    (N x K/2) bytes with their blocked scales, K a multiple of 64."""
    M, K = _by_row(qa, sa_blk, "a", 4)
    N, Kb = _by_row(qb, sb_blk, "b", 4)
    _same_steps("a", K, "b", Kb)
    _shaped(out, "out", (M, N), tuple(TYPES))
    dev = _device(qa, sa_blk, qb, sb_blk, out)
    _call("mx_matmul_fp4", dev, stream, _ptr(qa), _ptr(sa_blk), _ptr(qb), _ptr(sb_blk), M, N, K,
          _ptr(out), TYPES[out.dtype])


def mx_matmul_swiglu(qx, sx_blk, qg, sg_blk, qu, su_blk, h, q0=None, s0_blk=None, bits=8,
                     stream=None):
    """h (M x F, bf16) = silu(X Wg^T) X Wu^T of MX operands X (M x K), Wg and Wu (F x K) with
    elements of `bits`; with q0 and s0_blk both projections' results are saved in 8 bits, as
    mx_swiglu saves its input."""
    M, K = _by_row(qx, sx_blk, "x", bits)
    F, Kg = _by_row(qg, sg_blk, "g", bits)
    Fu, Ku = _by_row(qu, su_blk, "u", bits)
    _same_steps("x", K, "g", Kg)
    _same_steps("x", K, "u", Ku)
    if F != Fu:
        raise ValueError("qg and qu must have equally many rows, got %d and %d" % (F, Fu))
    _shaped(h, "h", (M, F), BF16)
    _saved(q0, s0_blk, M, 2 * F)
    dev = _device(qx, sx_blk, qg, sg_blk, qu, su_blk, h, q0, s0_blk)
    _call("mx_matmul_swiglu", dev, stream, _ptr(qx), _ptr(sx_blk), _ptr(qg), _ptr(sg_blk), _ptr(qu),
          _ptr(su_blk), M, F, K, FORMATS[bits], _ptr(h), _ptr(q0), _ptr(s0_blk))


def mx_matmul_swiglu_backward(qdy, sdy_blk, qw, sw_blk, gu, q0, s0_blk, dgu, bits=8, stream=None):
    """dgu (M x 2F, bf16), the gradient of [g | u], from that of y = h W2^T: MX operands dY
    (M x K) and W2^T (F x K) with elements of `bits`, and gu (bf16), or with gu None the
    saved (q0, s0_blk)."""
    M, K = _by_row(qdy, sdy_blk, "dy", bits)
    F, Kw = _by_row(qw, sw_blk, "w", bits)
    _same_steps("dy", K, "w", Kw)
    if (gu is None) == (q0 is None):
        raise ValueError("give gu, or q0 and s0_blk")
    if gu is not None:
        _shaped(gu, "gu", (M, 2 * F), BF16)
    _saved(q0, s0_blk, M, 2 * F)
    _shaped(dgu, "dgu", (M, 2 * F), BF16)
    dev = _device(qdy, sdy_blk, qw, sw_blk, gu, q0, s0_blk, dgu)
    _call("mx_matmul_swiglu_backward", dev, stream, _ptr(qdy), _ptr(sdy_blk), _ptr(qw), _ptr(sw_blk),
          M, F, K, FORMATS[bits], _ptr(gu), _ptr(q0), _ptr(s0_blk), _ptr(dgu))


def _shaped(t, name, shape, dtypes):
    _dev_tensor(t, name, dtypes=dtypes)
    if tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))


def _saved(q0, s0_blk, M, C):
    """Checks the 8-bit saved form of an (M, C) tensor; both parts or neither."""
    if (q0 is None) != (s0_blk is None):
        raise ValueError("q0 and s0_blk go together")
    if q0 is not None:
        _dev_tensor(q0, "q0", M * C, BYTES)
        _dev_tensor(s0_blk, "s0_blk", mx_blocked_bytes(M, C // 32), BYTES)


def mx_layer_norm(x, w, b, eps, y, mean, rstd, q0=None, s0_blk=None, stream=None):
    """Layer norm of bf16 x (M x D) into caller buffers; with q0 and s0_blk its
    input is saved in 8 bits.  b may be None."""
    _dev_tensor(x, "x", dtypes=BF16, ndim=2)
    M, D = x.shape
    _shaped(w, "w", (D,), tuple(TYPES))
    if b is not None:
        _shaped(b, "b", (D,), (w.dtype,))
    _shaped(y, "y", (M, D), BF16)
    _shaped(mean, "mean", (M,), F32)
    _shaped(rstd, "rstd", (M,), F32)
    _saved(q0, s0_blk, M, D)
    dev = _device(x, w, b, y, mean, rstd, q0, s0_blk)
    _call("mx_layer_norm", dev, stream, _ptr(x), _ptr(w), _ptr(b), TYPES[w.dtype], M, D, eps,
          _ptr(y), _ptr(mean), _ptr(rstd), _ptr(q0), _ptr(s0_blk))


def mx_layer_norm_backward(dy, x, q0, s0_blk, w, mean, rstd, dx, dw, db, work, stream=None):
    """Backward of mx_layer_norm from x, or with x None from (q0, s0_blk); db
    may be None.  work: mx_layer_norm_backward_work_bytes(M, D) bytes."""
    _dev_tensor(dy, "dy", dtypes=BF16, ndim=2)
    M, D = dy.shape
    if (x is None) == (q0 is None):
        raise ValueError("give x, or q0 and s0_blk")
    if x is not None:
        _shaped(x, "x", (M, D), BF16)
    _saved(q0, s0_blk, M, D)
    _shaped(w, "w", (D,), tuple(TYPES))
    _shaped(mean, "mean", (M,), F32)
    _shaped(rstd, "rstd", (M,), F32)
    _shaped(dx, "dx", (M, D), BF16)
    _shaped(dw, "dw", (D,), (w.dtype,))
    if db is not None:
        _shaped(db, "db", (D,), (w.dtype,))
    _dev_tensor(work, "work", mx_layer_norm_backward_work_bytes(M, D))
    dev = _device(dy, x, q0, s0_blk, w, mean, rstd, dx, dw, db, work)
    _call("mx_layer_norm_backward", dev, stream, _ptr(dy), _ptr(x), _ptr(q0), _ptr(s0_blk), _ptr(w),
          TYPES[w.dtype], _ptr(mean), _ptr(rstd), M, D, _ptr(dx), _ptr(dw), _ptr(db), _ptr(work))


def mx_swiglu(gu, h, q0=None, s0_blk=None, stream=None):
    """Gated SiLU of bf16 gu (M x 2F) into h (M x F); with q0 and s0_blk its
    input is saved in 8 bits."""
    _dev_tensor(gu, "gu", dtypes=BF16, ndim=2)
    M, F2 = gu.shape
    if F2 % 2:
        raise ValueError("gu must have an even number of columns, got %d" % F2)
    _shaped(h, "h", (M, F2 // 2), BF16)
    _saved(q0, s0_blk, M, F2)
    _call("mx_swiglu", _device(gu, h, q0, s0_blk), stream, _ptr(gu), M, F2 // 2, _ptr(h), _ptr(q0),
          _ptr(s0_blk))


def mx_swiglu_backward(dh, gu, q0, s0_blk, dgu, stream=None):
    """Backward of mx_swiglu from gu, or with gu None from (q0, s0_blk)."""
    _dev_tensor(dh, "dh", dtypes=BF16, ndim=2)
    M, F = dh.shape
    if (gu is None) == (q0 is None):
        raise ValueError("give gu, or q0 and s0_blk")
    if gu is not None:
        _shaped(gu, "gu", (M, 2 * F), BF16)
    _saved(q0, s0_blk, M, 2 * F)
    _shaped(dgu, "dgu", (M, 2 * F), BF16)
    _call("mx_swiglu_backward", _device(dh, gu, q0, s0_blk, dgu), stream, _ptr(dh), _ptr(gu),
          _ptr(q0), _ptr(s0_blk), M, F, _ptr(dgu))


def mx_selftest_watchdog(wait_ns=50_000_000, stream=None):
    """Run the bounded-wait failure path on the device (no fault): a warp
    waits on a barrier that never completes and gives up after wait_ns."""
    _check(_lib().mx_selftest_watchdog(int(wait_ns), _stream(stream)), "mx_selftest_watchdog")


def mx_selftest_arm_stall(at, wait_ns=20_000_000):
    """Checked builds: arm a stall for this thread's next cast, tiled
    dequantisation or bulk-staged rowwise launch.  CTA 0 gives up waiting at
    its `at`-th tile and takes the abort path, without any fault (see
    include/mxfp8_cast.h).  A release build has no stall hook."""
    rc = _lib().mx_selftest_arm_stall(int(at), int(wait_ns))
    if rc == -1:
        raise RuntimeError("mx_selftest_arm_stall: release build, no stall hook compiled in")
    _check(rc, "mx_selftest_arm_stall")


def mx_bounds_check(clear=True):
    """Stores refused by a bounds-checked build of the library (-1: release
    build, no checks)."""
    rc = _lib().mx_bounds_check(1 if clear else 0)
    if rc < -1:
        raise MXError(rc, "mx_bounds_check")
    return rc


def mx_selftest_bounds(buf16, stream=None):
    """Bounds-checked builds: one refused store just past an 8-byte span over
    buf16 (a 16-byte CUDA tensor); returns 0, or -1 in a release build."""
    _dev_tensor(buf16, "buf16", 16)
    dev = _device(buf16)
    with torch.cuda.device(dev):
        rc = _lib().mx_selftest_bounds(_ptr(buf16), _stream(stream, dev))
    if rc < -1:
        raise MXError(rc, "mx_selftest_bounds")
    return rc


def mx_watchdog(clear=True):
    rc = _lib().mx_watchdog(1 if clear else 0)
    if rc < 0:
        raise MXError(rc, "mx_watchdog")
    return rc


# ---- allocating wrappers ------------------------------------------------------

def _u8(n, device):
    return torch.empty(n, dtype=torch.uint8, device=device)


def cast_dim0_dim1(x, stream=None):
    """Returns (q0 (M,K), s0_blk, q1 (K,M), s1_blk) as uint8 tensors."""
    r = _compiled("cast_dim0_dim1", x) if stream is None else None
    if r is not None:
        return r
    M, K = x.shape
    q0 = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    q1 = torch.empty((K, M), dtype=torch.uint8, device=x.device)
    s0 = _u8(mx_blocked_bytes(M, K // 32), x.device)
    s1 = _u8(mx_blocked_bytes(K, M // 32), x.device)
    mx_cast_dim0_dim1(x, q0, s0, q1, s1, stream)
    return q0, s0, q1, s1


def cast_dim0(x, stream=None):
    r = _compiled("cast_dim0", x) if stream is None else None
    if r is not None:
        return r
    M, K = x.shape
    q0 = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    s0 = _u8(mx_blocked_bytes(M, K // 32), x.device)
    mx_cast_dim0(x, q0, s0, stream)
    return q0, s0


def cast_dim1(x, stream=None):
    r = _compiled("cast_dim1", x) if stream is None else None
    if r is not None:
        return r
    M, K = x.shape
    q1 = torch.empty((K, M), dtype=torch.uint8, device=x.device)
    s1 = _u8(mx_blocked_bytes(K, M // 32), x.device)
    mx_cast_dim1(x, q1, s1, stream)
    return q1, s1


def scales_to_blocked(s, stream=None):
    R, C = s.shape
    out = _u8(mx_blocked_bytes(R, C), s.device)
    mx_scales_to_blocked(s, out, stream)
    return out


def cast_grouped_m(x, offs, stream=None):
    """offs: int32 CUDA tensor of cumulative group ends.  Returns
    (q0, s0_blk, s0_row_offs, q1, s1_blk, s1_col_offs, status)."""
    M, K = x.shape
    G = offs.numel()
    dev = x.device
    q0 = torch.empty((M, K), dtype=torch.uint8, device=dev)
    q1 = torch.empty((K, M), dtype=torch.uint8, device=dev)
    s0 = _u8(mx_grouped_m_scale_bytes(M, K, G, 0), dev)
    s1 = _u8(mx_grouped_m_scale_bytes(M, K, G, 1), dev)
    r0 = torch.empty(G + 1, dtype=torch.int64, device=dev)
    c1 = torch.empty(G + 1, dtype=torch.int64, device=dev)
    st = torch.empty(1, dtype=torch.int32, device=dev)
    mx_cast_grouped_m(x, offs, q0, s0, r0, q1, s1, c1, st, stream)
    return q0, s0, r0, q1, s1, c1, st


def cast_3d_dim1(w, stream=None):
    E, N, K = w.shape
    q1 = torch.empty((K, E * N), dtype=torch.uint8, device=w.device)
    s1 = _u8(mx_3d_scale_bytes(E, N, K), w.device)
    mx_cast_3d_dim1(w, q1, s1, stream)
    return q1, s1


def cast_3d_dim0(w, stream=None):
    """Returns (q0 (E, N, K), s0_blk) as uint8 tensors."""
    E, N, K = w.shape
    q0 = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    s0 = _u8(mx_3d_dim0_scale_bytes(E, N, K), w.device)
    mx_cast_3d_dim0(w, q0, s0, stream)
    return q0, s0


def cast_3d_dim0_dim1(w, stream=None):
    """Returns (q0 (E, N, K), s0_blk, q1 (K, E*N), s1_blk)."""
    E, N, K = w.shape
    q0 = torch.empty((E, N, K), dtype=torch.uint8, device=w.device)
    q1 = torch.empty((K, E * N), dtype=torch.uint8, device=w.device)
    s0 = _u8(mx_3d_dim0_scale_bytes(E, N, K), w.device)
    s1 = _u8(mx_3d_scale_bytes(E, N, K), w.device)
    mx_cast_3d_dim0_dim1(w, q0, s0, q1, s1, stream)
    return q0, s0, q1, s1


def dequant_blocked(q, s_blk, stream=None):
    """bf16 tensor of the same shape as the 2D uint8 tensor q."""
    R, C = q.shape
    out = torch.empty((R, C), dtype=torch.bfloat16, device=q.device)
    mx_dequant_blocked(q, s_blk, out, stream)
    return out


def cast_tensorwise(x, stream=None):
    """Returns (q uint8 shaped like x, scale float32 (1,), amax float32 (1,))."""
    q = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(1, dtype=torch.float32, device=x.device)
    amax = torch.empty(1, dtype=torch.float32, device=x.device)
    mx_cast_tensorwise(x, q, scale, amax, stream)
    return q, scale, amax


def cast_rowwise(x, stream=None):
    """Returns (q (M, K) uint8, scale (M,) bfloat16)."""
    M, K = x.shape
    q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    scale = torch.empty(M, dtype=torch.bfloat16, device=x.device)
    mx_cast_rowwise(x, q, scale, stream)
    return q, scale


# The training operators below are called per layer, on tensors that may take the
# GPU a few microseconds: their usual calls go through the compiled wrappers,
# which answer None where an argument is not what they know; the checked path
# then works, or raises the error that says what is wrong.

def _compiled(name, *args):
    """The outputs of compiled wrapper `name`, or None."""
    lib = _LIB or _lib()
    if _CALL is None:
        return None
    r = getattr(_CALL, name)(lib.addresses["mx_" + name], *args)
    if type(r) is int:
        raise MXError(r, "mx_" + name)
    return r


def _on_stream(stream, t):
    """Context for a call on `stream` (a torch.cuda.Stream or a raw handle): it
    becomes the current stream, so that what the call allocates is that
    stream's and goes back to the allocator in its order."""
    _stream(stream, _device(t))
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    return torch.cuda.stream(stream)


def _split_saved(saved):
    """(tensor, None, None) of a bf16 tensor, (None, q0, s0_blk) of a pair."""
    return (saved, None, None) if isinstance(saved, torch.Tensor) else (None, *saved)


def matmul(qa, sa_blk, qb, sb_blk, out_dtype=torch.bfloat16, stream=None):
    """A B^T of MX operands as a (M, N) tensor of out_dtype."""
    if stream is not None:
        with _on_stream(stream, qa):
            return matmul(qa, sa_blk, qb, sb_blk, out_dtype)
    if out_dtype not in TYPES:
        raise TypeError("out_dtype must be one of %s, got %s"
                        % (", ".join(str(d) for d in TYPES), out_dtype))
    out = _compiled("matmul", qa, sa_blk, qb, sb_blk, TYPES[out_dtype])
    if out is None:
        out = torch.empty((qa.shape[0], qb.shape[0]), dtype=out_dtype, device=qa.device)
        mx_matmul(qa, sa_blk, qb, sb_blk, out)
    return out


def cast_fp4_dim0(x, stream=None):
    """Returns (q0 (M, K/2), s0_blk) as uint8 tensors, two e2m1 values a byte."""
    if stream is not None:
        with _on_stream(stream, x):
            return cast_fp4_dim0(x)
    r = _compiled("cast_fp4_dim0", x)
    if r is not None:
        return r
    M, K = x.shape
    q0 = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    s0 = _u8(mx_blocked_bytes(M, K // 32), x.device)
    mx_cast_fp4_dim0(x, q0, s0)
    return q0, s0


def cast_fp4_dim1(x, stream=None):
    """Returns (q1 (K, M/2), s1_blk)."""
    if stream is not None:
        with _on_stream(stream, x):
            return cast_fp4_dim1(x)
    r = _compiled("cast_fp4_dim1", x)
    if r is not None:
        return r
    M, K = x.shape
    q1 = torch.empty((K, M // 2), dtype=torch.uint8, device=x.device)
    s1 = _u8(mx_blocked_bytes(K, M // 32), x.device)
    mx_cast_fp4_dim1(x, q1, s1)
    return q1, s1


def cast_fp4_dim0_dim1(x, stream=None):
    """Returns (q0 (M, K/2), s0_blk, q1 (K, M/2), s1_blk)."""
    if stream is not None:
        with _on_stream(stream, x):
            return cast_fp4_dim0_dim1(x)
    r = _compiled("cast_fp4_dim0_dim1", x)
    if r is not None:
        return r
    M, K = x.shape
    q0 = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    q1 = torch.empty((K, M // 2), dtype=torch.uint8, device=x.device)
    s0 = _u8(mx_blocked_bytes(M, K // 32), x.device)
    s1 = _u8(mx_blocked_bytes(K, M // 32), x.device)
    mx_cast_fp4_dim0_dim1(x, q0, s0, q1, s1)
    return q0, s0, q1, s1


def dequant_fp4(q, s_blk, stream=None):
    """bf16 (R, C) of MX-FP4 bytes q (R, C/2)."""
    if stream is not None:
        with _on_stream(stream, q):
            return dequant_fp4(q, s_blk)
    out = _compiled("dequant_fp4", q, s_blk)
    if out is None:
        R, C2 = q.shape
        out = torch.empty((R, 2 * C2), dtype=torch.bfloat16, device=q.device)
        mx_dequant_fp4(q, s_blk, out)
    return out


def matmul_fp4(qa, sa_blk, qb, sb_blk, out_dtype=torch.bfloat16, stream=None):
    """A B^T of MX-FP4 operands as a (M, N) tensor of out_dtype.  A row's last bits may be
    others in a batch of another M."""
    if stream is not None:
        with _on_stream(stream, qa):
            return matmul_fp4(qa, sa_blk, qb, sb_blk, out_dtype)
    if out_dtype not in TYPES:
        raise TypeError("out_dtype must be one of %s, got %s"
                        % (", ".join(str(d) for d in TYPES), out_dtype))
    out = _compiled("matmul_fp4", qa, sa_blk, qb, sb_blk, TYPES[out_dtype])
    if out is None:
        out = torch.empty((qa.shape[0], qb.shape[0]), dtype=out_dtype, device=qa.device)
        mx_matmul_fp4(qa, sa_blk, qb, sb_blk, out)
    return out


def _gate_and_up(qw, sw_blk, bits):
    """(qg, sg_blk, qu, su_blk) of two pairs, or of the cast of [Wg; Wu] as views of it."""
    if not isinstance(qw, torch.Tensor):
        return qw[0], sw_blk[0], qw[1], sw_blk[1]
    F2, K = _by_row(qw, sw_blk, "w", bits)
    F = F2 // 2
    if F2 % 256:
        raise ValueError("the halves of %d rows of qw do not begin on a scale tile of 128 rows: cast "
                         "them apart and give pairs (gate, up)" % F2)
    n = mx_blocked_bytes(F, K // 32)
    s = sw_blk.view(-1)
    return qw[:F], s[:n], qw[F:], s[n:]


def matmul_swiglu(qx, sx_blk, qw, sw_blk, save=False, bits=8, stream=None):
    """h = silu(g) u, g = X Wg^T, u = X Wu^T, of MX operands with elements of `bits` (8 or 4):
    X (M, K), and either Wg and Wu (F, K) as pairs (gate, up) of bytes and of scales, or,
    with F a multiple of 128, [Wg; Wu] (2F, K) in one.  Returns h (M, F), with save=True
    (h, q0, s0_blk): [g | u] saved in 8 bits for the backward pass.  A row's last bits may be
    others in a batch of another M and, past 1792 steps K (in 4 bits 2560), with the save."""
    if stream is not None:
        with _on_stream(stream, qx):
            return matmul_swiglu(qx, sx_blk, qw, sw_blk, save, bits)
    if bits not in FORMATS:
        raise ValueError("bits must be 8 or 4, got %r" % (bits,))
    r = _compiled("matmul_swiglu", qx, sx_blk, qw, sw_blk, FORMATS[bits], save)
    if r is not None:
        return r
    qg, sg, qu, su = _gate_and_up(qw, sw_blk, bits)
    M, F = qx.shape[0], qg.shape[0]
    h = torch.empty((M, F), dtype=torch.bfloat16, device=qx.device)
    if not save:
        mx_matmul_swiglu(qx, sx_blk, qg, sg, qu, su, h, bits=bits)
        return h
    q0 = torch.empty((M, 2 * F), dtype=torch.uint8, device=qx.device)
    s0 = _u8(mx_blocked_bytes(M, 2 * F // 32), qx.device)
    mx_matmul_swiglu(qx, sx_blk, qg, sg, qu, su, h, q0, s0, bits)
    return h, q0, s0


def matmul_swiglu_backward(qdy, sdy_blk, qw, sw_blk, saved, bits=8, stream=None):
    """The gradient of [g | u] (M, 2F) from that of y = h W2^T: MX operands dY (M, K) and
    W2^T (F, K) with elements of `bits`.  saved: bf16 [g | u], or the forward pass's pair
    (q0, s0_blk)."""
    if stream is not None:
        with _on_stream(stream, qdy):
            return matmul_swiglu_backward(qdy, sdy_blk, qw, sw_blk, saved, bits)
    if bits not in FORMATS:
        raise ValueError("bits must be 8 or 4, got %r" % (bits,))
    r = _compiled("matmul_swiglu_backward", qdy, sdy_blk, qw, sw_blk, FORMATS[bits], saved)
    if r is not None:
        return r
    gu, q0, s0 = _split_saved(saved)
    dgu = torch.empty((qdy.shape[0], 2 * qw.shape[0]), dtype=torch.bfloat16, device=qdy.device)
    mx_matmul_swiglu_backward(qdy, sdy_blk, qw, sw_blk, gu, q0, s0, dgu, bits)
    return dgu


def layer_norm(x, w, b=None, eps=1e-5, save=False, stream=None):
    """Layer norm of bf16 x (M, D).  Returns (y, mean, rstd), with save=True
    (y, mean, rstd, q0, s0_blk): x saved in 8 bits for the backward pass."""
    if stream is not None:
        with _on_stream(stream, x):
            return layer_norm(x, w, b, eps, save)
    r = _compiled("layer_norm", x, w, b, eps, save)
    if r is not None:
        return r
    M, D = x.shape
    y = torch.empty((M, D), dtype=torch.bfloat16, device=x.device)
    mean = torch.empty(M, dtype=torch.float32, device=x.device)
    rstd = torch.empty(M, dtype=torch.float32, device=x.device)
    if not save:
        mx_layer_norm(x, w, b, eps, y, mean, rstd)
        return y, mean, rstd
    q0 = torch.empty((M, D), dtype=torch.uint8, device=x.device)
    s0 = _u8(mx_blocked_bytes(M, D // 32), x.device)
    mx_layer_norm(x, w, b, eps, y, mean, rstd, q0, s0)
    return y, mean, rstd, q0, s0


def layer_norm_backward(dy, saved, w, mean, rstd, bias=True, stream=None):
    """saved: the forward pass's bf16 x, or the pair (q0, s0_blk).  Returns
    (dx, dw, db), the last two in w's type; db is None with bias=False."""
    if stream is not None:
        with _on_stream(stream, dy):
            return layer_norm_backward(dy, saved, w, mean, rstd, bias)
    r = _compiled("layer_norm_backward",
                  (_LIB or _lib()).addresses["mx_layer_norm_backward_work_bytes"], dy, saved, w,
                  mean, rstd, bias)
    if r is not None:
        return r
    x, q0, s0 = _split_saved(saved)
    M, D = dy.shape
    dx = torch.empty((M, D), dtype=torch.bfloat16, device=dy.device)
    dw = torch.empty(D, dtype=w.dtype, device=dy.device)
    db = torch.empty(D, dtype=w.dtype, device=dy.device) if bias else None
    work = _u8(mx_layer_norm_backward_work_bytes(M, D), dy.device)
    mx_layer_norm_backward(dy, x, q0, s0, w, mean, rstd, dx, dw, db, work)
    return dx, dw, db


def swiglu(gu, save=False, stream=None):
    """h = silu(g) u of bf16 gu = [g | u] (M, 2F).  Returns h (M, F), with
    save=True (h, q0, s0_blk): gu saved in 8 bits for the backward pass."""
    if stream is not None:
        with _on_stream(stream, gu):
            return swiglu(gu, save)
    r = _compiled("swiglu", gu, save)
    if r is not None:
        return r
    M, F2 = gu.shape
    h = torch.empty((M, F2 // 2), dtype=torch.bfloat16, device=gu.device)
    if not save:
        mx_swiglu(gu, h)
        return h
    q0 = torch.empty((M, F2), dtype=torch.uint8, device=gu.device)
    s0 = _u8(mx_blocked_bytes(M, F2 // 32), gu.device)
    mx_swiglu(gu, h, q0, s0)
    return h, q0, s0


def swiglu_backward(dh, saved, stream=None):
    """saved: the forward pass's bf16 gu, or the pair (q0, s0_blk).  Returns
    the gradient of gu (M, 2F)."""
    if stream is not None:
        with _on_stream(stream, dh):
            return swiglu_backward(dh, saved)
    r = _compiled("swiglu_backward", dh, saved)
    if r is not None:
        return r
    gu, q0, s0 = _split_saved(saved)
    M, F = dh.shape
    dgu = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=dh.device)
    mx_swiglu_backward(dh, gu, q0, s0, dgu)
    return dgu
