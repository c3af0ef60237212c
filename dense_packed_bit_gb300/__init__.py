"""dense_packed_bit_gb300 -- fp32 dense GEMM, packed 2-bit GEMV / skinny GEMM and packed
4-bit GEMV on GB300.

Thin ctypes binding over libmm.so (the C ABI declared in include/mm.h).  The
functions keep the C names and argument order; tensors are torch CUDA tensors
(only their device pointers are passed) and `stream` defaults to torch's
current stream.  Every step of the computation runs in libmm's CUDA kernels:
there is no CPU or PyTorch fallback, and a missing or unloadable libmm.so is
an error.
"""
from __future__ import annotations

import ctypes
import os
import threading

__all__ = [
    "MMError", "load_library", "library_path", "mm_version", "mm_last_error",
    "mm_gemm_f32", "mm_gemm_f32_ex", "mm_gemv_packed2", "mm_gemv_packed2_ex",
    "mm_gemm_packed2", "mm_gemm_packed2_ex", "mm_gemv_packed4", "mm_gemv_packed4_ex",
    "mm_check_device_error", "mm_gemm_f32_splitk", "mm_gemm_f32_splitk_workspace", "mm_gemm_f32_splitk_noalloc",
    "MM_SPLITK_NOALLOC_MAX_FLOATS", "mm_gemm_f32_bias_act", "MM_ACT_NONE", "MM_ACT_GELU_TANH",
    "mm_gemv_packed2_strided_batched", "mm_gemv_packed2_strided_batched_ex", "mm_gemm_f32_bias_act_splitk",
    "mm_gemm_f32_split_plan", "mm_gemm_f32_splitk_ex", "mm_gemm_f32_splitk_workspace_ex", "mm_gemm_f32_split_plan_ex",
    "mm_probe_bounded_wait", "mm_attention_fwd", "mm_attention_bwd",
    "mm_cache", "mm_cache_reserve", "mm_cache_append", "mm_cache_compact", "mm_cache_fork", "mm_cache_free",
    "mm_cache_copy_pages", "mm_cache_attention_workspace", "mm_cache_attention", "mm_cache_attention_tree",
    "mm_sample", "MM_F16", "MM_BF16", "MM_F32",
    "MM_OK", "MM_ERR_INVALID_ARG", "MM_ERR_UNSUPPORTED", "MM_ERR_CUDA", "MM_ERR_TIMEOUT",
    "MM_GEMM_AUTO", "MM_GEMM_FFMA", "MM_GEMM_TF32X3",
    "MM_DEQ_AUTO", "MM_DEQ_SELECT", "MM_DEQ_AFFINE", "MM_DEQ_MMA", "MM_DEQ_FP8", "MM_DEQ_TC", "MM_DEQ_MXF4",
]

MM_OK, MM_ERR_INVALID_ARG, MM_ERR_UNSUPPORTED, MM_ERR_CUDA, MM_ERR_TIMEOUT = 0, 1, 2, 3, 4
MM_GEMM_AUTO, MM_GEMM_FFMA, MM_GEMM_TF32X3 = 0, 1, 2
MM_DEQ_AUTO, MM_DEQ_SELECT, MM_DEQ_AFFINE, MM_DEQ_MMA, MM_DEQ_FP8, MM_DEQ_TC, MM_DEQ_MXF4 = 0, 1, 2, 3, 4, 5, 6
MM_SPLITK_NOALLOC_MAX_FLOATS = 4194304  # floats of the static split-K scratch (16 MiB), as in mm.h
MM_ACT_NONE, MM_ACT_GELU_TANH = 0, 1
MM_F16, MM_BF16, MM_F32 = 0, 1, 2

_PKG = os.path.dirname(os.path.abspath(__file__))
_lock = threading.Lock()
_lib = None
_torch = None
_cuda = False  # CUDA was seen to be initialised

# symbol -> (argtypes, restype); mirrors include/mm.h
_P, _I64, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class GemmOpts(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int), ("tile", ctypes.c_int), ("splitk", ctypes.c_int), ("reserved", ctypes.c_int * 5)]


class GemvOpts(ctypes.Structure):
    _fields_ = [("split", ctypes.c_int), ("rows_per_lane", ctypes.c_int), ("warps", ctypes.c_int),
                ("dequant", ctypes.c_int), ("pdl", ctypes.c_int), ("weights_static", ctypes.c_int),
                ("independent", ctypes.c_int), ("staging", ctypes.c_int), ("reserved", ctypes.c_int * 4)]


class GemmPacked2Opts(ctypes.Structure):
    _fields_ = [("tile", ctypes.c_int), ("splitk", ctypes.c_int), ("pdl", ctypes.c_int),
                ("weights_static", ctypes.c_int), ("ntok", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


class Gemv4Opts(ctypes.Structure):
    _fields_ = [("blocks", ctypes.c_int), ("pdl", ctypes.c_int), ("weights_static", ctypes.c_int),
                ("independent", ctypes.c_int), ("staging", ctypes.c_int), ("reserved", ctypes.c_int * 3)]


class Cache(ctypes.Structure):
    """mm_cache of mm.h; mm_cache() makes one from tensors."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("refs", ctypes.c_void_p), ("layers", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("page_size", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("seqs", ctypes.c_int64), ("max_pages", ctypes.c_int64), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64),
                ("dtype", ctypes.c_int), ("reserved", ctypes.c_int * 5)]


_PC, _PI64, _F = ctypes.POINTER(Cache), ctypes.POINTER(ctypes.c_int64), ctypes.c_float

SIGNATURES = {
    "mm_version": ([], ctypes.c_int),
    "mm_last_error": ([], ctypes.c_char_p),
    "mm_gemm_f32": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P], ctypes.c_int),
    "mm_gemm_f32_ex": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                        ctypes.POINTER(GemmOpts)], ctypes.c_int),
    "mm_gemv_packed2": ([_P, _P, _P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "mm_gemv_packed2_ex": ([_P, _P, _P, _P, _I64, _I64, _P, _P, ctypes.POINTER(GemvOpts)], ctypes.c_int),
    "mm_gemm_packed2": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _P], ctypes.c_int),
    "mm_gemv_packed4": ([_P, _P, _P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "mm_gemv_packed4_ex": ([_P, _P, _P, _P, _I64, _I64, _P, _P, ctypes.POINTER(Gemv4Opts)], ctypes.c_int),
    "mm_gemm_packed2_ex": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _P, ctypes.POINTER(GemmPacked2Opts)],
                           ctypes.c_int),
    "mm_check_device_error": ([_P], ctypes.c_int),
    "mm_gemm_f32_splitk_workspace": ([_I64, _I64, _I64, _I, ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
    "mm_gemm_f32_splitk": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _P, _I64, _P],
                           ctypes.c_int),
    "mm_gemm_f32_splitk_noalloc": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _P],
                                   ctypes.c_int),
    "mm_gemm_f32_bias_act": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I, _P, _I64, _P], ctypes.c_int),
    "mm_gemm_f32_split_plan": ([_I64, _I64, _I64, _I, _P, _P], ctypes.c_int),
    "mm_gemm_f32_splitk_ex": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _I, _P, _I64, _P,
                               ctypes.POINTER(GemmOpts)], ctypes.c_int),
    "mm_gemm_f32_splitk_workspace_ex": ([_I64, _I64, _I64, _I, ctypes.POINTER(GemmOpts),
                                         ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
    "mm_gemm_f32_split_plan_ex": ([_I64, _I64, _I64, _I, ctypes.POINTER(GemmOpts), _P, _P], ctypes.c_int),
    "mm_gemm_f32_bias_act_splitk": ([_I, _I, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I, _P, _I64, _I, _P, _I64,
                                     _P], ctypes.c_int),
    "mm_gemv_packed2_strided_batched": ([_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P],
                                        ctypes.c_int),
    "mm_gemv_packed2_strided_batched_ex": ([_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I64, _I64, _I64, _P, _P,
                                            ctypes.POINTER(GemvOpts)], ctypes.c_int),
    "mm_probe_bounded_wait": ([_I, ctypes.c_uint64, _P, _P], ctypes.c_int),
    "mm_cache_reserve": ([_PC, _P, _P, _P], ctypes.c_int),
    "mm_cache_append": ([_PC, _I64, _P, _P, _I64, _P, _I64, _I64, _P], ctypes.c_int),
    "mm_cache_compact": ([_PC, _P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "mm_cache_fork": ([_PC, _P, _P, _I64, _P, _P], ctypes.c_int),
    "mm_cache_free": ([_PC, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "mm_cache_copy_pages": ([_PC, _P, _P, _I64, _P], ctypes.c_int),
    "mm_cache_attention_workspace": ([_PC, _I64, _I64, _I64, _PI64], ctypes.c_int),
    "mm_cache_attention": ([_PC, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _I64, _F, _P, _I64, _P, _I64, _P],
                           ctypes.c_int),
    "mm_cache_attention_tree": ([_PC, _I64, _P, _I64, _I64, _P, _I64, _I64, _P, _I64, _I64, _I64, _F, _P, _I64, _P,
                                 _I64, _P], ctypes.c_int),
    "mm_sample": ([_P, _I, _I64, _I64, _I64, _P, _P, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "mm_attention_fwd": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, ctypes.c_float, _P], ctypes.c_int),
    "mm_attention_bwd": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, ctypes.c_float, _P],
                         ctypes.c_int),
}


class MMError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"libmm status {status}: {message}")
        self.status = status


def library_path() -> str:
    return os.environ.get("MM_LIBRARY", os.path.join(_PKG, "libmm.so"))


def load_library():
    """Load libmm.so (built by dense_packed_bit_gb300.build); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise MMError(MM_ERR_UNSUPPORTED,
                              f"{path} not found: build it with `python -m dense_packed_bit_gb300.build`")
            lib = ctypes.CDLL(path)
            for name, (argt, rest) in SIGNATURES.items():
                fn = getattr(lib, name)
                fn.argtypes = argt
                fn.restype = rest
            _lib = lib
    return _lib


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        torch = _torch_module()
        global _cuda
        if _cuda or torch.cuda.is_initialized():  # the current stream's handle without an object around it
            _cuda = True
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _codebook(cb, n=4):
    if cb is None:
        return None
    vals = [float(v) for v in (cb.tolist() if hasattr(cb, "tolist") else cb)]
    if len(vals) != n:
        raise ValueError(f"codebook needs {n} entries")
    return (ctypes.c_float * n)(*vals)


def _check(status: int):
    if status != MM_OK:
        msg = load_library().mm_last_error()
        raise MMError(status, msg.decode() if msg else "")


def mm_version() -> int:
    return load_library().mm_version()


def mm_last_error() -> str:
    return load_library().mm_last_error().decode()


def mm_gemm_f32(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, stream=None):
    _check(load_library().mm_gemm_f32(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                      _ptr(C), ldc, _stream(stream)))


def mm_gemm_f32_ex(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, stream=None, *, path=0, tile=0, splitk=0):
    o = GemmOpts(path, tile, splitk)
    _check(load_library().mm_gemm_f32_ex(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                         _ptr(C), ldc, _stream(stream), ctypes.byref(o)))


def mm_gemm_f32_splitk_workspace(M, N, K, splitk=0) -> int:
    """Floats of workspace mm_gemm_f32_splitk needs for these sizes and split (0 = automatic)."""
    out = ctypes.c_int64(0)
    _check(load_library().mm_gemm_f32_splitk_workspace(M, N, K, splitk, ctypes.byref(out)))
    return out.value


def mm_gemm_f32_splitk(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, splitk, workspace, workspace_floats,
                       stream=None):
    _check(load_library().mm_gemm_f32_splitk(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                             _ptr(C), ldc, int(splitk), _ptr(workspace), int(workspace_floats),
                                             _stream(stream)))


def mm_gemm_f32_split_plan(M, N, K, sms):
    """(splitk, workspace_floats) of the automatic split on a GPU with `sms` SMs; no device needed."""
    sk = ctypes.c_int(0)
    fl = ctypes.c_int64(0)
    _check(load_library().mm_gemm_f32_split_plan(M, N, K, int(sms), ctypes.byref(sk), ctypes.byref(fl)))
    return sk.value, fl.value


def mm_gemm_f32_splitk_ex(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, splitk, workspace, workspace_floats,
                          stream=None, *, path=0, tile=0, opt_splitk=0):
    """mm_gemm_f32_splitk with a kernel choice (path 1: the FFMA kernel and its stream-K tail)."""
    o = GemmOpts(path, tile, opt_splitk)
    _check(load_library().mm_gemm_f32_splitk_ex(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                                _ptr(C), ldc, int(splitk), _ptr(workspace), int(workspace_floats),
                                                _stream(stream), ctypes.byref(o)))


def mm_gemm_f32_splitk_workspace_ex(M, N, K, splitk=0, *, path=0, tile=0, opt_splitk=0) -> int:
    """Floats of workspace mm_gemm_f32_splitk_ex needs for these sizes, split and options."""
    o = GemmOpts(path, tile, opt_splitk)
    out = ctypes.c_int64(0)
    _check(load_library().mm_gemm_f32_splitk_workspace_ex(M, N, K, int(splitk), ctypes.byref(o), ctypes.byref(out)))
    return out.value


def mm_gemm_f32_split_plan_ex(M, N, K, sms, *, path=0, tile=0, opt_splitk=0):
    """(splitk, workspace_floats) of mm_gemm_f32_splitk_ex's automatic split for `sms` SMs; no device needed."""
    o = GemmOpts(path, tile, opt_splitk)
    sk = ctypes.c_int(0)
    fl = ctypes.c_int64(0)
    _check(load_library().mm_gemm_f32_split_plan_ex(M, N, K, int(sms), ctypes.byref(o), ctypes.byref(sk),
                                                    ctypes.byref(fl)))
    return sk.value, fl.value


def mm_gemm_f32_bias_act_splitk(transA, transB, M, N, K, A, lda, B, ldb, bias, act, C, ldc, splitk=0,
                                workspace=None, workspace_floats=0, stream=None):
    """mm_gemm_f32_bias_act with the K split of mm_gemm_f32_splitk (0: automatic, -1: stream-K)."""
    _check(load_library().mm_gemm_f32_bias_act_splitk(
        int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb, _ptr(bias), int(act), _ptr(C), ldc,
        int(splitk), _ptr(workspace), workspace_floats, _stream(stream)))


def mm_gemv_packed2_strided_batched(codes, codes_stride, scales, scales_stride, x, x_stride, y, y_stride, batch,
                                    rows, cols, codebook, stream=None):
    """y_b = W_b x_b for b < batch, matrix b's operands at b times the strides (x_stride 0: shared x)."""
    _check(load_library().mm_gemv_packed2_strided_batched(
        _ptr(codes), codes_stride, _ptr(scales), scales_stride, _ptr(x), x_stride, _ptr(y), y_stride, batch, rows,
        cols, _codebook(codebook), _stream(stream)))


def mm_gemv_packed2_strided_batched_ex(codes, codes_stride, scales, scales_stride, x, x_stride, y, y_stride, batch,
                                       rows, cols, codebook, stream=None, *, dequant=0, rows_per_lane=0, pdl=0,
                                       weights_static=0, independent=0):
    """mm_gemv_packed2_strided_batched with a decode choice (dequant: 0, MM_DEQ_AFFINE or MM_DEQ_MXF4;
    rows_per_lane: 127-row tiles per CTA for MM_DEQ_MXF4, 0 = automatic; pdl / weights_static /
    independent: programmatic dependent launch options of the fp4 decode)."""
    o = GemvOpts(0, rows_per_lane, 0, dequant, pdl, weights_static, independent, -1)
    _check(load_library().mm_gemv_packed2_strided_batched_ex(
        _ptr(codes), codes_stride, _ptr(scales), scales_stride, _ptr(x), x_stride, _ptr(y), y_stride, batch, rows,
        cols, _codebook(codebook), _stream(stream), ctypes.byref(o)))


def mm_gemm_f32_bias_act(transA, transB, M, N, K, A, lda, B, ldb, bias, act, C, ldc, stream=None):
    """C = act(op(A) op(B) + bias): GPT-2's linear layer (bias per column) and GELU (act=1)."""
    _check(load_library().mm_gemm_f32_bias_act(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                               _ptr(bias), int(act), _ptr(C), ldc, _stream(stream)))


def mm_gemm_f32_splitk_noalloc(transA, transB, M, N, K, A, lda, B, ldb, C, ldc, splitk=0, stream=None):
    """Split-K GEMM into the library's static scratch: for callers that cannot allocate device
    memory (or hand over a workspace) where they multiply.  Calls that overlap on the GPU race."""
    _check(load_library().mm_gemm_f32_splitk_noalloc(int(transA), int(transB), M, N, K, _ptr(A), lda, _ptr(B), ldb,
                                                     _ptr(C), ldc, int(splitk), _stream(stream)))


def mm_gemv_packed2(codes, scales, x, y, rows, cols, codebook, stream=None):
    _check(load_library().mm_gemv_packed2(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), rows, cols,
                                          _codebook(codebook), _stream(stream)))


def mm_gemv_packed2_ex(codes, scales, x, y, rows, cols, codebook, stream=None, *, split=0,
                       rows_per_lane=0, warps=0, dequant=0, pdl=0, weights_static=0, independent=0, staging=-1):
    o = GemvOpts(split, rows_per_lane, warps, dequant, pdl, weights_static, independent, staging)
    _check(load_library().mm_gemv_packed2_ex(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), rows, cols,
                                             _codebook(codebook), _stream(stream), ctypes.byref(o)))


def mm_gemm_packed2(codes, scales, X, Y, M, rows, cols, codebook, stream=None):
    _check(load_library().mm_gemm_packed2(_ptr(codes), _ptr(scales), _ptr(X), _ptr(Y), M, rows, cols,
                                          _codebook(codebook), _stream(stream)))


def mm_gemm_packed2_ex(codes, scales, X, Y, M, rows, cols, codebook, stream=None, *, tile=0, splitk=0, pdl=0,
                       weights_static=0, ntok=0):
    o = GemmPacked2Opts(tile, splitk, pdl, weights_static, ntok)
    _check(load_library().mm_gemm_packed2_ex(_ptr(codes), _ptr(scales), _ptr(X), _ptr(Y), M, rows, cols,
                                             _codebook(codebook), _stream(stream), ctypes.byref(o)))


def mm_check_device_error(stream=None):
    _check(load_library().mm_check_device_error(_stream(stream)))


def mm_probe_bounded_wait(arrive, limit_ns, out=None, stream=None):
    """One bounded device wait that completes (arrive=1) or runs out after limit_ns (arrive=0);
    out: None or a device int64 tensor of 2 receiving (completed, ns waited)."""
    _check(load_library().mm_probe_bounded_wait(int(arrive), int(limit_ns), _ptr(out), _stream(stream)))


def mm_gemv_packed4(codes, scales, x, y, rows, cols, codebook, stream=None):
    _check(load_library().mm_gemv_packed4(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), rows, cols,
                                          _codebook(codebook, 16), _stream(stream)))


def mm_gemv_packed4_ex(codes, scales, x, y, rows, cols, codebook, stream=None, *, blocks=0, pdl=0,
                       weights_static=0, independent=0, staging=-1):
    o = Gemv4Opts(blocks, pdl, weights_static, independent, staging)
    _check(load_library().mm_gemv_packed4_ex(_ptr(codes), _ptr(scales), _ptr(x), _ptr(y), rows, cols,
                                             _codebook(codebook, 16), _stream(stream), ctypes.byref(o)))


def mm_attention_fwd(Q, K, V, O, L, heads, T, D, causal, scale, stream=None):
    """O = softmax(scale Q K^T (+ causal mask)) V per head, L = the rows' log-sum-exp; [heads][T][D] fp32."""
    _check(load_library().mm_attention_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(L), heads, T, D, int(causal),
                                           float(scale), _stream(stream)))


def mm_attention_bwd(Q, K, V, O, dO, L, dQ, dK, dV, heads, T, D, causal, scale, stream=None):
    """Gradients of sum(O * dO) with respect to Q, K, V, from the forward's O and L."""
    _check(load_library().mm_attention_bwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(L), _ptr(dQ),
                                           _ptr(dK), _ptr(dV), heads, T, D, int(causal), float(scale),
                                           _stream(stream)))


def _dtype(t) -> int:
    dtype, torch = t.dtype, _torch_module()
    if dtype is torch.float32:
        return MM_F32
    if dtype is torch.float16:
        return MM_F16
    if dtype is torch.bfloat16:
        return MM_BF16
    raise ValueError(f"no kernel takes {dtype}")


def _int32(t, what, shape):
    if str(t.dtype) != "torch.int32" or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{what} must be a contiguous int32 tensor of shape {tuple(shape)}")


# What the library cannot see of a tensor whose address it gets: its type, its strides, its length, where it lies.  None and
# plain addresses are passed on as they are.

def _torch_module():
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    return _torch


def _refuse(what):
    raise MMError(MM_ERR_INVALID_ARG, what)


def _array(t, what, dtype, n, also=None):
    """Address of at least n contiguous elements of `dtype` (or `also`) on the GPU."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= n:
        return t.data_ptr()
    if t.dtype is not dtype and (also is None or t.dtype is not also):
        _refuse(f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        _refuse(f"{what} must be contiguous")
    if t.numel() < n:
        _refuse(f"{what} has {t.numel()} elements, not {n}")
    if not t.is_cuda:
        _refuse(f"{what} is not on the GPU")
    return t.data_ptr()


def _tokens(t, what, cache, tokens, row, heads):
    """Address of `tokens` rows, `row` elements apart, of heads side by side: 16-bit elements of the cache's type, or bit
    patterns of it."""
    if t is None or t.__class__ is int:
        return t
    dim, torch = cache.head_dim, _torch_module()
    n = (tokens - 1) * row + heads * dim
    if t.dtype is not (torch.bfloat16 if cache.dtype == MM_BF16 else torch.float16) and t.dtype is not torch.int16:
        _refuse(f"{what} must have the cache's type, not {t.dtype}")
    if t.is_contiguous() and t.is_cuda and t.numel() >= n:
        return t.data_ptr()
    shape, stride = t.shape, t.stride()
    if stride and stride[-1] != 1 and shape[-1] > 1 or len(shape) == 3 and shape[1] == heads > 1 and shape[2] == dim != stride[1]:
        _refuse(f"{what} must have the heads of a token side by side")
    _reach(t, what, n)
    return t.data_ptr()


def _reach(t, what, n):
    """t holds n elements from its first to its last, on the GPU."""
    if t.numel() < n and 1 + sum((a - 1) * b for a, b in zip(t.shape, t.stride())) < n:
        _refuse(f"{what} ends before the {n} elements that the call's sizes span")
    if not t.is_cuda:
        _refuse(f"{what} is not on the GPU")


def _bytes(t, what, n):
    """Address of n bytes on the GPU."""
    if t is None or t.__class__ is int:
        return t
    if not t.is_contiguous() or t.nbytes < n:
        _refuse(f"{what} must be {n} contiguous bytes")
    if not t.is_cuda:
        _refuse(f"{what} is not on the GPU")
    return t.data_ptr()


def mm_cache(k, v, table, lens, refs=None) -> Cache:
    """The description of a paged cache: k, v [layers][pages][kv_heads][page_size][head_dim] (any strides
    with contiguous rows, the same for both), table [seqs][max_pages], lens [seqs] and refs [pages] int32.
    It holds the tensors, so it is made once and kept as long as they are used."""
    if k.dim() != 5 or k.shape != v.shape or k.stride() != v.stride() or k.dtype != v.dtype or k.stride(4) != 1:
        raise ValueError("k and v must be alike, [layers][pages][kv_heads][page_size][head_dim] with contiguous rows")
    seqs, max_pages = table.shape
    _int32(table, "table", (seqs, max_pages))
    _int32(lens, "lens", (seqs,))
    if refs is not None:
        _int32(refs, "refs", (k.shape[1],))
    if not all(t.is_cuda for t in (k, v, table, lens, refs) if t is not None):
        raise ValueError("k, v, table, lens and refs must be on the GPU")
    c = Cache(k.data_ptr(), v.data_ptr(), table.data_ptr(), lens.data_ptr(), _ptr(refs), *k.shape, seqs, max_pages,
              *k.stride()[:4], _dtype(k))
    c.tensors = (k, v, table, lens, refs)
    return c


def mm_cache_reserve(cache, need, missing, stream=None):
    """Pages for lens[s] + need[s] tokens of every sequence; missing[0]: pages lacking (nothing is changed then)."""
    i32 = _torch_module().int32
    _check(load_library().mm_cache_reserve(cache, _array(need, "need", i32, cache.seqs), _array(missing, "missing", i32, 1),
                                           _stream(stream)))


def mm_cache_append(cache, layer, K, V, kv_token_stride, q_start, tokens, max_new, stream=None):
    """New tokens' keys and values [tokens][kv_heads][head_dim] into the slots behind lens."""
    heads = cache.kv_heads
    _check(load_library().mm_cache_append(cache, layer, _tokens(K, "K", cache, tokens, kv_token_stride, heads),
                                          _tokens(V, "V", cache, tokens, kv_token_stride, heads), kv_token_stride,
                                          _array(q_start, "q_start", _torch_module().int32, cache.seqs + 1), tokens,
                                          max_new, _stream(stream)))


def mm_cache_compact(cache, q_start, keep, kept, tokens, max_new, stream=None):
    """Keeps kept[s] of each sequence's new tokens (keep: which, ascending; None: the first ones), moved
    together; lens grows by kept, pages without a token are released."""
    i32, seqs = _torch_module().int32, cache.seqs
    _check(load_library().mm_cache_compact(cache, _array(q_start, "q_start", i32, seqs + 1), _array(keep, "keep", i32, tokens),
                                           _array(kept, "kept", i32, seqs), tokens, max_new, _stream(stream)))


def mm_cache_fork(cache, parents, children, n, missing, stream=None):
    """children[i] becomes a copy of parents[i]: full pages shared, the last partial page copied."""
    i32 = _torch_module().int32
    _check(load_library().mm_cache_fork(cache, _array(parents, "parents", i32, n), _array(children, "children", i32, n), n,
                                        _array(missing, "missing", i32, 1), _stream(stream)))


def mm_cache_free(cache, list, n, window=0, sinks=0, stream=None):
    """Releases the pages of sequences list[:n]: all of them, or with a window those no later query sees."""
    _check(load_library().mm_cache_free(cache, _array(list, "list", _torch_module().int32, n), n, window, sinks,
                                        _stream(stream)))


def mm_cache_copy_pages(cache, src, dst, n, stream=None):
    """Page src[i] into page dst[i], i < n, in all layers."""
    i32 = _torch_module().int32
    _check(load_library().mm_cache_copy_pages(cache, _array(src, "src", i32, n), _array(dst, "dst", i32, n), n,
                                              _stream(stream)))


def mm_cache_attention_workspace(cache, heads, tokens, max_q) -> int:
    """Bytes of workspace mm_cache_attention and _tree need for these sizes (zeroed once before its first use)."""
    out = ctypes.c_int64(0)
    _check(load_library().mm_cache_attention_workspace(cache, heads, tokens, max_q, ctypes.byref(out)))
    return out.value


def mm_cache_attention(cache, layer, Q, q_stride, heads, q_start, tokens, max_q, window, sinks, scale, O, o_stride,
                       workspace, workspace_bytes, stream=None):
    """O = attention of new tokens Q [tokens][heads][head_dim] over the cache, with a window and sinks."""
    _check(load_library().mm_cache_attention(cache, layer, _tokens(Q, "Q", cache, tokens, q_stride, heads), q_stride, heads,
                                             _array(q_start, "q_start", _torch_module().int32, cache.seqs + 1), tokens,
                                             max_q, window, sinks, scale, _tokens(O, "O", cache, tokens, o_stride, heads), o_stride,
                                             _bytes(workspace, "workspace", workspace_bytes), workspace_bytes,
                                             _stream(stream)))


def mm_cache_attention_tree(cache, layer, Q, q_stride, heads, q_start, tokens, max_q, mask, mask_words, window, sinks,
                            scale, O, o_stride, workspace, workspace_bytes, stream=None):
    """mm_cache_attention for a tree of drafted tokens: mask [tokens][mask_words], bit t: sees drafted token t."""
    torch = _torch_module()
    _check(load_library().mm_cache_attention_tree(cache, layer, _tokens(Q, "Q", cache, tokens, q_stride, heads), q_stride, heads,
                                                  _array(q_start, "q_start", torch.int32, cache.seqs + 1), tokens, max_q,
                                                  _array(mask, "mask", torch.int32, tokens * mask_words, torch.uint32),
                                                  mask_words, window, sinks, scale, _tokens(O, "O", cache, tokens, o_stride, heads),
                                                  o_stride, _bytes(workspace, "workspace", workspace_bytes),
                                                  workspace_bytes, _stream(stream)))


def mm_sample(logits, rows, vocab, stride, temperature, top_k, top_p, min_p, u, tokens, logprobs=None, stream=None):
    """tokens[r]: the next token of row r by temperature, top-k, top-p and min-p from the uniform number u[r]
    (each parameter a [rows] tensor or None: off); logprobs[r]: log of its probability among those kept."""
    dtype, torch = _dtype(logits), _torch_module()
    f32, i32 = torch.float32, torch.int32
    if not logits.is_contiguous() and logits.stride(-1) != 1 and vocab > 1:
        _refuse("the logits of a row must be contiguous")
    _reach(logits, "logits", (rows - 1) * stride + vocab)
    _check(load_library().mm_sample(logits.data_ptr(), dtype, rows, vocab, stride,
                                    _array(temperature, "temperature", f32, rows), _array(top_k, "top_k", i32, rows),
                                    _array(top_p, "top_p", f32, rows), _array(min_p, "min_p", f32, rows),
                                    _array(u, "u", f32, rows), _array(tokens, "tokens", i32, rows),
                                    _array(logprobs, "logprobs", f32, rows), _stream(stream)))
