"""Thin ctypes binding over libq4k.so (include/q4k.h, include/q4k_mx.h,
include/q4k_bench.h).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their data pointers, sizes and the current torch
stream to the C entry point of the same name, and raises on a non-zero
return code.  There is no fallback: if libq4k.so is missing the first call
raises.
"""
import ctypes
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq4k.so")

Q4K_OK = 0
Q4K_EINVAL_DIM = -1
Q4K_ENULL = -2
Q4K_EALIGN = -3
Q4K_EHIP = -4
Q4K_ESCRATCH = -5
Q4K_EINVAL_TYPE = -6

# Value types and block formats of the MX operators (include/q4k_mx.h).
MX_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
MX_FORMAT = {"fp4": 4, "fp8": 8}
ROTARY_LAYOUT = {"half": 0, "interleaved": 1}
ROTARY_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

EXPORTED = (
    "q4k_gemv", "q4k_matmul", "ternary_gemv_codes", "ternary_gemv", "ternary_matmul",
    "q4k_gemv_shaped", "q4k_gemv_walk_shaped", "q4_0_gemv", "q4_0_gemv_shaped", "q6k_gemv",
    "q6k_gemv_shaped",
    "q4k_tiled_size", "q4k_relayout_tiled", "q4k_gemv_tiled", "q4k_gemv_tiled_shaped",
    "q4k_matmul_tiled", "q4k_matmul_shaped", "q4k_matmul_tiled_shaped", "ternary_matmul_shaped",
    "q4k_matmul_noalloc",
    "q4k_strerror",
    "mx_quantize", "mx_dequantize", "mx_rmsnorm", "mxfp4_matmul", "mxfp4_moe_workspace_size",
    "mxfp4_moe",
    "mx_rotary", "mx_rotary_frequencies", "mx_cache_write", "mx_cache_read",
    "mx_attention_workspace_size", "mx_attention",
    "q4k_bench_empty", "q4k_bench_delay", "q4k_bench_stream_read", "q4k_bench_copy",
)

_lib = None


class Q4KError(ValueError):
    """A non-zero return code from libq4k.so."""

    def __init__(self, code, func):
        msg = lib().q4k_strerror(code).decode()
        super().__init__(f"{func}: {msg} (code {code})")
        self.code = code


def lib():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is not built: run `python -m q4_packed_weight_amd.build` "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(LIB_PATH)
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    DBL = ctypes.c_double
    sig = {
        "q4k_gemv": [P, P, I64, I64, P, P],
        "q4k_matmul": [P, P, I64, I64, I64, P, P],
        "q4k_matmul_noalloc": [P, P, I64, I64, I64, P, P],
        "ternary_gemv_codes": [P, P, I64, I64, P, P],
        "ternary_gemv": [P, P, F, I64, I64, P, P],
        "ternary_matmul": [P, P, F, I64, I64, I64, P, P],
        "ternary_matmul_shaped": [P, P, F, I64, I64, I64, P, P, I],
        "q4k_gemv_shaped": [P, P, I64, I64, P, P, I, I, I],
        "q4_0_gemv": [P, P, I64, I64, P, P],
        "q4_0_gemv_shaped": [P, P, I64, I64, P, P, I, I, I],
        "q6k_gemv": [P, P, I64, I64, P, P],
        "q6k_gemv_shaped": [P, P, I64, I64, P, P, I, I, I],
        "q4k_relayout_tiled": [P, I64, I64, P, P],
        "q4k_gemv_tiled": [P, P, I64, I64, P, P],
        "q4k_gemv_tiled_shaped": [P, P, I64, I64, P, P, I, I, I],
        "q4k_gemv_walk_shaped": [P, P, I64, I64, P, P, I, I, I],
        "q4k_matmul_tiled": [P, P, I64, I64, I64, P, P],
        "q4k_matmul_shaped": [P, P, I64, I64, I64, P, P, I],
        "q4k_matmul_tiled_shaped": [P, P, I64, I64, I64, P, P, I],
        "mx_quantize": [P, I, I, I64, I64, P, P, P],
        "mx_dequantize": [P, P, I, I64, I64, P, I, P],
        "mx_rmsnorm": [P, P, P, F, I, I64, I64, P, P, I, P, P, P],
        "mxfp4_matmul": [P, P, I, P, P, I64, I64, I64, P, I, P],
        "mxfp4_moe": [P, I, P, P, P, P, P, P, I64, I64, I64, I64, I64, P, P, I64, P],
        "mx_rotary": [P, I64, I, P, P, F, I64, I64, I64, I64, I, P, I64, P],
        "mx_rotary_frequencies": [I64, DBL, I, DBL, DBL, DBL, DBL, P, P],
        "mx_cache_write": [P, I64, P, I64, I, P, I64, I64, I64, I, P, P, P, P, I64, I64, P],
        "mx_cache_read": [P, I64, I64, I64, I, P, P, P, P, I64, I64, P, I64, P, I64, I, P],
        "mx_attention": [P, I64, I, P, P, P, I64, I64, I64, I64, I64, I64, I64, F, I, I64, I, P, P,
                         P, P, I64, I64, P, I64, P, I64, P],
        "q4k_bench_empty": [P],
        "q4k_bench_delay": [I64, P],
        "q4k_bench_stream_read": [P, I64, P, I64, P],
        "q4k_bench_copy": [P, P, I64, P],
    }
    for name, args in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = I
    L.q4k_tiled_size.argtypes = [I64, I64]
    L.q4k_tiled_size.restype = I64
    L.mxfp4_moe_workspace_size.argtypes = [I64, I64, I64, I64, I64]
    L.mxfp4_moe_workspace_size.restype = I64
    L.mx_attention_workspace_size.argtypes = [I64] * 8
    L.mx_attention_workspace_size.restype = I64
    L.q4k_strerror.argtypes = [I]
    L.q4k_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's handle without a Stream object around it, which takes
# longer to make than everything else here; a torch built without a GPU lacks
# these names, and its public call says so.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None or _current_device is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_current_device())


def _check(rc, func):
    if rc != Q4K_OK:
        raise Q4KError(rc, func)


def _expect(t, dtype, name, need=0):
    """Type/layout/size marshalling check; `need` is the element count the
    dimensions imply (0 = not checked here, the C side validates dims)."""
    if t is None:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if need > 0 and t.numel() < need:
        raise ValueError(f"{name} has {t.numel()} elements, the dimensions need {need}")


def _q4k_need(K, N):
    return N * (K // 256) * 144 if (K > 0 and N > 0 and K % 256 == 0) else 0


def _pos(*v):
    return all(int(a) > 0 for a in v)


def q4k_gemv(x, w_blocks, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4k_gemv(_ptr(x), _ptr(w_blocks), int(input_dim), int(output_dim),
                          _ptr(y), _stream(stream)), "q4k_gemv")
    return y


def q4k_gemv_shaped(x, w_blocks, input_dim, output_dim, y, rows_per_lane=0,
                    k_waves=0, workgroup_waves=0, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4k_gemv_shaped(_ptr(x), _ptr(w_blocks), int(input_dim),
                                 int(output_dim), _ptr(y), _stream(stream),
                                 int(rows_per_lane), int(k_waves), int(workgroup_waves)),
           "q4k_gemv_shaped")
    return y


def q4k_matmul(X, w_blocks, n_tokens, input_dim, output_dim, Y, stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    ok = _pos(M, K, N)
    _expect(X, torch.float32, "X", M * K if ok else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N) if ok else 0)
    _expect(Y, torch.float32, "Y", M * N if ok else 0)
    _check(lib().q4k_matmul(_ptr(X), _ptr(w_blocks), int(n_tokens), int(input_dim),
                            int(output_dim), _ptr(Y), _stream(stream)), "q4k_matmul")
    return Y


def q4k_matmul_noalloc(X, w_blocks, n_tokens, input_dim, output_dim, Y, stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    ok = _pos(M, K, N)
    _expect(X, torch.float32, "X", M * K if ok else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N) if ok else 0)
    _expect(Y, torch.float32, "Y", M * N if ok else 0)
    _check(lib().q4k_matmul_noalloc(_ptr(X), _ptr(w_blocks), M, K, N, _ptr(Y), _stream(stream)),
           "q4k_matmul_noalloc")
    return Y


def _q4_0_need(K, N):
    return N * (K // 32) * 18 if (K > 0 and N > 0 and K % 32 == 0) else 0


def q4_0_gemv(x, w_blocks, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4_0_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4_0_gemv(_ptr(x), _ptr(w_blocks), K, N, _ptr(y), _stream(stream)),
           "q4_0_gemv")
    return y


def q4_0_gemv_shaped(x, w_blocks, input_dim, output_dim, y, rows_per_lane=0,
                     k_waves=0, workgroup_waves=0, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4_0_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4_0_gemv_shaped(_ptr(x), _ptr(w_blocks), K, N, _ptr(y), _stream(stream),
                                  int(rows_per_lane), int(k_waves), int(workgroup_waves)),
           "q4_0_gemv_shaped")
    return y


def q4k_tiled_size(input_dim, output_dim):
    """Bytes of the tiled order (raises on invalid dimensions)."""
    n = lib().q4k_tiled_size(int(input_dim), int(output_dim))
    _check(n if n < 0 else Q4K_OK, "q4k_tiled_size")
    return n


def _tiled_need(K, N):
    return ((N + 15) // 16) * (K // 256) * 2304 if (K > 0 and N > 0 and K % 256 == 0) else 0


def q4k_relayout_tiled(w_blocks, input_dim, output_dim, w_tiled, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N))
    _expect(w_tiled, torch.uint8, "w_tiled", _tiled_need(K, N))
    _check(lib().q4k_relayout_tiled(_ptr(w_blocks), K, N, _ptr(w_tiled), _stream(stream)),
           "q4k_relayout_tiled")
    return w_tiled


def q4k_gemv_tiled(x, w_tiled, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_tiled, torch.uint8, "w_tiled", _tiled_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4k_gemv_tiled(_ptr(x), _ptr(w_tiled), K, N, _ptr(y), _stream(stream)),
           "q4k_gemv_tiled")
    return y


def q4k_matmul_shaped(X, w_blocks, n_tokens, input_dim, output_dim, Y, form=0, stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    _expect(X, torch.float32, "X", M * K if _pos(M, K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N))
    _expect(Y, torch.float32, "Y", M * N if _pos(M, K, N) else 0)
    _check(lib().q4k_matmul_shaped(_ptr(X), _ptr(w_blocks), M, K, N, _ptr(Y), _stream(stream),
                                   int(form)), "q4k_matmul_shaped")
    return Y


def q4k_matmul_tiled(X, w_tiled, n_tokens, input_dim, output_dim, Y, stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    _expect(X, torch.float32, "X", M * K if _pos(M, K, N) else 0)
    _expect(w_tiled, torch.uint8, "w_tiled", _tiled_need(K, N))
    _expect(Y, torch.float32, "Y", M * N if _pos(M, K, N) else 0)
    _check(lib().q4k_matmul_tiled(_ptr(X), _ptr(w_tiled), M, K, N, _ptr(Y), _stream(stream)),
           "q4k_matmul_tiled")
    return Y


def q4k_matmul_tiled_shaped(X, w_tiled, n_tokens, input_dim, output_dim, Y, form=0,
                            stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    _expect(X, torch.float32, "X", M * K if _pos(M, K, N) else 0)
    _expect(w_tiled, torch.uint8, "w_tiled", _tiled_need(K, N))
    _expect(Y, torch.float32, "Y", M * N if _pos(M, K, N) else 0)
    _check(lib().q4k_matmul_tiled_shaped(_ptr(X), _ptr(w_tiled), M, K, N, _ptr(Y),
                                         _stream(stream), int(form)),
           "q4k_matmul_tiled_shaped")
    return Y


def q4k_gemv_walk_shaped(x, w_blocks, input_dim, output_dim, y, waves=0, row_groups=0,
                         depth=0, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q4k_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4k_gemv_walk_shaped(_ptr(x), _ptr(w_blocks), K, N, _ptr(y), _stream(stream),
                                      int(waves), int(row_groups), int(depth)),
           "q4k_gemv_walk_shaped")
    return y


def q4k_gemv_tiled_shaped(x, w_tiled, input_dim, output_dim, y, waves=0, row_groups=0,
                          depth=0, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_tiled, torch.uint8, "w_tiled", _tiled_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q4k_gemv_tiled_shaped(_ptr(x), _ptr(w_tiled), K, N, _ptr(y), _stream(stream),
                                       int(waves), int(row_groups), int(depth)),
           "q4k_gemv_tiled_shaped")
    return y


def _q6k_need(K, N):
    return N * (K // 256) * 210 if (K > 0 and N > 0 and K % 256 == 0) else 0


def q6k_gemv(x, w_blocks, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q6k_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q6k_gemv(_ptr(x), _ptr(w_blocks), K, N, _ptr(y), _stream(stream)),
           "q6k_gemv")
    return y


def q6k_gemv_shaped(x, w_blocks, input_dim, output_dim, y, rows_per_lane=0,
                    k_waves=0, workgroup_waves=0, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _pos(K, N) else 0)
    _expect(w_blocks, torch.uint8, "w_blocks", _q6k_need(K, N))
    _expect(y, torch.float32, "y", N if _pos(K, N) else 0)
    _check(lib().q6k_gemv_shaped(_ptr(x), _ptr(w_blocks), K, N, _ptr(y), _stream(stream),
                                 int(rows_per_lane), int(k_waves), int(workgroup_waves)),
           "q6k_gemv_shaped")
    return y


def _ternary_need(K, N):
    return N * (K // 4) if (K > 0 and N > 0 and K % 4 == 0) else 0


def ternary_gemv_codes(x, codes, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _ternary_need(K, N) else 0)
    _expect(codes, torch.uint8, "codes", _ternary_need(K, N))
    _expect(y, torch.float32, "y", N if _ternary_need(K, N) else 0)
    _check(lib().ternary_gemv_codes(_ptr(x), _ptr(codes), int(input_dim),
                                    int(output_dim), _ptr(y), _stream(stream)),
           "ternary_gemv_codes")
    return y


def ternary_gemv(x, codes, scale, input_dim, output_dim, y, stream=None):
    K, N = int(input_dim), int(output_dim)
    _expect(x, torch.float32, "x", K if _ternary_need(K, N) else 0)
    _expect(codes, torch.uint8, "codes", _ternary_need(K, N))
    _expect(y, torch.float32, "y", N if _ternary_need(K, N) else 0)
    _check(lib().ternary_gemv(_ptr(x), _ptr(codes), float(scale), int(input_dim),
                              int(output_dim), _ptr(y), _stream(stream)), "ternary_gemv")
    return y


def ternary_matmul(X, codes, scale, n_tokens, input_dim, output_dim, Y, stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    ok = M > 0 and _ternary_need(K, N) > 0
    _expect(X, torch.float32, "X", M * K if ok else 0)
    _expect(codes, torch.uint8, "codes", _ternary_need(K, N))
    _expect(Y, torch.float32, "Y", M * N if ok else 0)
    _check(lib().ternary_matmul(_ptr(X), _ptr(codes), float(scale), M, K, N, _ptr(Y),
                                _stream(stream)), "ternary_matmul")
    return Y


def ternary_matmul_shaped(X, codes, scale, n_tokens, input_dim, output_dim, Y, form=0,
                          stream=None):
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    ok = M > 0 and _ternary_need(K, N) > 0
    _expect(X, torch.float32, "X", M * K if ok else 0)
    _expect(codes, torch.uint8, "codes", _ternary_need(K, N))
    _expect(Y, torch.float32, "Y", M * N if ok else 0)
    _check(lib().ternary_matmul_shaped(_ptr(X), _ptr(codes), float(scale), M, K, N, _ptr(Y),
                                       _stream(stream), int(form)), "ternary_matmul_shaped")
    return Y


def _mx_type(t, name):
    if t is None:
        raise ValueError(f"{name} is required")
    code = MX_TYPE.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _mx_format(fmt):
    code = MX_FORMAT.get(fmt)
    if code is None:
        raise ValueError(f"MX format must be 'fp4' or 'fp8', got {fmt!r}")
    return code


def _arg(t, dtype, name, need):
    """The pointer of a tensor that passes _expect's checks."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.is_contiguous() and t.is_cuda and t.numel() >= need):
        _expect(t, dtype, name, need)
    return t.data_ptr()


def _mx_need(rows, K):
    """Values of a matrix in MX blocks (0 where the C side refuses the sizes)."""
    return rows * K if rows > 0 and K > 0 and K % 32 == 0 else 0


def mx_quantize(x, n_rows, input_dim, fmt, codes, scales, stream=None):
    """Rows of x (fp32, bf16 or fp16) to MX blocks; fmt is "fp4" or "fp8"."""
    R, K = int(n_rows), int(input_dim)
    t, f, n = _mx_type(x, "x"), _mx_format(fmt), _mx_need(R, K)
    rc = lib().mx_quantize(_arg(x, x.dtype, "x", n), t, f, R, K,
                           _arg(codes, torch.uint8, "codes", n * f // 8),
                           _arg(scales, torch.uint8, "scales", n // 32), _stream(stream))
    _check(rc, "mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, n_rows, input_dim, fmt, y, stream=None):
    """The values of MX blocks, rounded to y's type."""
    R, K = int(n_rows), int(input_dim)
    t, f, n = _mx_type(y, "y"), _mx_format(fmt), _mx_need(R, K)
    rc = lib().mx_dequantize(_arg(codes, torch.uint8, "codes", n * f // 8),
                             _arg(scales, torch.uint8, "scales", n // 32), f, R, K,
                             _arg(y, y.dtype, "y", n), t, _stream(stream))
    _check(rc, "mx_dequantize")
    return y


def mx_rmsnorm(x, residual, weight, eps, n_rows, input_dim, fmt, residual_out, y, codes, scales,
               stream=None):
    """Residual addition and RMS norm with MX blocks out; residual,
    residual_out, y, and codes with scales (fmt then unused) may be None."""
    R, K = int(n_rows), int(input_dim)
    t, n = _mx_type(x, "x"), _mx_need(R, K)
    f = _mx_format(fmt) if codes is not None or scales is not None else 0
    d = x.dtype
    rc = lib().mx_rmsnorm(_arg(x, d, "x", n), _arg(residual, d, "residual", n),
                          _arg(weight, d, "weight", K if n else 0), float(eps), t, R, K,
                          _arg(residual_out, d, "residual_out", n), _arg(y, d, "y", n), f,
                          _arg(codes, torch.uint8, "codes", n * f // 8),
                          _arg(scales, torch.uint8, "scales", n // 32), _stream(stream))
    _check(rc, "mx_rmsnorm")
    return codes, scales


def mxfp4_matmul(a_codes, a_scales, a_fmt, w_codes, w_scales, n_tokens, input_dim, output_dim, Y,
                 stream=None):
    """Y = A W^T of MX activations (a_fmt "fp8" or "fp4") and MXFP4 weights."""
    M, K, N = int(n_tokens), int(input_dim), int(output_dim)
    t, f, a, w = _mx_type(Y, "Y"), _mx_format(a_fmt), _mx_need(M, K), _mx_need(N, K)
    rc = lib().mxfp4_matmul(_arg(a_codes, torch.uint8, "a_codes", a * f // 8),
                            _arg(a_scales, torch.uint8, "a_scales", a // 32), f,
                            _arg(w_codes, torch.uint8, "w_codes", w // 2),
                            _arg(w_scales, torch.uint8, "w_scales", w // 32), M, K, N,
                            _arg(Y, Y.dtype, "Y", M * N if a and w else 0), t, _stream(stream))
    _check(rc, "mxfp4_matmul")
    return Y


def mxfp4_moe_workspace_size(n_tokens, input_dim, ffn_dim, n_experts, top_k):
    """Bytes of mxfp4_moe's workspace (raises on invalid dimensions)."""
    n = lib().mxfp4_moe_workspace_size(int(n_tokens), int(input_dim), int(ffn_dim),
                                       int(n_experts), int(top_k))
    _check(n if n < 0 else Q4K_OK, "mxfp4_moe_workspace_size")
    return n


def mxfp4_moe(x, router, router_bias, up_codes, up_scales, down_codes, down_scales, n_tokens,
              input_dim, ffn_dim, n_experts, top_k, y, workspace, stream=None):
    """A mixture-of-experts layer with MXFP4 experts; router_bias may be None."""
    T, H, F, E, k = int(n_tokens), int(input_dim), int(ffn_dim), int(n_experts), int(top_k)
    t, d, u8 = _mx_type(x, "x"), x.dtype, torch.uint8
    n = _mx_need(T, H)
    up = _mx_need(E * 2 * F, H) if F > 0 else 0
    down = _mx_need(E * H, F) if H > 0 else 0
    rc = lib().mxfp4_moe(_arg(x, d, "x", n), t, _arg(router, d, "router", _mx_need(E, H)),
                         _arg(router_bias, torch.float32, "router_bias", max(E, 0)),
                         _arg(up_codes, u8, "up_codes", up // 2),
                         _arg(up_scales, u8, "up_scales", up // 32),
                         _arg(down_codes, u8, "down_codes", down // 2),
                         _arg(down_scales, u8, "down_scales", down // 32), T, H, F, E, k,
                         _arg(y, d, "y", n), _arg(workspace, u8, "workspace", 0),
                         0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, "mxfp4_moe")
    return y


def _choice(table, key, name):
    code = table.get(key)
    if code is None:
        raise ValueError(f"{name} must be one of {', '.join(table)}, got {key!r}")
    return code


_device = torch.cuda.current_device if _current_device is None else _current_device


def _here(t):
    """The current device, not asked for where t needs none to be refused."""
    return _device() if t.is_cuda else None


def _elsewhere(t, name, here):
    if t.get_device() != here:
        raise ValueError(f"{name} is on {t.device}, the current device is another")


def _local(t, dtype, name, need, here):
    """_arg for a tensor that has to be on device `here`: pools, tables and positions
    are read where the kernels run."""
    if t is None:
        return None
    if not (t.dtype is dtype and t.is_contiguous() and t.get_device() == here
            and t.numel() >= need):
        _expect(t, dtype, name, need)
        _elsewhere(t, name, here)
    return t.data_ptr()


def _rows(t, dtype, name, rows, heads, head_dim, here):
    """(pointer, values from a row to the next) of [rows][heads * head_dim] or
    [rows][heads][head_dim] values; rows may lie apart, as slices of a wider
    matrix do."""
    width = heads * head_dim
    if t is None:
        return None, width
    shape = t.shape
    if (t.dtype is dtype and t.get_device() == here and t.is_contiguous() and rows > 0 and width > 0
            and (shape == (rows, width) or shape == (rows, heads, head_dim))):
        return t.data_ptr(), width
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    _elsewhere(t, name, here)
    stride = t.stride()
    if rows <= 0 or width <= 0:  # refused by the C side
        return t.data_ptr(), width
    if shape == (rows, width):
        whole = width == 1 or stride[1] == 1
    elif shape == (rows, heads, head_dim):
        whole = (head_dim == 1 or stride[2] == 1) and (heads == 1 or stride[1] == head_dim)
    else:
        raise ValueError(f"{name} must be [{rows}][{width}] or [{rows}][{heads}][{head_dim}], "
                         f"got {list(shape)}")
    if not whole:
        raise ValueError(f"{name}: a row's values must lie one after the other")
    return t.data_ptr(), stride[0] if rows > 1 else width


def mx_rotary(x, positions, frequencies, amplitude, n_tokens, n_heads, head_dim, rotary_dim,
              layout, y, stream=None):
    """Rotary positions; layout is "half" or "interleaved", y may be x."""
    T, H, D, R = int(n_tokens), int(n_heads), int(head_dim), int(rotary_dim)
    t, here, lay = _mx_type(x, "x"), _here(x), _choice(ROTARY_LAYOUT, layout, "layout")
    xp, xs = _rows(x, x.dtype, "x", T, H, D, here)
    yp, ys = _rows(y, x.dtype, "y", T, H, D, here)
    rc = lib().mx_rotary(xp, xs, t, _local(positions, torch.int64, "positions", max(T, 0), here),
                         _local(frequencies, torch.float64, "frequencies", max(R // 2, 0), here),
                         float(amplitude), T, H, D, R, lay, yp, ys, _stream(stream))
    _check(rc, "mx_rotary")
    return y


def mx_rotary_frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, trained=8192.0,
                          low=1.0, high=None):
    """(fp64 tensor on the host of rotary_dim / 2 frequencies, amplitude); the
    scaling is "none", "linear", "ntk", "yarn" or "bands".  Without `high` bands end
    at 4 turns and YaRN's ramp at 32, as models trained with them have it."""
    if high is None:
        high = 4.0 if scaling == "bands" else 32.0
    n = int(rotary_dim)
    # a size that the C side refuses gets no table
    f = torch.zeros(n // 2 if 0 < n <= 512 else 0, dtype=torch.float64)
    amplitude = ctypes.c_double(1.0)
    rc = lib().mx_rotary_frequencies(n, float(base), _choice(ROTARY_SCALING, scaling, "scaling"),
                                     float(factor), float(trained), float(low), float(high),
                                     f.data_ptr(), ctypes.addressof(amplitude))
    _check(rc, "mx_rotary_frequencies")
    return f, amplitude.value


def _pool(k_codes, k_scales, v_codes, v_scales, n_pages, page_size, heads, head_dim, f, here):
    n = _mx_need(n_pages * heads * page_size, head_dim) if heads > 0 and page_size > 0 else 0
    return [_local(t, torch.uint8, name, need, here) for t, name, need in (
        (k_codes, "k_codes", n * f // 8), (k_scales, "k_scales", n // 32),
        (v_codes, "v_codes", n * f // 8), (v_scales, "v_scales", n // 32))]


def mx_cache_write(k, v, slots, n_tokens, n_heads, head_dim, fmt, k_codes, k_scales, v_codes,
                   v_scales, n_pages, page_size, stream=None):
    """Rows of keys and values to the blocks of their slots; -1 leaves a token out."""
    T, H, D, N, B = int(n_tokens), int(n_heads), int(head_dim), int(n_pages), int(page_size)
    t, f, here = _mx_type(k, "k"), _mx_format(fmt), _here(k)
    kp, ks = _rows(k, k.dtype, "k", T, H, D, here)
    vp, vs = _rows(v, k.dtype, "v", T, H, D, here)
    pool = _pool(k_codes, k_scales, v_codes, v_scales, N, B, H, D, f, here)
    rc = lib().mx_cache_write(kp, ks, vp, vs, t,
                              _local(slots, torch.int64, "slots", max(T, 0), here), T, H, D, f,
                              *pool, N, B, _stream(stream))
    _check(rc, "mx_cache_write")


def mx_cache_read(slots, n_tokens, n_heads, head_dim, fmt, k_codes, k_scales, v_codes, v_scales,
                  n_pages, page_size, k, v, stream=None):
    """The values of slots, rounded to k's and v's type; -1 reads as zeros."""
    T, H, D, N, B = int(n_tokens), int(n_heads), int(head_dim), int(n_pages), int(page_size)
    t, f, here = _mx_type(k, "k"), _mx_format(fmt), _here(k)
    kp, ks = _rows(k, k.dtype, "k", T, H, D, here)
    vp, vs = _rows(v, k.dtype, "v", T, H, D, here)
    pool = _pool(k_codes, k_scales, v_codes, v_scales, N, B, H, D, f, here)
    rc = lib().mx_cache_read(_local(slots, torch.int64, "slots", max(T, 0), here), T, H, D, f,
                             *pool, N, B, kp, ks, vp, vs, t, _stream(stream))
    _check(rc, "mx_cache_read")
    return k, v


def mx_attention_workspace_size(n_tokens, n_heads, n_kv_heads, head_dim, n_seqs, pages_per_seq,
                                page_size, max_queries):
    """Bytes of mx_attention's workspace (raises on invalid dimensions)."""
    n = lib().mx_attention_workspace_size(int(n_tokens), int(n_heads), int(n_kv_heads),
                                          int(head_dim), int(n_seqs), int(pages_per_seq),
                                          int(page_size), int(max_queries))
    _check(n if n < 0 else Q4K_OK, "mx_attention_workspace_size")
    return n


def mx_attention(q, query_starts, key_counts, pages, n_tokens, n_heads, n_kv_heads, head_dim,
                 n_seqs, pages_per_seq, max_queries, scale, causal, window, fmt, k_codes, k_scales,
                 v_codes, v_scales, n_pages, page_size, y, workspace, stream=None):
    """Attention of sequences' new tokens over their cached keys and values;
    workspace may be None where mx_attention_workspace_size gives 0."""
    T, H, HK, D = int(n_tokens), int(n_heads), int(n_kv_heads), int(head_dim)
    S, P, N, B = int(n_seqs), int(pages_per_seq), int(n_pages), int(page_size)
    t, f, i32, here = _mx_type(q, "q"), _mx_format(fmt), torch.int32, _here(q)
    qp, qs = _rows(q, q.dtype, "q", T, H, D, here)
    yp, ys = _rows(y, q.dtype, "y", T, H, D, here)
    pool = _pool(k_codes, k_scales, v_codes, v_scales, N, B, HK, D, f, here)
    rc = lib().mx_attention(qp, qs, t,
                            _local(query_starts, i32, "query_starts", max(S + 1, 0), here),
                            _local(key_counts, i32, "key_counts", max(S, 0), here),
                            _local(pages, i32, "pages", max(S, 0) * max(P, 0), here), T, H, HK, D,
                            S, P, int(max_queries), float(scale), int(bool(causal)), int(window),
                            f, *pool, N, B, yp, ys,
                            _local(workspace, torch.uint8, "workspace", 0, here),
                            0 if workspace is None else workspace.numel(), _stream(stream))
    _check(rc, "mx_attention")
    return y


def bench_empty(stream=None):
    _check(lib().q4k_bench_empty(_stream(stream)), "q4k_bench_empty")


def bench_delay(ns, stream=None):
    _check(lib().q4k_bench_delay(int(ns), _stream(stream)), "q4k_bench_delay")


def bench_stream_read(src, sink, stream=None):
    _expect(sink, torch.int32, "sink")
    _check(lib().q4k_bench_stream_read(_ptr(src), src.numel() * src.element_size(),
                                       _ptr(sink), sink.numel(), _stream(stream)),
           "q4k_bench_stream_read")


def bench_copy(src, dst, stream=None):
    n = src.numel() * src.element_size()
    assert dst.numel() * dst.element_size() >= n
    _check(lib().q4k_bench_copy(_ptr(src), _ptr(dst), n, _stream(stream)),
           "q4k_bench_copy")
