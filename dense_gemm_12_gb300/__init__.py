"""dense_gemm_12_gb300 -- GB300 (sm_103a) dense GEMM, C <- alpha*(A x B) + beta*C.

Python binding of the C ABI in ``include/gemm12.h`` (``libgemm12.so``).  The
functions named like the C entry points take the same arguments (device
pointers as integers, a stream handle as an integer) and only marshal them;
every step of the GEMM runs in the library's CUDA kernels.  The tensor
helpers ``sgemm`` / ``bf16gemm`` derive pointers, leading dimensions and the
current stream from torch tensors and call the same entry points.

There is no fallback: if the compiled library is missing, loading fails with
an error that says how to build it.
"""
from __future__ import annotations

import ctypes
import os
import threading

from . import _build

__all__ = [
    "GemmError", "load_library", "library_path", "gemm_sgemm", "gemm_bf16gemm",
    "gemm_bf16gemm_decode_static", "gemm_bf16gemm_epilogue", "bf16gemm_epilogue", "ACT", "OUT",
    "gemm_bf16gemm_fused", "bf16gemm_fused", "GemmOutput",
    "gemm_sgemm_config", "gemm_bf16gemm_config", "gemm_get_config", "gemm_get_model_config",
    "GemmConfig", "KERNELS", "SPLIT_STREAM",
    "gemm_status_string", "gemm_check_device_error", "gemm_shutdown", "gemm_release_stream",
    "gemm_select_path", "gemm_split_parts", "gemm_split_cluster", "gemm_quantization", "gemm_version", "sgemm", "bf16gemm",
    "STATUS", "PATHS",
    "RmsnormArgs", "RmsnormGradArgs", "BLOCK", "gemm_rmsnorm", "gemm_rmsnorm_backward",
    "gemm_fp8_quantize", "gemm_fp8gemm", "gemm_fp8gemm_grouped", "gemm_bf16gemm_grouped",
    "gemm_bf16gemm_grouped_wgrad", "rmsnorm", "rmsnorm_backward", "fp8_quantize", "fp8gemm",
    "fp8gemm_grouped", "bf16gemm_grouped", "bf16gemm_grouped_wgrad",
]

STATUS = {
    0: "GEMM_OK", 1: "GEMM_ERR_INVALID_VALUE", 2: "GEMM_ERR_MISALIGNED",
    3: "GEMM_ERR_UNSUPPORTED", 4: "GEMM_ERR_LAUNCH", 5: "GEMM_ERR_DEVICE_TIMEOUT",
    6: "GEMM_ERR_NO_MEMORY",
}
PATHS = {
    0: "none", 1: "scale_c", 2: "simt_tma", 3: "simt_generic", 4: "tc_bf16",
    5: "tc_decode", 6: "simt_bf16", 7: "tc_bf16_pair", 8: "simt_staged", 9: "tc_staged",
}


class GemmError(RuntimeError):
    """A C-ABI call returned a status other than GEMM_OK."""

    def __init__(self, status: int, where: str):
        self.status = int(status)
        super().__init__("%s: %s" % (where, gemm_status_string(status)))


class GemmOutput(ctypes.Structure):
    """Mirror of gemm_output_t (include/gemm12.h)."""
    _fields_ = [
        ("beta", ctypes.c_float), ("C", ctypes.c_void_p), ("ldc", ctypes.c_int64),
        ("bias", ctypes.c_void_p), ("act", ctypes.c_int),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("d_scale", ctypes.c_float), ("amax", ctypes.c_void_p),
        ("D", ctypes.c_void_p), ("ldd", ctypes.c_int64), ("d_type", ctypes.c_int),
    ]


class GemmConfig(ctypes.Structure):
    """Mirror of gemm_config_t (include/gemm12.h)."""
    _fields_ = [("kernel", ctypes.c_int), ("split", ctypes.c_int), ("group_m", ctypes.c_int)]


class RmsnormArgs(ctypes.Structure):
    """Mirror of gemm_rmsnorm_t (include/gemm12.h)."""
    _fields_ = [
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64), ("x_type", ctypes.c_int),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64), ("residual_type", ctypes.c_int),
        ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("h_type", ctypes.c_int),
        ("weight", ctypes.c_void_p), ("eps", ctypes.c_float),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64), ("y_type", ctypes.c_int),
        ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64),
        ("scales", ctypes.c_void_p), ("ld_scales", ctypes.c_int64), ("rstd", ctypes.c_void_p),
    ]


class RmsnormGradArgs(ctypes.Structure):
    """Mirror of gemm_rmsnorm_grad_t (include/gemm12.h)."""
    _fields_ = [
        ("dy", ctypes.c_void_p), ("lddy", ctypes.c_int64), ("dy_type", ctypes.c_int),
        ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64), ("h_type", ctypes.c_int),
        ("weight", ctypes.c_void_p), ("rstd", ctypes.c_void_p),
        ("residual_grad", ctypes.c_void_p), ("ldrg", ctypes.c_int64),
        ("residual_grad_type", ctypes.c_int),
        ("dh", ctypes.c_void_p), ("lddh", ctypes.c_int64), ("dh_type", ctypes.c_int),
        ("dweight", ctypes.c_void_p),
    ]


KERNELS = {"auto": 0, "single_cta": 1, "cta_pair": 2, "wide": 3}
# gemm_config_t.split value for the stream-K tail (fp32 only): GEMM_SPLIT_STREAM.
SPLIT_STREAM = -1


class _Quantization(ctypes.Structure):
    _fields_ = [
        ("tiles_m", ctypes.c_int64), ("tiles_n", ctypes.c_int64), ("tiles", ctypes.c_int64),
        ("covered_m", ctypes.c_int64), ("covered_n", ctypes.c_int64),
        ("useful_fraction", ctypes.c_double), ("per_wave", ctypes.c_int64),
        ("waves", ctypes.c_int64), ("wave_efficiency", ctypes.c_double),
    ]


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load_library(build_if_missing: bool = False):
    """Load libgemm12.so (optionally compiling it first) and declare signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if build_if_missing:
            path = _build.build()
        if not os.path.exists(path):
            raise RuntimeError(
                "libgemm12.so is not built (expected at %s); run "
                "`python -c 'import __graft_entry__ as g; g.build()'`" % path)
        lib = ctypes.CDLL(path)
        i64, f32, vp, cint = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
        gemm_args = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, vp]
        lib.gemm_sgemm.argtypes = gemm_args
        lib.gemm_sgemm.restype = cint
        lib.gemm_bf16gemm.argtypes = gemm_args
        lib.gemm_bf16gemm.restype = cint
        lib.gemm_bf16gemm_decode_static.argtypes = gemm_args
        lib.gemm_bf16gemm_decode_static.restype = cint
        lib.gemm_bf16gemm_epilogue.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64,
                                               vp, cint, vp, i64, cint, vp]
        lib.gemm_bf16gemm_epilogue.restype = cint
        lib.gemm_bf16gemm_fused.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64,
                                            ctypes.POINTER(GemmOutput), vp]
        lib.gemm_bf16gemm_fused.restype = cint
        cfg_p = ctypes.POINTER(GemmConfig)
        lib.gemm_sgemm_config.argtypes = gemm_args[:-1] + [cfg_p, vp]
        lib.gemm_sgemm_config.restype = cint
        lib.gemm_bf16gemm_config.argtypes = gemm_args[:-1] + [cfg_p, vp]
        lib.gemm_bf16gemm_config.restype = cint
        lib.gemm_get_config.argtypes = [cint, i64, i64, i64, cfg_p, ctypes.POINTER(cint)]
        lib.gemm_get_config.restype = cint
        lib.gemm_get_model_config.argtypes = [cint, i64, i64, i64, cfg_p]
        lib.gemm_get_model_config.restype = cint
        lib.gemm_status_string.argtypes = [cint]
        lib.gemm_status_string.restype = ctypes.c_char_p
        lib.gemm_check_device_error.argtypes = [vp]
        lib.gemm_check_device_error.restype = cint
        lib.gemm_shutdown.argtypes = []
        lib.gemm_shutdown.restype = cint
        lib.gemm_release_stream.argtypes = [vp]
        lib.gemm_release_stream.restype = cint
        lib.gemm_select_path.argtypes = [cint, i64, i64, i64, f32, vp, i64, vp, i64]
        lib.gemm_select_path.restype = cint
        lib.gemm_quantization.argtypes = [i64, i64, i64, i64, i64, i64,
                                          ctypes.POINTER(_Quantization)]
        lib.gemm_quantization.restype = cint
        lib.gemm_split_parts.argtypes = [cint, i64, i64, i64]
        lib.gemm_split_parts.restype = cint
        lib.gemm_split_cluster.argtypes = [cint, i64, i64, i64, cfg_p]
        lib.gemm_split_cluster.restype = cint
        lib.gemm_rmsnorm.argtypes = [i64, i64, ctypes.POINTER(RmsnormArgs), vp]
        lib.gemm_rmsnorm.restype = cint
        lib.gemm_rmsnorm_backward.argtypes = [i64, i64, ctypes.POINTER(RmsnormGradArgs), vp]
        lib.gemm_rmsnorm_backward.restype = cint
        lib.gemm_fp8_quantize.argtypes = [i64, i64, vp, i64, cint, cint, cint, vp, i64, vp, i64, vp]
        lib.gemm_fp8_quantize.restype = cint
        lib.gemm_fp8gemm.argtypes = [i64, i64, i64, f32, vp, i64, vp, i64, vp, i64, vp, i64, cint,
                                     f32, vp, i64, cint, vp]
        lib.gemm_fp8gemm.restype = cint
        lib.gemm_fp8gemm_grouped.argtypes = [i64, vp, i64, i64, i64, f32, vp, i64, vp, i64, vp, i64,
                                             i64, vp, i64, i64, cint, f32, vp, i64, cint, vp]
        lib.gemm_fp8gemm_grouped.restype = cint
        lib.gemm_bf16gemm_grouped.argtypes = [i64, vp, i64, i64, i64, f32, vp, i64, vp, i64, i64,
                                              cint, f32, vp, i64, cint, vp]
        lib.gemm_bf16gemm_grouped.restype = cint
        lib.gemm_bf16gemm_grouped_wgrad.argtypes = [i64, vp, i64, i64, i64, f32, vp, i64, vp, i64,
                                                    f32, vp, i64, i64, cint, vp]
        lib.gemm_bf16gemm_grouped_wgrad.restype = cint
        lib.gemm_version.argtypes = []
        lib.gemm_version.restype = cint
        _lib = lib
        return lib


# ----------------------------------------------------------- C-ABI mirrors
def gemm_sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """fp32 SGEMM; pointers are device addresses (int). Returns the status."""
    return load_library().gemm_sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16gemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """bf16-in / fp32-out GEMM; pointers are device addresses. Returns the status."""
    return load_library().gemm_bf16gemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream)


def gemm_bf16gemm_decode_static(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=0) -> int:
    """Decode-shaped bf16 GEMM that allocates nothing (scratch in a fixed
    library-owned array); see include/gemm12.h. Returns the status."""
    return load_library().gemm_bf16gemm_decode_static(M, N, K, alpha, A, lda, B, ldb, beta, C,
                                                      ldc, stream)


ACT = {"none": 0, "relu": 1, "gelu": 2}
OUT = {"f32": 0, "bf16": 1, "f8e4m3": 2, "s8": 3}


def gemm_bf16gemm_epilogue(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias, act, D, ldd,
                           d_type, stream=0) -> int:
    """bf16 GEMM with fused bias / activation / output type (see include/gemm12.h).
    act and d_type are the C enum values (ACT / OUT). Returns the status."""
    return load_library().gemm_bf16gemm_epilogue(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                                 bias, act, D, ldd, d_type, stream)


def gemm_bf16gemm_fused(M, N, K, alpha, A, lda, B, ldb, out: "GemmOutput", stream=0) -> int:
    """bf16 GEMM with the general output stage (gemm_output_t). Returns the status."""
    return load_library().gemm_bf16gemm_fused(M, N, K, alpha, A, lda, B, ldb, ctypes.byref(out),
                                              stream)


def _config(cfg):
    if cfg is None:
        return None
    if isinstance(cfg, GemmConfig):
        return ctypes.byref(cfg)
    kernel = cfg.get("kernel", 0)
    split = cfg.get("split", 0)
    c = GemmConfig(KERNELS[kernel] if isinstance(kernel, str) else int(kernel),
                   SPLIT_STREAM if split == "stream" else int(split), int(cfg.get("group_m", 0)))
    return ctypes.byref(c)


def gemm_sgemm_config(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, cfg, stream=0) -> int:
    """gemm_sgemm with a pinned launch configuration (GemmConfig or a dict with
    kernel / split / group_m; None = automatic). Returns the status."""
    return load_library().gemm_sgemm_config(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                            _config(cfg), stream)


def gemm_bf16gemm_config(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, cfg, stream=0) -> int:
    """gemm_bf16gemm with a pinned launch configuration. Returns the status."""
    return load_library().gemm_bf16gemm_config(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                                               _config(cfg), stream)


def gemm_get_config(is_bf16, M, N, K):
    """(config dict, from_table) automatic dispatch uses for a shape on the current
    device; raises GemmError without a usable device."""
    c = GemmConfig()
    t = ctypes.c_int(0)
    st = load_library().gemm_get_config(int(bool(is_bf16)), M, N, K, ctypes.byref(c),
                                        ctypes.byref(t))
    if st != 0:
        raise GemmError(st, "gemm_get_config")
    names = {v: k for k, v in KERNELS.items()}
    return {"kernel": names[c.kernel], "split": c.split, "group_m": c.group_m}, bool(t.value)


def gemm_get_model_config(is_bf16, M, N, K):
    """The configuration the cost model alone chooses (ignoring the sweep's table)."""
    c = GemmConfig()
    st = load_library().gemm_get_model_config(int(bool(is_bf16)), M, N, K, ctypes.byref(c))
    if st != 0:
        raise GemmError(st, "gemm_get_model_config")
    names = {v: k for k, v in KERNELS.items()}
    return {"kernel": names[c.kernel], "split": c.split, "group_m": c.group_m}


def gemm_status_string(status: int) -> str:
    return load_library().gemm_status_string(int(status)).decode()


def gemm_check_device_error(stream=0) -> int:
    return load_library().gemm_check_device_error(stream)


def gemm_shutdown() -> int:
    return load_library().gemm_shutdown()


def gemm_release_stream(stream=0) -> int:
    """Free the scratch and staging buffers kept for `stream` (stream-ordered)."""
    return load_library().gemm_release_stream(stream)


def gemm_select_path(is_bf16, M, N, K, alpha, A, lda, B, ldb) -> str:
    """Name of the kernel path a call with these arguments takes (host-only):
    "simt_tma" / "simt_generic" / "simt_staged" (fp32 on the CUDA cores, with
    operands loaded by TMA, by generic loads, or from an aligned staging copy),
    "tc_bf16" / "tc_bf16_pair" / "tc_decode" / "tc_staged" (bf16 on the tensor
    cores), "simt_bf16" (bf16 widened on the CUDA cores), "scale_c", "none"."""
    return PATHS[load_library().gemm_select_path(int(bool(is_bf16)), M, N, K, alpha, A, lda,
                                                 B, ldb)]


def gemm_split_parts(is_bf16, M, N, K) -> int:
    """k-ranges per work item of the last round (1 = no split; 0 = no device)."""
    return load_library().gemm_split_parts(int(bool(is_bf16)), M, N, K)


def gemm_split_cluster(is_bf16, M, N, K, config=None) -> int:
    """TMA operands: the cluster size S whose CTAs add a tile's k-parts in
    distributed shared memory, 1 if they meet in global memory or nothing is
    split, 0 for invalid input or no device.  `config` as for the _config calls."""
    return load_library().gemm_split_cluster(int(bool(is_bf16)), M, N, K, _config(config))


def gemm_quantization(M, N, BM, BN, num_sms, ctas_per_sm) -> dict:
    """Tile / wave quantization of a launch (host-only arithmetic)."""
    q = _Quantization()
    st = load_library().gemm_quantization(M, N, BM, BN, num_sms, ctas_per_sm, ctypes.byref(q))
    if st != 0:
        raise GemmError(st, "gemm_quantization")
    return {name: getattr(q, name) for name, _ in _Quantization._fields_}


def gemm_version() -> int:
    return load_library().gemm_version()


# gemm_block_t: the shape of an fp8 matrix's scaled blocks.
BLOCK = {"rows": 0, "tiles": 1}


def gemm_rmsnorm(rows, dim, args: "RmsnormArgs", stream=0) -> int:
    """Root-mean-square norm (gemm_rmsnorm_t). Returns the status."""
    return load_library().gemm_rmsnorm(rows, dim, ctypes.byref(args), stream)


def gemm_rmsnorm_backward(rows, dim, args: "RmsnormGradArgs", stream=0) -> int:
    """Its gradients (gemm_rmsnorm_grad_t). Returns the status."""
    return load_library().gemm_rmsnorm_backward(rows, dim, ctypes.byref(args), stream)


def gemm_fp8_quantize(rows, cols, x, ldx, x_type, block, transpose, q, ldq, scales, ld_scales,
                      stream=0) -> int:
    """A matrix or its transpose in fp8 with block scales. Returns the status."""
    return load_library().gemm_fp8_quantize(rows, cols, x, ldx, x_type, block, transpose, q, ldq,
                                            scales, ld_scales, stream)


def gemm_fp8gemm(M, N, K, alpha, A, lda, a_scales, ld_as, B, ldb, b_scales, ld_bs, b_block, beta, D,
                 ldd, d_type, stream=0) -> int:
    """fp8 GEMM with block scales, B given as N x K. Returns the status."""
    return load_library().gemm_fp8gemm(M, N, K, alpha, A, lda, a_scales, ld_as, B, ldb, b_scales,
                                       ld_bs, b_block, beta, D, ldd, d_type, stream)


def gemm_fp8gemm_grouped(G, offsets, rows, N, K, alpha, A, lda, a_scales, ld_as, B, ldb, stride_b,
                         b_scales, ld_bs, stride_bs, b_block, beta, D, ldd, d_type,
                         stream=0) -> int:
    """fp8 products grouped by expert. Returns the status."""
    return load_library().gemm_fp8gemm_grouped(G, offsets, rows, N, K, alpha, A, lda, a_scales,
                                               ld_as, B, ldb, stride_b, b_scales, ld_bs, stride_bs,
                                               b_block, beta, D, ldd, d_type, stream)


def gemm_bf16gemm_grouped(G, offsets, rows, N, K, alpha, A, lda, B, ldb, stride_b, transpose_b,
                          beta, D, ldd, d_type, stream=0) -> int:
    """bf16 products grouped by expert. Returns the status."""
    return load_library().gemm_bf16gemm_grouped(G, offsets, rows, N, K, alpha, A, lda, B, ldb,
                                                stride_b, transpose_b, beta, D, ldd, d_type, stream)


def gemm_bf16gemm_grouped_wgrad(G, offsets, rows, N, K, alpha, A, lda, dD, lddd, beta, dB, ldb,
                                stride_b, d_type, stream=0) -> int:
    """Their gradient with respect to B. Returns the status."""
    return load_library().gemm_bf16gemm_grouped_wgrad(G, offsets, rows, N, K, alpha, A, lda, dD,
                                                      lddd, beta, dB, ldb, stride_b, d_type, stream)


# ------------------------------------------------------------ tensor helpers
def _row_major_ld(t, name):
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("%s must be row-major (unit column stride)" % name)
    return t.stride(0) if rows > 1 else max(cols, 1)


def _stream_handle(stream, device):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream


def sgemm(A, B, C, alpha=1.0, beta=0.0, stream=None):
    """C <- alpha*(A @ B) + beta*C in place for fp32 CUDA tensors (row-major views)."""
    import torch
    for t, n in ((A, "A"), (B, "B"), (C, "C")):
        if t.dtype != torch.float32 or not t.is_cuda:
            raise TypeError("%s must be a float32 CUDA tensor" % n)
    M, K = A.shape
    N = B.shape[1]
    if B.shape[0] != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(C.shape)))
    st = gemm_sgemm(M, N, K, float(alpha), A.data_ptr(), _row_major_ld(A, "A"), B.data_ptr(),
                    _row_major_ld(B, "B"), float(beta), C.data_ptr(), _row_major_ld(C, "C"),
                    _stream_handle(stream, C.device))
    if st != 0:
        raise GemmError(st, "gemm_sgemm")
    return C


def bf16gemm(A, B, C, alpha=1.0, beta=0.0, stream=None):
    """C <- alpha*(A @ B) + beta*C in place; A, B bf16 CUDA tensors, C fp32."""
    import torch
    for t, n, dt in ((A, "A", torch.bfloat16), (B, "B", torch.bfloat16), (C, "C", torch.float32)):
        if t.dtype != dt or not t.is_cuda:
            raise TypeError("%s must be a %s CUDA tensor" % (n, dt))
    M, K = A.shape
    N = B.shape[1]
    if B.shape[0] != K or tuple(C.shape) != (M, N):
        raise ValueError("shape mismatch: A %s, B %s, C %s" % (tuple(A.shape), tuple(B.shape),
                                                               tuple(C.shape)))
    st = gemm_bf16gemm(M, N, K, float(alpha), A.data_ptr(), _row_major_ld(A, "A"), B.data_ptr(),
                       _row_major_ld(B, "B"), float(beta), C.data_ptr(), _row_major_ld(C, "C"),
                       _stream_handle(stream, C.device))
    if st != 0:
        raise GemmError(st, "gemm_bf16gemm")
    return C


def bf16gemm_epilogue(A, B, D, C=None, alpha=1.0, beta=0.0, bias=None, act="none", stream=None):
    """D <- act(alpha*(A @ B) + beta*C + bias); A, B bf16, C and bias fp32, D fp32
    or bf16 (all CUDA tensors, row-major)."""
    import torch
    for t, n in ((A, "A"), (B, "B")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError("%s must be a bfloat16 CUDA tensor" % n)
    if D.dtype not in (torch.float32, torch.bfloat16) or not D.is_cuda:
        raise TypeError("D must be a float32 or bfloat16 CUDA tensor")
    M, K = A.shape
    N = B.shape[1]
    if B.shape[0] != K or tuple(D.shape) != (M, N):
        raise ValueError("shape mismatch")
    c_ptr, ldc = 0, max(N, 1)
    if C is not None:
        if C.dtype != torch.float32 or tuple(C.shape) != (M, N):
            raise TypeError("C must be a float32 (M, N) tensor")
        c_ptr, ldc = C.data_ptr(), _row_major_ld(C, "C")
    b_ptr = 0
    if bias is not None:
        if bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous float32 tensor of N values")
        b_ptr = bias.data_ptr()
    st = gemm_bf16gemm_epilogue(M, N, K, float(alpha), A.data_ptr(), _row_major_ld(A, "A"),
                                B.data_ptr(), _row_major_ld(B, "B"), float(beta), c_ptr, ldc,
                                b_ptr, ACT[act], D.data_ptr(), _row_major_ld(D, "D"),
                                OUT["bf16" if D.dtype == torch.bfloat16 else "f32"],
                                _stream_handle(stream, D.device))
    if st != 0:
        raise GemmError(st, "gemm_bf16gemm_epilogue")
    return D


def _out_type(torch, D):
    kinds = {torch.float32: "f32", torch.bfloat16: "bf16", torch.int8: "s8"}
    if hasattr(torch, "float8_e4m3fn"):
        kinds[torch.float8_e4m3fn] = "f8e4m3"
    if D.dtype not in kinds or not D.is_cuda:
        raise TypeError("D must be a float32, bfloat16, float8_e4m3fn or int8 CUDA tensor")
    return OUT[kinds[D.dtype]]


def bf16gemm_fused(A, B, D, C=None, alpha=1.0, beta=0.0, bias=None, act="none", residual=None,
                   d_scale=1.0, amax=None, stream=None):
    """v = act(alpha*(A @ B) + beta*C + bias) + residual; D <- convert(d_scale * v) in D's
    dtype (float32, bfloat16, float8_e4m3fn or int8); amax (a float32 CUDA tensor of one
    element, or None) is raised to max |v|.  A, B bf16; C, bias, residual fp32."""
    import torch
    for t, n in ((A, "A"), (B, "B")):
        if t.dtype != torch.bfloat16 or not t.is_cuda:
            raise TypeError("%s must be a bfloat16 CUDA tensor" % n)
    M, K = A.shape
    N = B.shape[1]
    if B.shape[0] != K or tuple(D.shape) != (M, N):
        raise ValueError("shape mismatch")
    o = GemmOutput()
    o.beta = float(beta)
    o.C, o.ldc = 0, max(N, 1)
    if C is not None:
        if C.dtype != torch.float32 or tuple(C.shape) != (M, N):
            raise TypeError("C must be a float32 (M, N) tensor")
        o.C, o.ldc = C.data_ptr(), _row_major_ld(C, "C")
    o.bias = 0
    if bias is not None:
        if bias.dtype != torch.float32 or bias.numel() != N or not bias.is_contiguous():
            raise TypeError("bias must be a contiguous float32 tensor of N values")
        o.bias = bias.data_ptr()
    o.act = ACT[act]
    o.residual, o.ldr = 0, max(N, 1)
    if residual is not None:
        if residual.dtype != torch.float32 or tuple(residual.shape) != (M, N):
            raise TypeError("residual must be a float32 (M, N) tensor")
        o.residual, o.ldr = residual.data_ptr(), _row_major_ld(residual, "residual")
    o.d_scale = float(d_scale)
    o.amax = 0
    if amax is not None:
        if amax.dtype != torch.float32 or amax.numel() != 1 or not amax.is_cuda:
            raise TypeError("amax must be a float32 CUDA tensor of one element")
        o.amax = amax.data_ptr()
    o.D, o.ldd, o.d_type = D.data_ptr(), _row_major_ld(D, "D"), _out_type(torch, D)
    st = gemm_bf16gemm_fused(M, N, K, float(alpha), A.data_ptr(), _row_major_ld(A, "A"),
                             B.data_ptr(), _row_major_ld(B, "B"), o, _stream_handle(stream, D.device))
    if st != 0:
        raise GemmError(st, "gemm_bf16gemm_fused")
    return D


# ------------------------------------------- operators around the GEMMs
# A call of a small operator takes a few microseconds on the GPU, so these
# helpers look at each tensor once: the device number (-1 on the host), dtype,
# shape and strides.
_TORCH = None       # torch, its current-stream getter and the dtypes used below
_FLOAT_CODES = {}   # dtype -> gemm_out_t


def _torch_once():
    global _TORCH
    if _TORCH is None:
        import torch
        _FLOAT_CODES.update({torch.float32: OUT["f32"], torch.bfloat16: OUT["bf16"]})
        getter = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if getter is None:
            def getter(index):
                return torch.cuda.current_stream(index).cuda_stream
        _TORCH = (getter, torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32)
    return _TORCH


def _stream_of(dev, stream):
    if dev < 0:
        raise TypeError("all tensors must be CUDA tensors")
    return _TORCH[0](dev) if stream is None else stream.cuda_stream


def _array(t, shape, dtype, dev, name):
    """(address, leading dimension) of a row-major matrix (or of each of a batch), checked."""
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError("%s must be a %s tensor on the other operands' device" % (name, dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError("%s must be row-major (unit column stride)" % name)
    return t.data_ptr(), strides[-2] if shape[-2] > 1 else max(shape[-1], 1)


def _float_array(t, shape, dev, name):
    """(address, leading dimension, type) of a float32 or bfloat16 matrix."""
    code = _FLOAT_CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s must be a float32 or bfloat16 tensor" % name)
    return (*_array(t, shape, t.dtype, dev, name), code)


def _vector(t, n, dtype, dev, name):
    """Address of a contiguous vector of n values."""
    if t.dtype != dtype or t.get_device() != dev:
        raise TypeError("%s must be a %s tensor on the other operands' device" % (name, dtype))
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous vector of %d values" % (name, n))
    return t.data_ptr()


def _batch_stride(t, ld):
    return t.stride(0) if t.shape[0] > 1 else t.shape[1] * ld


def rmsnorm(x, weight, eps=1e-6, residual=None, h=None, y=None, q=None, scales=None, rstd=None,
            stream=None):
    """h = x + residual; y = h / sqrt(mean(h^2) + eps) * weight over the last dimension of x
    (rows, dim), into the given outputs: h, y (float32 or bfloat16), q with scales (y in
    float8_e4m3fn, scales (ceil(dim / 128), rows) float32) and rstd (rows,).  weight is float32.
    h may be the residual itself and y may be x itself."""
    _, f8, f32, _, _ = _torch_once()
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    shape, dev = x.shape, x.get_device()
    rows, dim = shape
    handle = _stream_of(dev, stream)
    if (q is None) != (scales is None):
        raise ValueError("q and scales come together")
    none = (None, 0, 0)
    a = RmsnormArgs(
        *_float_array(x, shape, dev, "x"),
        *(none if residual is None else _float_array(residual, shape, dev, "residual")),
        *(none if h is None else _float_array(h, shape, dev, "h")),
        _vector(weight, dim, f32, dev, "weight"), eps,
        *(none if y is None else _float_array(y, shape, dev, "y")),
        *((None, 0) if q is None else _array(q, shape, f8, dev, "q")),
        *((None, 0) if q is None else _array(scales, (-(-dim // 128), rows), f32, dev, "scales")),
        None if rstd is None else _vector(rstd, rows, f32, dev, "rstd"))
    st = load_library().gemm_rmsnorm(rows, dim, ctypes.byref(a), handle)
    if st != 0:
        raise GemmError(st, "gemm_rmsnorm")


def rmsnorm_backward(dy, h, weight, rstd, dh, dweight=None, residual_grad=None, stream=None):
    """Gradients of rmsnorm's y: dh <- the gradient with respect to h (and so x and the
    residual) plus residual_grad, dweight (dim,) <- the one with respect to the weight."""
    f32 = _torch_once()[2]
    if dy.dim() != 2:
        raise ValueError("dy must be 2-D")
    shape, dev = dy.shape, dy.get_device()
    rows, dim = shape
    handle = _stream_of(dev, stream)
    a = RmsnormGradArgs(
        *_float_array(dy, shape, dev, "dy"), *_float_array(h, shape, dev, "h"),
        _vector(weight, dim, f32, dev, "weight"), _vector(rstd, rows, f32, dev, "rstd"),
        *((None, 0, 0) if residual_grad is None else
          _float_array(residual_grad, shape, dev, "residual_grad")),
        *_float_array(dh, shape, dev, "dh"),
        None if dweight is None else _vector(dweight, dim, f32, dev, "dweight"))
    st = load_library().gemm_rmsnorm_backward(rows, dim, ctypes.byref(a), handle)
    if st != 0:
        raise GemmError(st, "gemm_rmsnorm_backward")
    return dh


def fp8_quantize(x, q, scales, block="rows", transpose=False, stream=None):
    """x (rows, cols), float32 or bfloat16, or its transpose, into q (float8_e4m3fn) with one
    float32 scale per 1 x 128 ("rows") or 128 x 128 ("tiles") block of q: scales[b, r] is that
    of columns 128 b .. 128 b + 127 and row (or block of rows) r."""
    _, f8, f32, _, _ = _torch_once()
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    dev = x.get_device()
    handle = _stream_of(dev, stream)
    code = BLOCK[block]
    qr, qc = (cols, rows) if transpose else (rows, cols)
    px, ldx, x_type = _float_array(x, x.shape, dev, "x")
    pq, ldq = _array(q, (qr, qc), f8, dev, "q")
    ps, lds = _array(scales, (-(-qc // 128), -(-qr // 128) if code else qr), f32, dev, "scales")
    st = load_library().gemm_fp8_quantize(rows, cols, px, ldx, x_type, code, 1 if transpose else 0,
                                          pq, ldq, ps, lds, handle)
    if st != 0:
        raise GemmError(st, "gemm_fp8_quantize")
    return q


def _b_scales(b_scales, lead, kb, N, dev):
    """(address, leading dimension, block) of B's scales: one per row, or per 128 rows."""
    last = b_scales.shape[-1] if b_scales.dim() else -1
    block = 0 if last == N else 1
    return (*_array(b_scales, (*lead, kb, N if block == 0 else -(-N // 128)), _TORCH[2], dev,
                    "b_scales"), block)


def fp8gemm(A, a_scales, B, b_scales, D, alpha=1.0, beta=0.0, stream=None):
    """D <- alpha*(A @ B^T) + beta*D in place: A (M, K) and B (N, K) float8_e4m3fn, D float32 or
    bfloat16; a_scales (ceil(K / 128), M); b_scales (ceil(K / 128), N), or ceil(N / 128) in place
    of N for 128 x 128 blocks (see fp8_quantize)."""
    _, f8, f32, _, _ = _torch_once()
    if A.dim() != 2 or B.dim() != 2:
        raise ValueError("A and B must be 2-D")
    M, K = A.shape
    N = B.shape[0]
    dev = D.get_device()
    handle = _stream_of(dev, stream)
    kb = -(-K // 128)
    pa, lda = _array(A, (M, K), f8, dev, "A")
    pb, ldb = _array(B, (N, K), f8, dev, "B")
    psa, ld_as = _array(a_scales, (kb, M), f32, dev, "a_scales")
    psb, ld_bs, block = _b_scales(b_scales, (), kb, N, dev)
    pd, ldd, code = _float_array(D, (M, N), dev, "D")
    st = load_library().gemm_fp8gemm(M, N, K, alpha, pa, lda, psa, ld_as, pb, ldb, psb, ld_bs,
                                     block, beta, pd, ldd, code, handle)
    if st != 0:
        raise GemmError(st, "gemm_fp8gemm")
    return D


def fp8gemm_grouped(A, a_scales, B, b_scales, offsets, D, alpha=1.0, beta=0.0, stream=None):
    """fp8gemm for the rows offsets[g] .. offsets[g + 1] - 1 of A and D with B[g] (G, N, K) and
    b_scales[g]; offsets (G + 1,) int32, on the device."""
    _, f8, f32, _, i32 = _torch_once()
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be 2-D and B 3-D")
    M, K = A.shape
    G, N = B.shape[0], B.shape[1]
    dev = D.get_device()
    handle = _stream_of(dev, stream)
    kb = -(-K // 128)
    pa, lda = _array(A, (M, K), f8, dev, "A")
    pb, ldb = _array(B, (G, N, K), f8, dev, "B")
    psa, ld_as = _array(a_scales, (kb, M), f32, dev, "a_scales")
    psb, ld_bs, block = _b_scales(b_scales, (G,), kb, N, dev)
    pd, ldd, code = _float_array(D, (M, N), dev, "D")
    st = load_library().gemm_fp8gemm_grouped(
        G, _vector(offsets, G + 1, i32, dev, "offsets"), M, N, K, alpha, pa, lda, psa, ld_as, pb,
        ldb, _batch_stride(B, ldb), psb, ld_bs, _batch_stride(b_scales, ld_bs), block, beta, pd,
        ldd, code, handle)
    if st != 0:
        raise GemmError(st, "gemm_fp8gemm_grouped")
    return D


def bf16gemm_grouped(A, B, offsets, D, alpha=1.0, beta=0.0, transpose_b=False, stream=None):
    """D[t] <- alpha*(A[t] @ B[g]) + beta*D[t] in place for the rows t = offsets[g] ..
    offsets[g + 1] - 1 of each group; A (rows, K) and B (G, K, N) bfloat16 -- with transpose_b
    (G, N, K), and D = A @ B[g]^T --, D float32 or bfloat16, offsets (G + 1,) int32 on the device."""
    _, _, _, b16, i32 = _torch_once()
    if A.dim() != 2 or B.dim() != 3:
        raise ValueError("A must be 2-D and B 3-D")
    rows, K = A.shape
    G = B.shape[0]
    N = B.shape[1 if transpose_b else 2]
    dev = D.get_device()
    handle = _stream_of(dev, stream)
    pa, lda = _array(A, (rows, K), b16, dev, "A")
    pb, ldb = _array(B, (G, N, K) if transpose_b else (G, K, N), b16, dev, "B")
    pd, ldd, code = _float_array(D, (rows, N), dev, "D")
    st = load_library().gemm_bf16gemm_grouped(
        G, _vector(offsets, G + 1, i32, dev, "offsets"), rows, N, K, alpha, pa, lda, pb, ldb,
        _batch_stride(B, ldb), 1 if transpose_b else 0, beta, pd, ldd, code, handle)
    if st != 0:
        raise GemmError(st, "gemm_bf16gemm_grouped")
    return D


def bf16gemm_grouped_wgrad(A, dD, offsets, dB, alpha=1.0, beta=0.0, stream=None):
    """dB[g] <- alpha*(A_g^T @ dD_g) + beta*dB[g] in place: A (rows, K) and dD (rows, N) bfloat16,
    dB (G, K, N) float32 or bfloat16; a group without rows gets beta*dB[g]."""
    _, _, _, b16, i32 = _torch_once()
    if A.dim() != 2 or dD.dim() != 2 or dB.dim() != 3:
        raise ValueError("A and dD must be 2-D and dB 3-D")
    rows, K = A.shape
    N, G = dD.shape[1], dB.shape[0]
    dev = dB.get_device()
    handle = _stream_of(dev, stream)
    pa, lda = _array(A, (rows, K), b16, dev, "A")
    pd, lddd = _array(dD, (rows, N), b16, dev, "dD")
    pb, ldb, code = _float_array(dB, (G, K, N), dev, "dB")
    st = load_library().gemm_bf16gemm_grouped_wgrad(
        G, _vector(offsets, G + 1, i32, dev, "offsets"), rows, N, K, alpha, pa, lda, pd, lddd, beta,
        pb, ldb, _batch_stride(dB, ldb), code, handle)
    if st != 0:
        raise GemmError(st, "gemm_bf16gemm_grouped_wgrad")
    return dB
