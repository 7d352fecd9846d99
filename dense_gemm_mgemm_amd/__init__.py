"""Python binding of libmgemm (dense GEMM for MI355X / gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libmgemm.so``.  The functions carry the names of the C entry
points declared in ``include/mgemm.h``.  Operands are passed as device
pointers (ints) or as torch tensors on the GPU, whose ``data_ptr()`` is
taken; torch is used for device memory and streams only.

There is no fallback: if ``libmgemm.so`` is missing or fails to load, every
entry point raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmgemm.so")

(MGEMM_SUCCESS, MGEMM_ERR_INVALID_ARG, MGEMM_ERR_UNSUPPORTED, MGEMM_ERR_HIP, MGEMM_ERR_ALLOC,
 MGEMM_ERR_SCRATCH) = range(6)
MGEMM_ROW_MAJOR, MGEMM_COL_MAJOR = 0, 1
MGEMM_F32, MGEMM_F16, MGEMM_BF16 = 0, 1, 2
KERNELS = ["auto", "general", "f32_mfma", "h_mfma_256x256", "h_mfma_256x192", "h_mfma_128x128",
           "skinny", "reserved_7", "f32_fast", "f32_fast_128",
           "h_dma_256x256", "skinny_sk", "h_dma_256x192", "f32_fast_u",
           "f8_mfma_256x256", "f8_general", "f8_mfma_256x192", "f32_sk", "h_dma_128x192",
           "h_dma_64x192", "f8_mfma_128x192",
           "mx4_general", "mx4_skinny", "mx4_mfma_256x256", "mx4_mfma_256x192", "mx4_mfma_128x192",
           "mx4_mfma_64x192"]
MGEMM_KERNEL_AUTO = 0
MGEMM_EPILOGUE_NONE, MGEMM_EPILOGUE_SILU = 0, 1
_EPILOGUE = {"none": MGEMM_EPILOGUE_NONE, "silu": MGEMM_EPILOGUE_SILU}

_LAYOUT = {"row": MGEMM_ROW_MAJOR, "col": MGEMM_COL_MAJOR}
_DTYPE = {"f32": MGEMM_F32, "f16": MGEMM_F16, "bf16": MGEMM_BF16}

EXPORTED = ["mgemm_create", "mgemm_destroy", "mgemm_run", "mgemm_run_kernel", "mgemm_run_ex",
            "mgemm_run_variant", "mgemm_run_gated", "mgemm_run_gated_ex", "mgemm_select_kernel",
            "mgemm_select_variant", "mgemm_tune", "mgemm_table_export", "mgemm_table_import",
            "mgemm_table_clear", "mgemm_weighted_choice", "mgemm_quantize_fp8", "mgemm_run_fp8",
            "mgemm_status_string",
            "mgemm_kernel_name", "mgemm_num_cu", "mgemm_run_noalloc", "mgemm_set_clock_stamps",
            "mgemm_run_acc32", "mgemm_quantize_mx4", "mgemm_dequantize_mx4", "mgemm_run_mx4",
            "mgemm_linear_mx4", "mgemm_gated_mx4", "mgemm_gated_workspace",
            "mgemm_gated_forward", "mgemm_gated_backward", "mgemm_set_gated_tile", "mgemm_set_mx4_kernel"]


class MgemmError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s (status %d)" % (what, _status_str(status), status))
        self.status = status


_lib = None

MGEMM_MAX_KSPLIT = 32


class MgemmVariant(ctypes.Structure):
    """mgemm_variant_t: a kernel (mgemm_kernel_t) and its number of K ranges."""
    _fields_ = [("kernel", ctypes.c_int32), ("ksplit", ctypes.c_int32)]


class MgemmTuneResult(ctypes.Structure):
    """mgemm_tune_result_t."""
    _fields_ = [("chosen", MgemmVariant), ("chosen_us", ctypes.c_float), ("model", MgemmVariant),
                ("model_us", ctypes.c_float)]


def load(path: str | None = None):
    """Load libmgemm.so (raises OSError if it is not built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise OSError("libmgemm.so is not built (%s); run `python -m dense_gemm_mgemm_amd.build`" % p)
    lib = ctypes.CDLL(p)
    i64, f32, vp, ci = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    run_args = [ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, f32, vp, i64, ci, vp]
    lib.mgemm_create.argtypes = [ctypes.POINTER(vp)]
    lib.mgemm_destroy.argtypes = [vp]
    lib.mgemm_run.argtypes = [vp] + run_args
    lib.mgemm_run_kernel.argtypes = [vp, ci] + run_args
    lib.mgemm_run_ex.argtypes = [vp, ci] + run_args[:-1] + [ci, vp]
    lib.mgemm_run_gated.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp, i64, vp, i64, ci, vp]
    lib.mgemm_run_gated_ex.argtypes = [vp, ctypes.c_int32, i64, i64, i64, vp, i64, vp, vp, i64, vp,
                                       i64, ci, vp]
    lib.mgemm_run_variant.argtypes = [vp, ctypes.POINTER(MgemmVariant)] + run_args[:-1] + [ci, vp]
    lib.mgemm_select_variant.argtypes = [vp] + run_args[:-1] + [ctypes.POINTER(MgemmVariant)]
    lib.mgemm_run_noalloc.argtypes = [ctypes.POINTER(MgemmVariant)] + run_args[:-1] + [ci, vp]
    pi64, pdbl = ctypes.POINTER(i64), ctypes.POINTER(ctypes.c_double)
    lib.mgemm_tune.argtypes = [vp, ci, ci, ci, ctypes.c_int32, pi64, pi64, pi64, pdbl,
                               ctypes.POINTER(MgemmTuneResult), vp]
    lib.mgemm_table_export.argtypes = [vp, ctypes.c_char_p, ctypes.c_size_t,
                                       ctypes.POINTER(ctypes.c_size_t)]
    lib.mgemm_table_import.argtypes = [vp, ctypes.c_char_p]
    lib.mgemm_table_clear.argtypes = [vp]
    lib.mgemm_weighted_choice.argtypes = [ctypes.c_int32, ctypes.c_int32, pdbl, pdbl]
    lib.mgemm_weighted_choice.restype = ctypes.c_int32
    lib.mgemm_quantize_fp8.argtypes = [vp, i64, i64, vp, i64, ci, vp, i64, vp, vp]
    lib.mgemm_run_fp8.argtypes = [vp, ci, ctypes.c_int32, i64, i64, i64, f32, vp, i64, vp, vp, i64,
                                  vp, f32, vp, i64, ci, vp]
    lib.mgemm_select_kernel.argtypes = [vp] + run_args[:-1] + [ctypes.POINTER(ci)]
    for name in ("mgemm_create", "mgemm_destroy", "mgemm_run", "mgemm_run_kernel", "mgemm_run_ex",
                 "mgemm_run_gated", "mgemm_run_gated_ex", "mgemm_run_variant",
                 "mgemm_select_variant", "mgemm_select_kernel", "mgemm_tune", "mgemm_table_export",
                 "mgemm_table_import", "mgemm_table_clear", "mgemm_quantize_fp8",
                 "mgemm_run_fp8", "mgemm_run_noalloc", "mgemm_run_acc32"):
        getattr(lib, name).restype = ci
    lib.mgemm_run_acc32.argtypes = [vp, ci, ci, ci, i64, i64, i64, f32, vp, i64, vp, i64, vp, i64,
                                    ci, vp]
    lib.mgemm_quantize_mx4.argtypes = [vp, i64, i64, vp, i64, ci, vp, i64, vp, i64, vp]
    lib.mgemm_dequantize_mx4.argtypes = [vp, i64, i64, vp, i64, vp, i64, vp, i64, ci, vp]
    lib.mgemm_run_mx4.argtypes = [vp, ci, ctypes.c_int32, i64, i64, i64, f32, vp, i64, vp, i64, vp,
                                  i64, vp, i64, f32, vp, i64, ci, vp]
    lib.mgemm_linear_mx4.argtypes = [vp, i64, i64, i64, vp, i64, ci, vp, i64, vp, i64, vp, i64, ci, vp]
    lib.mgemm_gated_mx4.argtypes = [vp, i64, i64, i64, vp, i64, ci, vp, vp, vp, vp, i64, i64, vp, i64,
                                    ci, vp]
    lib.mgemm_set_mx4_kernel.argtypes = [vp, ci, ctypes.c_int32]
    for name in ("mgemm_quantize_mx4", "mgemm_dequantize_mx4", "mgemm_run_mx4", "mgemm_linear_mx4",
                 "mgemm_gated_mx4", "mgemm_set_mx4_kernel"):
        getattr(lib, name).restype = ci
    gated = [vp, ci, i64, i64, i64, vp, i64, vp, vp, i64]
    lib.mgemm_gated_workspace.argtypes = gated[1:] + [ci, ctypes.c_int32, ctypes.c_int32, pi64]
    lib.mgemm_gated_forward.argtypes = gated + [vp, i64, vp, vp, i64, ci, vp, i64, vp]
    lib.mgemm_gated_backward.argtypes = gated + [vp, vp, i64, vp, i64, vp, i64, vp, vp, i64, f32, ci, vp, i64, vp]
    lib.mgemm_set_gated_tile.argtypes = [vp] + [ctypes.c_int32] * 3
    for name in ("mgemm_gated_workspace", "mgemm_gated_forward", "mgemm_gated_backward", "mgemm_set_gated_tile"):
        getattr(lib, name).restype = ci
    lib.mgemm_status_string.argtypes = [ci]
    lib.mgemm_status_string.restype = ctypes.c_char_p
    lib.mgemm_kernel_name.argtypes = [ci]
    lib.mgemm_kernel_name.restype = ctypes.c_char_p
    lib.mgemm_num_cu.argtypes = [vp]
    lib.mgemm_num_cu.restype = ci
    lib.mgemm_set_clock_stamps.argtypes = [vp, vp, i64]
    lib.mgemm_set_clock_stamps.restype = ci
    if path is None:
        _lib = lib
    return lib


def _status_str(s: int) -> str:
    try:
        return load().mgemm_status_string(s).decode()
    except OSError:
        return "status %d" % s


def _ptr(x) -> int | None:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _enum(x, table):
    return table[x] if isinstance(x, str) else int(x)


def _stream(s) -> int | None:
    if s is None:
        import torch
        # torch.cuda.current_stream().cuda_stream without the Stream object (2.8 us, of a call's 7).
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def mgemm_create() -> int:
    """Handle bound to the current HIP device."""
    h = ctypes.c_void_p()
    st = load().mgemm_create(ctypes.byref(h))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_create")
    return h.value


def mgemm_destroy(h: int) -> None:
    load().mgemm_destroy(h)


def _args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype):
    return (_enum(layoutA, _LAYOUT), _enum(layoutB, _LAYOUT), int(M), int(N), int(K), float(alpha),
            _ptr(A), int(lda), _ptr(B), int(ldb), float(beta), _ptr(C), int(ldc),
            _enum(dtype, _DTYPE))


def mgemm_run(h, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype,
              stream=None) -> None:
    """Enqueue C = alpha*op(A)op(B) + beta*C on `stream` (torch's current by default)."""
    st = load().mgemm_run(h, *_args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                                    ldc, dtype), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run")


def mgemm_run_kernel(h, kernel, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                     dtype, stream=None) -> None:
    """As mgemm_run with one kernel variant forced (name or number)."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_run_kernel(h, k, *_args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb,
                                              beta, C, ldc, dtype), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_kernel(%s)" % KERNELS[k] if 0 <= k < len(KERNELS) else k)


def mgemm_run_acc32(h, kernel, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, C32, ldc, dtype,
                    stream=None) -> None:
    """C32 (FP32, layoutA's order) = alpha*op(A)op(B): the 16-bit direct-to-LDS
    kernel's sums before the output rounding ("auto", "h_dma_256x256" or
    "h_dma_256x192")."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_run_acc32(h, k, _enum(layoutA, _LAYOUT), _enum(layoutB, _LAYOUT), int(M),
                                int(N), int(K), float(alpha), _ptr(A), int(lda), _ptr(B), int(ldb),
                                _ptr(C32), int(ldc), _enum(dtype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_acc32")


def mgemm_run_ex(h, kernel, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, dtype,
                 epilogue="none", stream=None) -> None:
    """As mgemm_run ("auto") or mgemm_run_kernel, with an output epilogue ("none" or "silu")."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_run_ex(h, k, *_args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta,
                                          C, ldc, dtype), _enum(epilogue, _EPILOGUE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_ex(%s, %s)" % (kernel, epilogue))


def mgemm_run_gated(h, M, N, K, X, ldx, Wg, Wu, ldw, Z, ldz, dtype, stream=None) -> None:
    """Enqueue Z = SiLU(X W_g) * (X W_u) (row-major, 16-bit) on `stream`."""
    st = load().mgemm_run_gated(h, int(M), int(N), int(K), _ptr(X), int(ldx), _ptr(Wg), _ptr(Wu),
                                int(ldw), _ptr(Z), int(ldz), _enum(dtype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_gated")


def mgemm_run_variant(h, kernel, ksplit, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                      ldc, dtype, epilogue="none", stream=None) -> None:
    """As mgemm_run_ex with a split of K (0: the library's choice, 1: none, n: at most n ranges)."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    v = MgemmVariant(k, int(ksplit))
    st = load().mgemm_run_variant(h, ctypes.byref(v), *_args(layoutA, layoutB, M, N, K, alpha, A,
                                                             lda, B, ldb, beta, C, ldc, dtype),
                                  _enum(epilogue, _EPILOGUE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_variant(%s, %d)" % (kernel, ksplit))


def mgemm_run_noalloc(kernel, ksplit, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C,
                      ldc, dtype, epilogue="none", stream=None) -> None:
    """mgemm_run_variant without a handle or any allocation (the library's
    static scratch array on the current device)."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    v = MgemmVariant(k, int(ksplit))
    st = load().mgemm_run_noalloc(ctypes.byref(v), *_args(layoutA, layoutB, M, N, K, alpha, A, lda,
                                                          B, ldb, beta, C, ldc, dtype),
                                  _enum(epilogue, _EPILOGUE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_noalloc(%s, %d)" % (kernel, ksplit))


def mgemm_run_gated_ex(h, ksplit, M, N, K, X, ldx, Wg, Wu, ldw, Z, ldz, dtype, stream=None) -> None:
    """mgemm_run_gated with a split of K (0: the library's choice)."""
    st = load().mgemm_run_gated_ex(h, int(ksplit), int(M), int(N), int(K), _ptr(X), int(ldx),
                                   _ptr(Wg), _ptr(Wu), int(ldw), _ptr(Z), int(ldz),
                                   _enum(dtype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_gated_ex(%d)" % ksplit)


def mgemm_select_variant(h, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                         dtype) -> tuple:
    """(kernel name, K ranges) that mgemm_run would launch (("auto", 0): scale-only or nothing)."""
    out = MgemmVariant()
    st = load().mgemm_select_variant(h, *_args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb,
                                               beta, C, ldc, dtype), ctypes.byref(out))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_select_variant")
    return load().mgemm_kernel_name(out.kernel).decode(), int(out.ksplit)


def mgemm_tune(h, dtype, layoutA, layoutB, shapes, calls=None, stream=None) -> list:
    """Measure every variant on each (M, N, K) and fill the handle's dispatch
    table (blocking).  Returns, per shape, the fastest variant and the model's
    choice with their measured times."""
    n = len(shapes)
    arr = lambda vals, t: (t * n)(*vals)
    Ms = arr([int(s[0]) for s in shapes], ctypes.c_int64)
    Ns = arr([int(s[1]) for s in shapes], ctypes.c_int64)
    Ks = arr([int(s[2]) for s in shapes], ctypes.c_int64)
    cw = None if calls is None else arr([float(c) for c in calls], ctypes.c_double)
    res = (MgemmTuneResult * n)()
    st = load().mgemm_tune(h, _enum(dtype, _DTYPE), _enum(layoutA, _LAYOUT), _enum(layoutB, _LAYOUT),
                           n, Ms, Ns, Ks, cw, res, _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_tune")
    name = lambda v: (load().mgemm_kernel_name(v.kernel).decode(), int(v.ksplit))
    return [{"shape": tuple(shapes[i]), "chosen": name(r.chosen), "chosen_us": r.chosen_us,
             "model": name(r.model), "model_us": r.model_us} for i, r in enumerate(res)]


def mgemm_table_export(h) -> str:
    """The handle's dispatch table as text."""
    n = ctypes.c_size_t()
    st = load().mgemm_table_export(h, None, 0, ctypes.byref(n))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_table_export")
    buf = ctypes.create_string_buffer(n.value + 1)
    st = load().mgemm_table_export(h, buf, n.value + 1, ctypes.byref(n))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_table_export")
    return buf.value.decode()


def mgemm_table_import(h, text: str) -> None:
    st = load().mgemm_table_import(h, text.encode())
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_table_import")


def mgemm_table_clear(h) -> None:
    st = load().mgemm_table_clear(h)
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_table_clear")


def mgemm_weighted_choice(times, calls=None) -> int:
    """Index of the variant (column of `times`, one row per shape) with the
    smallest call-weighted total time; -1 if none runs every called shape."""
    rows = [list(map(float, r)) for r in times]
    ns, nv = len(rows), len(rows[0]) if rows else 0
    flat = (ctypes.c_double * (ns * nv))(*[t for r in rows for t in r])
    cw = None if calls is None else (ctypes.c_double * ns)(*map(float, calls))
    return int(load().mgemm_weighted_choice(ns, nv, flat, cw))


def mgemm_quantize_fp8(h, M, K, X, ldx, xtype, Q, ldq, scales, stream=None) -> None:
    """Per-row E4M3 quantisation of X (M x K) into codes Q and FP32 scales."""
    st = load().mgemm_quantize_fp8(h, int(M), int(K), _ptr(X), int(ldx), _enum(xtype, _DTYPE),
                                   _ptr(Q), int(ldq), _ptr(scales), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_quantize_fp8")


def mgemm_run_fp8(h, kernel, M, N, K, alpha, A, lda, sa, B, ldb, sb, beta, C, ldc, ctype,
                  stream=None, ksplit=0) -> None:
    """C = alpha * sa[m] * sb[n] * sum_k A[m,k] B[n,k] + beta * C on E4M3 codes
    (ksplit: 0 = the library's choice, 1 = no split, n = at most n K ranges)."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_run_fp8(h, k, int(ksplit), int(M), int(N), int(K), float(alpha), _ptr(A),
                              int(lda), _ptr(sa), _ptr(B), int(ldb), _ptr(sb), float(beta),
                              _ptr(C), int(ldc), _enum(ctype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_fp8(%s, %d)" % (kernel, ksplit))


def mgemm_quantize_mx4(h, M, K, X, ldx, xtype, Q, ldq, S, lds, stream=None) -> None:
    """X (M x K) to MX4 codes Q (row stride ldq bytes) and scale bytes S (row stride lds)."""
    st = load().mgemm_quantize_mx4(h, int(M), int(K), _ptr(X), int(ldx), _enum(xtype, _DTYPE), _ptr(Q),
                                   int(ldq), _ptr(S), int(lds), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_quantize_mx4")


def mgemm_dequantize_mx4(h, M, K, Q, ldq, S, lds, Y, ldy, ytype, stream=None) -> None:
    """The values that MX4 codes and scales stand for, into Y (M x K)."""
    st = load().mgemm_dequantize_mx4(h, int(M), int(K), _ptr(Q), int(ldq), _ptr(S), int(lds), _ptr(Y),
                                     int(ldy), _enum(ytype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_dequantize_mx4")


def mgemm_run_mx4(h, kernel, M, N, K, alpha, A, lda, SA, ldsa, B, ldb, SB, ldsb, beta, C, ldc, ctype,
                  stream=None, ksplit=0) -> None:
    """C = alpha * A B^T + beta * C on MX4 codes and scales (ksplit: 0 = the
    library's choice, 1 = no split, n = at most n K ranges)."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_run_mx4(h, k, int(ksplit), int(M), int(N), int(K), float(alpha), _ptr(A), int(lda),
                              _ptr(SA), int(ldsa), _ptr(B), int(ldb), _ptr(SB), int(ldsb), float(beta),
                              _ptr(C), int(ldc), _enum(ctype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_run_mx4(%s, %d)" % (kernel, ksplit))


def mgemm_linear_mx4(h, M, N, K, X, ldx, xtype, B, ldb, SB, ldsb, Y, ldy, ytype, stream=None) -> None:
    """Y = Q(X) B^T: MX4 weights (N x K), activations quantised within the call."""
    st = load().mgemm_linear_mx4(h, int(M), int(N), int(K), _ptr(X), int(ldx), _enum(xtype, _DTYPE),
                                 _ptr(B), int(ldb), _ptr(SB), int(ldsb), _ptr(Y), int(ldy),
                                 _enum(ytype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_linear_mx4")


def mgemm_gated_mx4(h, M, N, K, X, ldx, xtype, Bg, SBg, Bu, SBu, ldb, ldsb, Z, ldz, ztype,
                    stream=None) -> None:
    """Z = SiLU(Q(X) Bg^T) * (Q(X) Bu^T): MX4 weights (N x K each), activations
    quantised within the call."""
    st = load().mgemm_gated_mx4(h, int(M), int(N), int(K), _ptr(X), int(ldx), _enum(xtype, _DTYPE),
                                _ptr(Bg), _ptr(SBg), _ptr(Bu), _ptr(SBu), int(ldb), int(ldsb), _ptr(Z),
                                int(ldz), _enum(ztype, _DTYPE), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_gated_mx4")


def mgemm_set_mx4_kernel(h, kernel="auto", ksplit=0) -> None:
    """Check hook: forces the kernel and split of the products in mgemm_linear_mx4
    and mgemm_gated_mx4; "auto", 0: the library's choice."""
    k = KERNELS.index(kernel) if isinstance(kernel, str) else int(kernel)
    st = load().mgemm_set_mx4_kernel(h, k, int(ksplit))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_set_mx4_kernel")


def mgemm_gated_workspace(layout, M, N, K, X, ldx, Wg, Wu, ldw, dtype, backward, stored) -> int:
    """Bytes of workspace that mgemm_gated_forward (backward False) or
    mgemm_gated_backward needs for these operands (stored: with G and U given)."""
    out = ctypes.c_int64()
    st = load().mgemm_gated_workspace(_enum(layout, _LAYOUT), int(M), int(N), int(K), _ptr(X), int(ldx), _ptr(Wg),
                                      _ptr(Wu), int(ldw), _enum(dtype, _DTYPE), int(bool(backward)),
                                      int(bool(stored)), ctypes.byref(out))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_gated_workspace")
    return int(out.value)


def mgemm_gated_forward(h, layout, M, N, K, X, ldx, Wg, Wu, ldw, Z, ldz, G, U, ldg, dtype, work, work_bytes,
                        stream=None) -> None:
    """Z = SiLU(X Wg) * (X Wu), with G = X Wg and U = X Wu stored unless both
    are None (weights K x N for layout "row", N x K for "col")."""
    st = load().mgemm_gated_forward(h, _enum(layout, _LAYOUT), int(M), int(N), int(K), _ptr(X), int(ldx), _ptr(Wg),
                                    _ptr(Wu), int(ldw), _ptr(Z), int(ldz), _ptr(G), _ptr(U), int(ldg),
                                    _enum(dtype, _DTYPE), _ptr(work), int(work_bytes), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_gated_forward")


def mgemm_gated_backward(h, layout, M, N, K, X, ldx, Wg, Wu, ldw, G, U, ldg, dZ, lddz, dX, lddx, dWg, dWu, lddw,
                         beta, dtype, work, work_bytes, stream=None) -> None:
    """dX (or None), and dWg, dWu = X^T d + beta * dW (or both None), from dZ;
    G and U as the forward pass stored them, or both None: computed again."""
    st = load().mgemm_gated_backward(h, _enum(layout, _LAYOUT), int(M), int(N), int(K), _ptr(X), int(ldx), _ptr(Wg),
                                     _ptr(Wu), int(ldw), _ptr(G), _ptr(U), int(ldg), _ptr(dZ), int(lddz), _ptr(dX),
                                     int(lddx), _ptr(dWg), _ptr(dWu), int(lddw), float(beta), _enum(dtype, _DTYPE),
                                     _ptr(work), int(work_bytes), _stream(stream))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_gated_backward")


def mgemm_set_gated_tile(h, product, size=0, ksplit=0) -> None:
    """Check hook: forces the tile of a product of the gated block (0 the forward
    pair, 1 dX, 2 the weights' gradients); 0: the library's choice."""
    st = load().mgemm_set_gated_tile(h, int(product), int(size), int(ksplit))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_set_gated_tile")


def mgemm_select_kernel(h, layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc,
                        dtype) -> str:
    """Name of the variant mgemm_run would launch ("auto": scale-only or nothing)."""
    out = ctypes.c_int()
    st = load().mgemm_select_kernel(h, *_args(layoutA, layoutB, M, N, K, alpha, A, lda, B, ldb,
                                              beta, C, ldc, dtype), ctypes.byref(out))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_select_kernel")
    return load().mgemm_kernel_name(out.value).decode()


def mgemm_status_string(s: int) -> str:
    return load().mgemm_status_string(s).decode()


def mgemm_kernel_name(k: int) -> str:
    return load().mgemm_kernel_name(k).decode()


def mgemm_num_cu(h) -> int:
    return load().mgemm_num_cu(h)


def mgemm_set_clock_stamps(h, buf, nblocks: int) -> None:
    """Measurement hook: buf (device, 4*nblocks int64, or None) receives each
    workgroup's (cycles at start, at end, 100 MHz ticks at start, at end)."""
    st = load().mgemm_set_clock_stamps(h, _ptr(buf), int(nblocks))
    if st != MGEMM_SUCCESS:
        raise MgemmError(st, "mgemm_set_clock_stamps")
