"""ctypes binding of ``libqlora_nf4.so``: the C ABI of ``include/qlora_nf4.h``, same names.

Argument marshalling only.  Loading the library needs no GPU; the device entry
points return ``QLORA_ERR_DEVICE`` when no gfx950 device is present.  There is no
fallback: if the shared library has not been built, loading raises.
"""

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libqlora_nf4.so")

QLORA_OK = 0
QLORA_ERR_NULL = -1
QLORA_ERR_SHAPE = -2
QLORA_ERR_RANK = -3
QLORA_ERR_DTYPE = -4
QLORA_ERR_WORKSPACE = -5
QLORA_ERR_ALIGN = -6
QLORA_ERR_DEVICE = -7
QLORA_ERR_LAUNCH = -8
QLORA_ERR_VALUE = -9
QLORA_MAX_PARTS = 8
QLORA_F32 = 0
QLORA_BF16 = 1
QLORA_QUANT_NF4 = 0
QLORA_QUANT_FP4 = 1
QLORA_CONST_DQ_INT8 = 0
QLORA_CONST_DQ_FP8 = 1
QLORA_CONST_FP32 = 2
QLORA_ACT_SILU = 0
QLORA_ACT_GELU_TANH = 1

EXPORTED = (
    "qlora_nf4_sizes", "qlora_nf4_codebook", "qlora_workspace_bytes", "qlora_status_string",
    "qlora_last_error", "qlora_quantize_nf4", "qlora_dequantize", "qlora_linear_fwd",
    "qlora_linear_bwd", "qlora_time_next_gemm", "qlora_adamw_step", "qlora_lora_merge",
    "qlora_lora_unmerge", "qlora_workspace_bytes_fused", "qlora_linear_fwd_fused",
    "qlora_linear_bwd_fused", "qlora_nf4_concat_rows", "qlora_quantize", "qlora_codebook",
    "qlora_linear_fwd_noalloc", "qlora_workspace_bytes_dropout", "qlora_linear_fwd_dropout",
    "qlora_linear_bwd_dropout", "qlora_dropout", "qlora_workspace_bytes_gated", "qlora_gated_fwd",
    "qlora_gated_bwd",
)
QLORA_NOALLOC_SCRATCH_BYTES = 16 << 20
QLORA_WORKSPACE_HEADER_BYTES = 65792  # leading workspace bytes that must be zero at first use


class qlora_nf4_weight(ctypes.Structure):
    _fields_ = [
        ("codes", ctypes.c_void_p),
        ("absmax_q", ctypes.c_void_p),
        ("dq_scale", ctypes.c_void_p),
        ("dq_offset", ctypes.c_void_p),
        ("n_rows", ctypes.c_int64),
        ("n_cols", ctypes.c_int64),
        ("absmax", ctypes.c_void_p),
        ("quant_type", ctypes.c_int32),
        ("const_type", ctypes.c_int32),
    ]


class qlora_drop(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64), ("offset", ctypes.c_uint64),
                ("counter", ctypes.c_void_p)]


_lib = None


def load(path=LIB_PATH):
    """Load (once) and return the ctypes library with prototypes set."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m bit_quantized_lora_nf4_amd.build`")
    # torch ships its own libamdhip64 under the same soname; load it first so that the
    # library and torch share one HIP runtime (device memory, streams, events).
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    lib = ctypes.CDLL(path)
    P, I64, I32, SZ, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    W = ctypes.POINTER(qlora_nf4_weight)
    lib.qlora_nf4_sizes.argtypes = [I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(I64), ctypes.POINTER(I64)]
    lib.qlora_nf4_sizes.restype = I32
    lib.qlora_nf4_codebook.argtypes = [ctypes.POINTER(F32), ctypes.POINTER(F32)]
    lib.qlora_nf4_codebook.restype = None
    lib.qlora_workspace_bytes.argtypes = [I32, I64, I64, I64, I32]
    lib.qlora_workspace_bytes.restype = SZ
    lib.qlora_status_string.argtypes = [I32]
    lib.qlora_status_string.restype = ctypes.c_char_p
    lib.qlora_last_error.argtypes = []
    lib.qlora_last_error.restype = ctypes.c_char_p
    lib.qlora_quantize_nf4.argtypes = [P, I32, I64, I64, P, P, P, P, P, P]
    lib.qlora_quantize_nf4.restype = I32
    lib.qlora_dequantize.argtypes = [W, P, I32, P]
    lib.qlora_dequantize.restype = I32
    lib.qlora_linear_fwd.argtypes = [W, P, I64, P, P, I32, F32, P, P, P, SZ, P]
    lib.qlora_linear_fwd.restype = I32
    lib.qlora_linear_fwd_noalloc.argtypes = [W, P, I64, P, P, I32, F32, P, P, P]
    lib.qlora_linear_fwd_noalloc.restype = I32
    lib.qlora_linear_bwd.argtypes = [W, P, P, I64, P, P, I32, F32, P, P, P, P, P, SZ, P]
    lib.qlora_linear_bwd.restype = I32
    lib.qlora_time_next_gemm.argtypes = [P, P]
    lib.qlora_time_next_gemm.restype = None
    D = ctypes.c_double
    lib.qlora_adamw_step.argtypes = [P, P, P, P, P, I64, D, D, D, D, D, I64, P]
    lib.qlora_adamw_step.restype = I32
    lib.qlora_lora_merge.argtypes = [W, P, P, I32, F32, P, P]
    lib.qlora_lora_merge.restype = I32
    lib.qlora_lora_unmerge.argtypes = [P, I64, I64, P, P, I32, F32, P, P]
    lib.qlora_lora_unmerge.restype = I32
    lib.qlora_workspace_bytes_fused.argtypes = [I32, I64, I64, I64, I32, I32]
    lib.qlora_workspace_bytes_fused.restype = SZ
    lib.qlora_linear_fwd_fused.argtypes = [W, I32, P, I64, P, P, I32, F32, P, P, P, SZ, P]
    lib.qlora_linear_fwd_fused.restype = I32
    lib.qlora_linear_bwd_fused.argtypes = [W, I32, P, P, I64, P, P, I32, F32, P, P, P, P, P, SZ, P]
    lib.qlora_linear_bwd_fused.restype = I32
    lib.qlora_nf4_concat_rows.argtypes = [W, I32, W, P]
    lib.qlora_nf4_concat_rows.restype = I32
    lib.qlora_quantize.argtypes = [P, I32, I64, I64, I32, I32, P, P, P, P, P, P]
    lib.qlora_quantize.restype = I32
    lib.qlora_codebook.argtypes = [I32, ctypes.POINTER(F32), ctypes.POINTER(F32)]
    lib.qlora_codebook.restype = I32
    D = ctypes.POINTER(qlora_drop)
    lib.qlora_workspace_bytes_dropout.argtypes = [I32, I64, I64, I64, I32, I32]
    lib.qlora_workspace_bytes_dropout.restype = SZ
    lib.qlora_linear_fwd_dropout.argtypes = [W, I32, P, I64, P, P, I32, F32, D, P, P, P, SZ, P]
    lib.qlora_linear_fwd_dropout.restype = I32
    lib.qlora_linear_bwd_dropout.argtypes = [W, I32, P, P, I64, P, P, I32, F32, D, P, P, P, P, P, SZ, P]
    lib.qlora_linear_bwd_dropout.restype = I32
    lib.qlora_dropout.argtypes = [P, I32, I64, D, P, P]
    lib.qlora_dropout.restype = I32
    lib.qlora_workspace_bytes_gated.argtypes = [I32, I64, I64, I64, I32]
    lib.qlora_workspace_bytes_gated.restype = SZ
    lib.qlora_gated_fwd.argtypes = [W, P, I64, P, P, I32, F32, I32, D, P, P, P, P, SZ, P]
    lib.qlora_gated_fwd.restype = I32
    lib.qlora_gated_bwd.argtypes = [W, P, P, P, I64, P, P, I32, F32, I32, D, P, P, P, P, P, SZ, P]
    lib.qlora_gated_bwd.restype = I32
    _lib = lib
    return lib


class QloraError(RuntimeError):
    def __init__(self, status, where):
        lib = load()
        msg = lib.qlora_last_error().decode(errors="replace")
        super().__init__(f"{where}: {lib.qlora_status_string(status).decode()} ({status}): {msg}")
        self.status = status


def check(status, where):
    if status != QLORA_OK:
        raise QloraError(status, where)


# ---- same-name thin wrappers (plain integers / pointers) ------------------------

def qlora_nf4_sizes(n_rows, n_cols):
    lib = load()
    cb, nb, ng = ctypes.c_size_t(), ctypes.c_int64(), ctypes.c_int64()
    check(lib.qlora_nf4_sizes(n_rows, n_cols, ctypes.byref(cb), ctypes.byref(nb), ctypes.byref(ng)),
          "qlora_nf4_sizes")
    return cb.value, nb.value, ng.value


def qlora_nf4_codebook():
    lib = load()
    q = (ctypes.c_float * 16)()
    t = (ctypes.c_float * 15)()
    lib.qlora_nf4_codebook(q, t)
    return list(q), list(t)


def qlora_codebook(quant_type):
    lib = load()
    q = (ctypes.c_float * 16)()
    t = (ctypes.c_float * 15)()
    check(lib.qlora_codebook(quant_type, q, t), "qlora_codebook")
    return list(q), list(t)


def qlora_workspace_bytes(op, M, K, N, r):
    return load().qlora_workspace_bytes(op, M, K, N, r)


def qlora_quantize_nf4(W, w_dtype, n_rows, n_cols, codes, absmax_q, dq_scale, dq_offset,
                       absmax_f32, stream):
    return load().qlora_quantize_nf4(W, w_dtype, n_rows, n_cols, codes, absmax_q, dq_scale,
                                     dq_offset, absmax_f32, stream)


def qlora_quantize(W, w_dtype, n_rows, n_cols, quant_type, const_type, codes, absmax_q, dq_scale,
                   dq_offset, absmax, stream):
    return load().qlora_quantize(W, w_dtype, n_rows, n_cols, quant_type, const_type, codes, absmax_q,
                                 dq_scale, dq_offset, absmax, stream)


def qlora_dequantize(w, out, out_dtype, stream):
    return load().qlora_dequantize(ctypes.byref(w), out, out_dtype, stream)


def qlora_linear_fwd(w, X, M, A, B, r, alpha, Y, U_saved, workspace, workspace_bytes, stream):
    return load().qlora_linear_fwd(ctypes.byref(w), X, M, A, B, r, alpha, Y, U_saved, workspace,
                                   workspace_bytes, stream)


def qlora_linear_fwd_noalloc(w, X, M, A, B, r, alpha, Y, U_saved, stream):
    return load().qlora_linear_fwd_noalloc(ctypes.byref(w), X, M, A, B, r, alpha, Y, U_saved, stream)


def qlora_linear_bwd(w, dY, X, M, A, B, r, alpha, U_saved, dX, dA, dB, workspace,
                     workspace_bytes, stream):
    return load().qlora_linear_bwd(ctypes.byref(w), dY, X, M, A, B, r, alpha, U_saved, dX, dA, dB,
                                   workspace, workspace_bytes, stream)


def qlora_time_next_gemm(start_event, stop_event):
    load().qlora_time_next_gemm(start_event, stop_event)


def qlora_adamw_step(param, param_bf16, grad, exp_avg, exp_avg_sq, n, lr, beta1, beta2, eps,
                     weight_decay, step, stream):
    return load().qlora_adamw_step(param, param_bf16, grad, exp_avg, exp_avg_sq, n, lr, beta1, beta2,
                                   eps, weight_decay, step, stream)


def qlora_lora_merge(w, A, B, r, alpha, out, stream):
    return load().qlora_lora_merge(ctypes.byref(w), A, B, r, alpha, out, stream)


def qlora_lora_unmerge(W_merged, n_rows, n_cols, A, B, r, alpha, out, stream):
    return load().qlora_lora_unmerge(W_merged, n_rows, n_cols, A, B, r, alpha, out, stream)


def qlora_workspace_bytes_fused(op, M, K, N, r, n_parts):
    return load().qlora_workspace_bytes_fused(op, M, K, N, r, n_parts)


def qlora_linear_fwd_fused(w, n_parts, X, M, A, B, r, alpha, Y, U_saved, workspace, workspace_bytes,
                           stream):
    return load().qlora_linear_fwd_fused(ctypes.byref(w), n_parts, X, M, A, B, r, alpha, Y, U_saved,
                                         workspace, workspace_bytes, stream)


def qlora_linear_bwd_fused(w, n_parts, dY, X, M, A, B, r, alpha, U_saved, dX, dA, dB, workspace,
                           workspace_bytes, stream):
    return load().qlora_linear_bwd_fused(ctypes.byref(w), n_parts, dY, X, M, A, B, r, alpha, U_saved, dX,
                                         dA, dB, workspace, workspace_bytes, stream)


def qlora_nf4_concat_rows(parts, out, stream):
    """parts: a sequence of qlora_nf4_weight descriptors."""
    arr = (qlora_nf4_weight * len(parts))(*parts)
    return load().qlora_nf4_concat_rows(arr, len(parts), ctypes.byref(out), stream)


def qlora_workspace_bytes_dropout(op, M, K, N, r, n_parts):
    return load().qlora_workspace_bytes_dropout(op, M, K, N, r, n_parts)


def qlora_linear_fwd_dropout(w, n_parts, X, M, A, B, r, alpha, drop, Y, U_saved, workspace, workspace_bytes,
                             stream):
    return load().qlora_linear_fwd_dropout(ctypes.byref(w), n_parts, X, M, A, B, r, alpha, _drop(drop), Y, U_saved,
                                           workspace, workspace_bytes, stream)


def qlora_linear_bwd_dropout(w, n_parts, dY, X, M, A, B, r, alpha, drop, U_saved, dX, dA, dB, workspace,
                             workspace_bytes, stream):
    return load().qlora_linear_bwd_dropout(ctypes.byref(w), n_parts, dY, X, M, A, B, r, alpha, _drop(drop), U_saved,
                                           dX, dA, dB, workspace, workspace_bytes, stream)


def qlora_dropout(X, dtype, n, drop, out, stream):
    return load().qlora_dropout(X, dtype, n, _drop(drop), out, stream)


def qlora_workspace_bytes_gated(op, M, K, P, r):
    return load().qlora_workspace_bytes_gated(op, M, K, P, r)


def qlora_gated_fwd(w, X, M, A, B, r, alpha, act, drop, H, Y_saved, U_saved, workspace, workspace_bytes, stream):
    return load().qlora_gated_fwd(ctypes.byref(w), X, M, A, B, r, alpha, act, _drop(drop), H, Y_saved, U_saved,
                                  workspace, workspace_bytes, stream)


def qlora_gated_bwd(w, dH, Y_saved, X, M, A, B, r, alpha, act, drop, U_saved, dX, dA, dB, workspace,
                    workspace_bytes, stream):
    return load().qlora_gated_bwd(ctypes.byref(w), dH, Y_saved, X, M, A, B, r, alpha, act, _drop(drop), U_saved, dX,
                                  dA, dB, workspace, workspace_bytes, stream)


def _drop(drop):
    return None if drop is None else ctypes.byref(drop)
