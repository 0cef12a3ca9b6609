"""Python binding of libozaki2: FP64 matrix products emulated by Ozaki Scheme II
on the INT8 matrix cores of MI355X (gfx950).

Argument marshalling only: every step of the product runs in the HIP kernels
of ``libozaki2.so`` (built in-tree by ``python -m rns_emulated_fp64_amd.build``).
There is no CPU fallback; loading fails loudly when the library is missing.

Functions named like the C ABI (``ozaki2_dgemm`` ...) take plain integers and
device pointers exactly as ``include/ozaki2.h`` documents. ``dgemm`` is the
convenience form on torch tensors (torch provides device memory and streams).
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libozaki2.so")

FAST = 0
ACCURATE = 1
ERR_NOALLOC_LIMIT = 4  # OZAKI2_ERR_NOALLOC_LIMIT
NOALLOC_MAX_WORKSPACE = 128 << 20  # OZAKI2_NOALLOC_MAX_WORKSPACE
FAST_ORIGINAL = 2  # comparison stand-in for the original fast-mode rule (see include/ozaki2.h)
MODES = {"fast": FAST, "accurate": ACCURATE, "original": FAST_ORIGINAL}
PHASES = ("scale", "split", "gemm", "crt")

#: every symbol include/ozaki2.h declares
EXPORTS = (
    "ozaki2_dgemm", "ozaki2_workspace_size", "ozaki2_dgemm_ws", "ozaki2_dgemm_debug",
    "ozaki2_debug_workspace_size", "ozaki2_max_moduli", "ozaki2_moduli", "ozaki2_scaling_constant",
    "ozaki2_crt_weight", "ozaki2_status_string", "ozaki2_timing_enable", "ozaki2_timing_read",
    "ozaki2_timing_read_calls",
    "ozaki2_finalize", "ozaki2_crt_debug", "ozaki2_sgemm", "ozaki2_sgemm_ws", "ozaki2_sgemm_debug",
    "ozaki2_zgemm", "ozaki2_zgemm_ws", "ozaki2_zgemm_debug", "ozaki2_cgemm", "ozaki2_cgemm_ws", "ozaki2_cgemm_debug",
    "ozaki2_zgemm_workspace_size", "ozaki2_dgemm_noalloc", "ozaki2_dgemm_check", "ozaki2_check_workspace_size",
    "ozaki2_crt_check_debug", "ozaki2_zcrt_debug",
    "ozaki2_quantize_rows", "ozaki2_i8gemm", "ozaki2_i8gemm_ws", "ozaki2_i8gemm_workspace_size",
    "ozaki2_i8linear", "ozaki2_i8linear_ws", "ozaki2_i8linear_workspace_size",
    "ozaki2_xent", "ozaki2_xent_ws", "ozaki2_xent_workspace_size", "ozaki2_i8xent", "ozaki2_i8xent_ws",
    "ozaki2_i8xent_workspace_size",
    "ozaki2_xent_grad", "ozaki2_xent_grad_ws", "ozaki2_xent_grad_workspace_size",
    "ozaki2_rmsnorm_quantize", "ozaki2_i8gemm_act", "ozaki2_i8gemm_act_ws", "ozaki2_i8linear_act", "ozaki2_i8linear_act_ws",
    "ozaki2_linear", "ozaki2_linear_ws", "ozaki2_linear_workspace_size", "ozaki2_linear_grad", "ozaki2_linear_grad_ws",
    "ozaki2_linear_grad_workspace_size", "ozaki2_sample", "ozaki2_sample_ws", "ozaki2_sample_workspace_size",
    "ozaki2_i8gemm_act_workspace_size", "ozaki2_i8linear_act_workspace_size",
)

_lib = None


class Ozaki2Error(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


def lib() -> ctypes.CDLL:
    """The loaded libozaki2.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m rns_emulated_fp64_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    i64, p, i32, sz, f64 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_double
    prod = [i64, i64, i64, p, i64, p, i64, p, i64, i32, i32]
    L.ozaki2_dgemm.argtypes = prod + [p]
    L.ozaki2_dgemm.restype = i32
    L.ozaki2_dgemm_noalloc.argtypes = prod + [p]
    L.ozaki2_dgemm_noalloc.restype = i32
    L.ozaki2_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    L.ozaki2_workspace_size.restype = sz
    L.ozaki2_debug_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    L.ozaki2_debug_workspace_size.restype = sz
    L.ozaki2_dgemm_ws.argtypes = prod + [p, sz, p]
    L.ozaki2_dgemm_ws.restype = i32
    L.ozaki2_dgemm_debug.argtypes = prod + [p, sz, p, p, p, p, p, p, p]
    L.ozaki2_dgemm_debug.restype = i32
    for prefix in ("ozaki2_sgemm", "ozaki2_zgemm", "ozaki2_cgemm"):
        for suffix in ("", "_ws", "_debug"):
            getattr(L, prefix + suffix).argtypes = getattr(L, "ozaki2_dgemm" + suffix).argtypes
            getattr(L, prefix + suffix).restype = i32
    L.ozaki2_zgemm_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    L.ozaki2_zgemm_workspace_size.restype = sz
    L.ozaki2_crt_debug.argtypes = [i64, i64, i32, p, p, p, p, i64, p, sz, p]
    L.ozaki2_crt_debug.restype = i32
    L.ozaki2_zcrt_debug.argtypes = L.ozaki2_crt_debug.argtypes
    L.ozaki2_zcrt_debug.restype = i32
    L.ozaki2_dgemm_check.argtypes = prod + [p, sz, p, p]
    L.ozaki2_dgemm_check.restype = i32
    L.ozaki2_check_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    L.ozaki2_check_workspace_size.restype = sz
    L.ozaki2_crt_check_debug.argtypes = [i64, i64, i32, p, p, p, p, i64, p, p, sz, p]
    L.ozaki2_crt_check_debug.restype = i32
    L.ozaki2_max_moduli.argtypes = []
    L.ozaki2_max_moduli.restype = i32
    L.ozaki2_moduli.argtypes = [i32, p]
    L.ozaki2_moduli.restype = i32
    L.ozaki2_scaling_constant.argtypes = [i32, p]
    L.ozaki2_scaling_constant.restype = i32
    L.ozaki2_crt_weight.argtypes = [i32, i32, p, i32]
    L.ozaki2_crt_weight.restype = i32
    L.ozaki2_status_string.argtypes = [i32]
    L.ozaki2_status_string.restype = ctypes.c_char_p
    L.ozaki2_timing_enable.argtypes = [i32, i32]
    L.ozaki2_timing_enable.restype = i32
    L.ozaki2_timing_read.argtypes = [p, p]
    L.ozaki2_timing_read.restype = i32
    L.ozaki2_timing_read_calls.argtypes = [p, i32, p]
    L.ozaki2_timing_read_calls.restype = i32
    L.ozaki2_quantize_rows.argtypes = [i64, i64, p, i64, i32, p, i64, p, p]
    L.ozaki2_quantize_rows.restype = i32
    i8 = [i64, i64, i64, p, i64, p, p, i64, p, p, p, i64, i32]
    L.ozaki2_i8gemm.argtypes = i8 + [p]
    L.ozaki2_i8gemm_ws.argtypes = i8 + [p, sz, p]
    i8 = [i64, i64, i64, p, i64, i32, p, i64, p, p, p, i64, i32]
    L.ozaki2_i8linear.argtypes = i8 + [p]
    L.ozaki2_i8linear_ws.argtypes = i8 + [p, sz, p]
    i8 = [i64, i64, i64, p, i64, p, p, i64, p, p, i32, p, i64, p, i64, i32]
    L.ozaki2_i8gemm_act.argtypes = i8 + [p]
    L.ozaki2_i8gemm_act_ws.argtypes = i8 + [p, sz, p]
    i8 = [i64, i64, i64, p, i64, i32, p, i64, p, p, i32, p, i64, p, i64, i32]
    L.ozaki2_i8linear_act.argtypes = i8 + [p]
    L.ozaki2_i8linear_act_ws.argtypes = i8 + [p, sz, p]
    for name in ("ozaki2_i8gemm_act", "ozaki2_i8linear_act"):
        getattr(L, name).restype = i32
        getattr(L, name + "_ws").restype = i32
        getattr(L, name + "_workspace_size").argtypes = [i64, i64, i64]
        getattr(L, name + "_workspace_size").restype = sz
    for name in ("ozaki2_i8gemm", "ozaki2_i8linear"):
        getattr(L, name).restype = i32
        getattr(L, name + "_ws").restype = i32
        getattr(L, name + "_workspace_size").argtypes = [i64, i64, i64]
        getattr(L, name + "_workspace_size").restype = sz
    xent = [i64, i64, i64, p, i64, p, i64, i32, p, i64, p, p]
    L.ozaki2_xent.argtypes = xent + [p]
    L.ozaki2_xent_ws.argtypes = xent + [p, sz, p]
    xent = [i64, i64, i64, p, i64, p, p, i64, p, p, i64, p, p]
    L.ozaki2_i8xent.argtypes = xent + [p]
    L.ozaki2_i8xent_ws.argtypes = xent + [p, sz, p]
    xent = [i64, i64, i64, p, i64, p, i64, i32, p, i64, p, p, p, i64, p, i64]
    L.ozaki2_xent_grad.argtypes = xent + [p]
    L.ozaki2_xent_grad_ws.argtypes = xent + [p, sz, p]
    for name in ("ozaki2_xent", "ozaki2_i8xent", "ozaki2_xent_grad"):
        getattr(L, name).restype = i32
        getattr(L, name + "_ws").restype = i32
    L.ozaki2_xent_workspace_size.argtypes = [i64, i64, i64]
    L.ozaki2_xent_workspace_size.restype = sz
    L.ozaki2_i8xent_workspace_size.argtypes = [i64, i64, i64]
    L.ozaki2_i8xent_workspace_size.restype = sz
    L.ozaki2_xent_grad_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    L.ozaki2_xent_grad_workspace_size.restype = sz
    lin = [i64, i64, i64, p, i64, p, i64, i32, p, i32, p, i64, p, i64, i32, p, i64]
    L.ozaki2_linear.argtypes = lin + [p]
    L.ozaki2_linear_ws.argtypes = lin + [p, sz, p]
    lin = [i64, i64, i64, p, i64, p, i64, p, i64, i32, i32, p, i64, p, i64, p, i64, p]
    L.ozaki2_linear_grad.argtypes = lin + [p]
    L.ozaki2_linear_grad_ws.argtypes = lin + [p, sz, p]
    for name in ("ozaki2_linear", "ozaki2_linear_grad"):
        getattr(L, name).restype = i32
        getattr(L, name + "_ws").restype = i32
    L.ozaki2_linear_workspace_size.argtypes = [i64, i64, i64]
    L.ozaki2_linear_workspace_size.restype = sz
    L.ozaki2_linear_grad_workspace_size.argtypes = [i64, i64, i64, i32, i32, i32]
    L.ozaki2_linear_grad_workspace_size.restype = sz
    smp = [i64, i64, p, i64, i32, p, f64, p, i64, p, f64, p, f64, p, p, p]
    L.ozaki2_sample.argtypes = smp + [p]
    L.ozaki2_sample.restype = i32
    L.ozaki2_sample_ws.argtypes = smp + [p, sz, p]
    L.ozaki2_sample_ws.restype = i32
    L.ozaki2_sample_workspace_size.argtypes = [i64, i64]
    L.ozaki2_sample_workspace_size.restype = sz
    L.ozaki2_rmsnorm_quantize.argtypes = [i64, i64, p, i64, i32, p, i64, p, f64, p, i64, p, p, i64, p]
    L.ozaki2_rmsnorm_quantize.restype = i32
    L.ozaki2_finalize.argtypes = []
    L.ozaki2_finalize.restype = None
    _lib = L
    return L


# ---- same names as the C ABI: plain integers / device pointers ----------------
def ozaki2_dgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream=0) -> int:
    return lib().ozaki2_dgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream)


def ozaki2_dgemm_noalloc(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream=0) -> int:
    return lib().ozaki2_dgemm_noalloc(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream)


def ozaki2_dgemm_check(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes, flags,
                       stream=0) -> int:
    return lib().ozaki2_dgemm_check(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                    flags, stream)


def ozaki2_check_workspace_size(m, n, k, num_moduli, mode) -> int:
    return lib().ozaki2_check_workspace_size(m, n, k, num_moduli, mode)


def ozaki2_crt_check_debug(m, n, num_moduli, residues, e, f, C, ldc, flags, workspace, workspace_bytes,
                           stream=0) -> int:
    return lib().ozaki2_crt_check_debug(m, n, num_moduli, residues, e, f, C, ldc, flags, workspace, workspace_bytes,
                                        stream)


def ozaki2_workspace_size(m, n, k, num_moduli, mode) -> int:
    return lib().ozaki2_workspace_size(m, n, k, num_moduli, mode)


def ozaki2_debug_workspace_size(m, n, k, num_moduli, mode) -> int:
    return lib().ozaki2_debug_workspace_size(m, n, k, num_moduli, mode)


def ozaki2_dgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_dgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace,
                                 workspace_bytes, stream)


def ozaki2_dgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                       e_out, f_out, resA_out, resB_out, prod_out, red_out, stream=0) -> int:
    return lib().ozaki2_dgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace,
                                    workspace_bytes, e_out, f_out, resA_out, resB_out, prod_out, red_out, stream)


def ozaki2_sgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream=0) -> int:
    return lib().ozaki2_sgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream)


def ozaki2_sgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_sgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                 stream)


def ozaki2_sgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                       e_out, f_out, resA_out, resB_out, prod_out, red_out, stream=0) -> int:
    return lib().ozaki2_sgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                    e_out, f_out, resA_out, resB_out, prod_out, red_out, stream)


def ozaki2_zgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode=FAST, stream=0) -> int:
    return lib().ozaki2_zgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream)


def ozaki2_zgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_zgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                 stream)


def ozaki2_zgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                       e_out, f_out, resA_out, resB_out, prod_out, red_out, stream=0) -> int:
    return lib().ozaki2_zgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                    e_out, f_out, resA_out, resB_out, prod_out, red_out, stream)


def ozaki2_cgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode=FAST, stream=0) -> int:
    return lib().ozaki2_cgemm(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, stream)


def ozaki2_cgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_cgemm_ws(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                 stream)


def ozaki2_cgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                       e_out, f_out, resA_out, resB_out, prod_out, red_out, stream=0) -> int:
    return lib().ozaki2_cgemm_debug(m, n, k, A, lda, B, ldb, C, ldc, num_moduli, mode, workspace, workspace_bytes,
                                    e_out, f_out, resA_out, resB_out, prod_out, red_out, stream)


def ozaki2_zgemm_workspace_size(m, n, k, num_moduli, debug=False) -> int:
    return lib().ozaki2_zgemm_workspace_size(m, n, k, num_moduli, 1 if debug else 0)


def ozaki2_quantize_rows(t, k, X, ldx, xtype, Q, ldq, scale, stream=0) -> int:
    return lib().ozaki2_quantize_rows(t, k, X, ldx, xtype, Q, ldq, scale, stream)


def ozaki2_i8gemm(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, C, ldc, ctype, stream=0) -> int:
    return lib().ozaki2_i8gemm(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, C, ldc, ctype, stream)


def ozaki2_i8gemm_ws(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, C, ldc, ctype, workspace, workspace_bytes,
                     stream=0) -> int:
    return lib().ozaki2_i8gemm_ws(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, C, ldc, ctype, workspace,
                                  workspace_bytes, stream)


def ozaki2_i8gemm_workspace_size(t, n, k) -> int:
    return lib().ozaki2_i8gemm_workspace_size(t, n, k)


def ozaki2_i8linear(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, C, ldc, ctype, stream=0) -> int:
    return lib().ozaki2_i8linear(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, C, ldc, ctype, stream)


def ozaki2_i8linear_ws(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, C, ldc, ctype, workspace, workspace_bytes,
                       stream=0) -> int:
    return lib().ozaki2_i8linear_ws(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, C, ldc, ctype, workspace,
                                    workspace_bytes, stream)


def ozaki2_i8linear_workspace_size(t, n, k) -> int:
    return lib().ozaki2_i8linear_workspace_size(t, n, k)


def ozaki2_xent(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, loss, lse, stream=0) -> int:
    return lib().ozaki2_xent(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, loss, lse, stream)


def ozaki2_xent_ws(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, loss, lse, workspace, workspace_bytes,
                   stream=0) -> int:
    return lib().ozaki2_xent_ws(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, loss, lse, workspace,
                                workspace_bytes, stream)


def ozaki2_xent_workspace_size(t, v, d) -> int:
    return lib().ozaki2_xent_workspace_size(t, v, d)


def ozaki2_i8xent(t, v, k, A, lda, a_scale, B, ldb, b_scale, targets, ignore_index, loss, lse, stream=0) -> int:
    return lib().ozaki2_i8xent(t, v, k, A, lda, a_scale, B, ldb, b_scale, targets, ignore_index, loss, lse, stream)


def ozaki2_i8xent_ws(t, v, k, A, lda, a_scale, B, ldb, b_scale, targets, ignore_index, loss, lse, workspace,
                     workspace_bytes, stream=0) -> int:
    return lib().ozaki2_i8xent_ws(t, v, k, A, lda, a_scale, B, ldb, b_scale, targets, ignore_index, loss, lse,
                                  workspace, workspace_bytes, stream)


def ozaki2_i8xent_workspace_size(t, v, k) -> int:
    return lib().ozaki2_i8xent_workspace_size(t, v, k)


def ozaki2_xent_grad(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, lse, grad_loss, dX, lddx, dW, lddw,
                     stream=0) -> int:
    return lib().ozaki2_xent_grad(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, lse, grad_loss, dX, lddx, dW,
                                  lddw, stream)


def ozaki2_xent_grad_ws(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, lse, grad_loss, dX, lddx, dW, lddw,
                        workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_xent_grad_ws(t, v, d, X, ldx, W, ldw, type, targets, ignore_index, lse, grad_loss, dX, lddx,
                                     dW, lddw, workspace, workspace_bytes, stream)


def ozaki2_xent_grad_workspace_size(t, v, d, want_dx=True, want_dw=True) -> int:
    return lib().ozaki2_xent_grad_workspace_size(t, v, d, 1 if want_dx else 0, 1 if want_dw else 0)


def ozaki2_i8gemm_act(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                      stream=0) -> int:
    return lib().ozaki2_i8gemm_act(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                                   stream)


def ozaki2_i8gemm_act_ws(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype, workspace,
                         workspace_bytes, stream=0) -> int:
    return lib().ozaki2_i8gemm_act_ws(t, n, k, A, lda, a_scale, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                                      workspace, workspace_bytes, stream)


def ozaki2_i8linear_act(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                        stream=0) -> int:
    return lib().ozaki2_i8linear_act(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                                     stream)


def ozaki2_i8linear_act_ws(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype, workspace,
                           workspace_bytes, stream=0) -> int:
    return lib().ozaki2_i8linear_act_ws(t, n, k, X, ldx, xtype, B, ldb, b_scale, bias, activation, residual, ldr, C, ldc, ctype,
                                        workspace, workspace_bytes, stream)


def ozaki2_i8gemm_act_workspace_size(t, n, k) -> int:
    return lib().ozaki2_i8gemm_act_workspace_size(t, n, k)


def ozaki2_i8linear_act_workspace_size(t, n, k) -> int:
    return lib().ozaki2_i8linear_act_workspace_size(t, n, k)


def ozaki2_linear(t, n, k, X, ldx, W, ldw, type, bias, activation, residual, ldr, Y, ldy, ytype, Z, ldz, stream=0) -> int:
    return lib().ozaki2_linear(t, n, k, X, ldx, W, ldw, type, bias, activation, residual, ldr, Y, ldy, ytype, Z, ldz, stream)


def ozaki2_linear_ws(t, n, k, X, ldx, W, ldw, type, bias, activation, residual, ldr, Y, ldy, ytype, Z, ldz, workspace,
                     workspace_bytes, stream=0) -> int:
    return lib().ozaki2_linear_ws(t, n, k, X, ldx, W, ldw, type, bias, activation, residual, ldr, Y, ldy, ytype, Z, ldz,
                                  workspace, workspace_bytes, stream)


def ozaki2_linear_workspace_size(t, n, k) -> int:
    return lib().ozaki2_linear_workspace_size(t, n, k)


def ozaki2_linear_grad(t, n, k, dY, lddy, X, ldx, W, ldw, type, activation, Z, ldz, dX, lddx, dW, lddw, dbias,
                       stream=0) -> int:
    return lib().ozaki2_linear_grad(t, n, k, dY, lddy, X, ldx, W, ldw, type, activation, Z, ldz, dX, lddx, dW, lddw, dbias,
                                    stream)


def ozaki2_linear_grad_ws(t, n, k, dY, lddy, X, ldx, W, ldw, type, activation, Z, ldz, dX, lddx, dW, lddw, dbias, workspace,
                          workspace_bytes, stream=0) -> int:
    return lib().ozaki2_linear_grad_ws(t, n, k, dY, lddy, X, ldx, W, ldw, type, activation, Z, ldz, dX, lddx, dW, lddw, dbias,
                                       workspace, workspace_bytes, stream)


def ozaki2_linear_grad_workspace_size(t, n, k, want_dx=True, want_dw=True, want_dbias=True) -> int:
    return lib().ozaki2_linear_grad_workspace_size(t, n, k, 1 if want_dx else 0, 1 if want_dw else 0, 1 if want_dbias else 0)


def ozaki2_sample(t, v, logits, ldl, type, u, temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p, min_ps, tokens,
                  logprobs, stream=0) -> int:
    return lib().ozaki2_sample(t, v, logits, ldl, type, u, temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p,
                               min_ps, tokens, logprobs, stream)


def ozaki2_sample_ws(t, v, logits, ldl, type, u, temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p, min_ps, tokens,
                     logprobs, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_sample_ws(t, v, logits, ldl, type, u, temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p,
                                  min_ps, tokens, logprobs, workspace, workspace_bytes, stream)


def ozaki2_sample_workspace_size(t, v) -> int:
    return lib().ozaki2_sample_workspace_size(t, v)


def ozaki2_rmsnorm_quantize(t, k, X, ldx, type, residual, ldr, weight, eps, Q, ldq, scale, sum, lds, stream=0) -> int:
    return lib().ozaki2_rmsnorm_quantize(t, k, X, ldx, type, residual, ldr, weight, eps, Q, ldq, scale, sum, lds, stream)


def ozaki2_crt_debug(m, n, num_moduli, residues, e, f, C, ldc, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_crt_debug(m, n, num_moduli, residues, e, f, C, ldc, workspace, workspace_bytes, stream)


def ozaki2_zcrt_debug(m, n, num_moduli, residues, e, f, C, ldc, workspace, workspace_bytes, stream=0) -> int:
    return lib().ozaki2_zcrt_debug(m, n, num_moduli, residues, e, f, C, ldc, workspace, workspace_bytes, stream)


def ozaki2_max_moduli() -> int:
    return lib().ozaki2_max_moduli()


def ozaki2_moduli(num_moduli: int) -> list[int]:
    out = (ctypes.c_int32 * max(num_moduli, 1))()
    st = lib().ozaki2_moduli(num_moduli, out)
    if st:
        raise Ozaki2Error(st, "ozaki2_moduli")
    return list(out)[:num_moduli]


def ozaki2_scaling_constant(num_moduli: int) -> float:
    out = ctypes.c_double()
    st = lib().ozaki2_scaling_constant(num_moduli, ctypes.byref(out))
    if st:
        raise Ozaki2Error(st, "ozaki2_scaling_constant")
    return out.value


def ozaki2_crt_weight(num_moduli: int, l: int) -> int:
    limbs = (ctypes.c_uint32 * 8)()
    used = lib().ozaki2_crt_weight(num_moduli, l, limbs, 8)
    if used < 0:
        raise Ozaki2Error(used, "ozaki2_crt_weight")
    return sum(int(limbs[i]) << (32 * i) for i in range(used))


def status_string(status: int) -> str:
    return lib().ozaki2_status_string(status).decode()


def ozaki2_timing_enable(max_calls: int, all_phases: bool = False) -> None:
    st = lib().ozaki2_timing_enable(max_calls, 1 if all_phases else 0)
    if st:
        raise Ozaki2Error(st, "ozaki2_timing_enable")


def ozaki2_timing_read() -> tuple[dict, int]:
    ms = (ctypes.c_double * 4)()
    calls = ctypes.c_int()
    st = lib().ozaki2_timing_read(ms, ctypes.byref(calls))
    if st:
        raise Ozaki2Error(st, "ozaki2_timing_read")
    return dict(zip(PHASES, list(ms))), calls.value


def ozaki2_timing_read_calls(max_calls: int) -> list:
    """Per timed call, a dict of milliseconds per phase; clears the record."""
    ms = (ctypes.c_double * (4 * max(max_calls, 1)))()
    calls = ctypes.c_int()
    st = lib().ozaki2_timing_read_calls(ms, max_calls, ctypes.byref(calls))
    if st:
        raise Ozaki2Error(st, "ozaki2_timing_read_calls")
    return [dict(zip(PHASES, list(ms[4 * c:4 * c + 4]))) for c in range(calls.value)]


def ozaki2_finalize() -> None:
    lib().ozaki2_finalize()


# ---- torch convenience -------------------------------------------------------
def _mode(mode) -> int:
    return MODES[mode] if isinstance(mode, str) else int(mode)


def dgemm(A, B, num_moduli: int = 16, mode="fast", out=None, workspace=None):
    """C = A @ B for float64 CUDA (HIP) tensors in row-major layout.

    Row-major C = A B is column-major C^T = B^T A^T, so the library is called
    with the operands swapped; the scaling is symmetric in the two operands.
    ``out`` (optional) must be a contiguous (m, n) tensor of the same dtype on
    the same device; ``workspace`` (optional) a device tensor of at least
    ``ozaki2_workspace_size`` bytes.
    """
    return _gemm(A, B, num_moduli, mode, out, workspace, "d")


def sgemm(A, B, num_moduli: int = 8, mode="fast", out=None, workspace=None):
    """C = A @ B for float32 CUDA (HIP) tensors (ozaki2_sgemm), as dgemm."""
    return _gemm(A, B, num_moduli, mode, out, workspace, "s")


def zgemm(A, B, num_moduli: int = 16, mode="fast", out=None, workspace=None):
    """C = A @ B for complex128 CUDA (HIP) tensors (ozaki2_zgemm, fast mode), as
    dgemm; a complex tensor's storage is the interleaved (re, im) layout the
    library takes. ``workspace`` needs ``ozaki2_zgemm_workspace_size`` bytes."""
    return _gemm(A, B, num_moduli, mode, out, workspace, "z")


def cgemm(A, B, num_moduli: int = 16, mode="fast", out=None, workspace=None):
    """C = A @ B for complex64 CUDA (HIP) tensors (ozaki2_cgemm), as zgemm."""
    return _gemm(A, B, num_moduli, mode, out, workspace, "c")


_KINDS = {  # dtype name, plain entry, workspace entry
    "d": ("float64", "ozaki2_dgemm"),
    "s": ("float32", "ozaki2_sgemm"),
    "z": ("complex128", "ozaki2_zgemm"),
    "c": ("complex64", "ozaki2_cgemm"),
}


def _gemm(A, B, num_moduli, mode, out, workspace, kind):
    import torch

    dname, entry = _KINDS[kind]
    dt = getattr(torch, dname)
    if A.dtype != dt or B.dtype != dt or not A.is_cuda or not B.is_cuda or A.device != B.device:
        raise TypeError(f"A and B must be {dt} tensors on the same GPU")
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError("shapes do not multiply")
    A = A.contiguous()
    B = B.contiguous()
    m, k = A.shape
    n = B.shape[1]
    if out is None:
        C = torch.empty((m, n), dtype=dt, device=A.device)
    else:
        if out.dtype != dt or out.device != A.device or tuple(out.shape) != (m, n) or not out.is_contiguous():
            raise ValueError(f"out must be a contiguous ({m}, {n}) {dt} tensor on {A.device}")
        C = out
    md = _mode(mode)
    plain, ws_form = globals()[entry], globals()[entry + "_ws"]
    if workspace is not None and (not workspace.is_cuda or workspace.device != A.device):
        raise ValueError(f"workspace must be a tensor on {A.device}")
    # the library launches on the current device: make it the operands' one
    with torch.cuda.device(A.device):
        stream = torch.cuda.current_stream(A.device).cuda_stream
        if workspace is None:
            st = plain(n, m, k, B.data_ptr(), max(n, 1), A.data_ptr(), max(k, 1), C.data_ptr(), max(n, 1),
                       num_moduli, md, stream)
        else:
            st = ws_form(n, m, k, B.data_ptr(), max(n, 1), A.data_ptr(), max(k, 1), C.data_ptr(), max(n, 1),
                         num_moduli, md, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                         stream)
    if st:
        raise Ozaki2Error(st, entry)
    return C


# ---- INT8 products with scales -----------------------------------------------
BF16, FP16, FP32 = 0, 1, 2  # enum ozaki2_type
_types = {}  # torch dtype -> enum ozaki2_type, filled on the first call
_torch = None


def _load_torch():
    global _torch
    import torch

    _types.update({torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32})
    _torch = torch
    return torch


def _type_of(dtype, what):
    kind = _types.get(dtype)
    if kind is None:
        raise TypeError(f"{what} must be bfloat16, float16 or float32, not {dtype}")
    return kind


def _rows(x, what):
    """A matrix whose rows are contiguous (a copy if they are not), and its pitch."""
    if x.dim() != 2:
        raise ValueError(f"{what} must be a matrix")
    (t, k), (pitch, step) = x.shape, x.stride()
    if step == 1 and pitch >= k > 0:
        return x, pitch
    if k > 1 and step != 1 or t > 1 and pitch < k:
        return x.contiguous(), max(k, 1)
    return x, max(pitch if t > 1 else k, 1)


def _vector(x, n, dtype, device, what):
    """A contiguous vector of n values on a device."""
    if x.dtype != dtype or x.device != device or x.numel() != n:
        raise ValueError(f"{what} must hold {n} {dtype} values on {device}")
    return x if x.is_contiguous() else x.contiguous()


def _call(fn, name, device, *args):
    """fn(*args, stream) on the current stream of a device, which the library needs to be the current one."""
    index = device.index
    if index == _torch._C._cuda_getDevice():
        st = fn(*args, _torch._C._cuda_getCurrentRawStream(index))
    else:
        with _torch.cuda.device(device):
            st = fn(*args, _torch._C._cuda_getCurrentRawStream(index))
    if st:
        raise Ozaki2Error(st, name)


def _workspace(size, given, device):
    """The caller's workspace or a new one from torch's allocator (which may be captured), its pointer and bytes."""
    torch = _torch or _load_torch()
    if given is not None:
        if given.device != device:
            raise ValueError(f"workspace must be a tensor on {device}")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if size == 0:
        return None, None, 0
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), size


def _product_out(t, n, dtype, out, device, like):
    """The caller's output or a new one on the device of ``like``, and its pitch."""
    if out is None:
        # (a third less time than torch.empty with a dtype and a device)
        return like.new_empty(t, n) if like.dtype == dtype else like.new_empty(t, n, dtype=dtype), max(n, 1)
    if out.dtype != dtype or out.device != device or tuple(out.shape) != (t, n) or n > 1 and out.stride(1) != 1 \
            or t > 1 and out.stride(0) < n:
        raise ValueError(f"out must be a ({t}, {n}) {dtype} tensor on {device} with contiguous rows")
    return out, max(out.stride(0) if t > 1 else n, 1)


def _overlap(a, b):
    """Whether the memory that two matrices reach from first to last element overlaps."""
    def span(x):
        last = sum((n - 1) * s for n, s in zip(x.shape, x.stride()))
        return x.data_ptr(), x.data_ptr() + (last + 1) * x.element_size()
    if not a.numel() or not b.numel():
        return False
    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


def quantize_rows(X):
    """Rows of X (float32, float16 or bfloat16) as int8 with a binary32 scale each: (q, scale) with
    scale = max|x| / 127 and q = rint(x / scale), with the binary32 roundings that include/ozaki2.h states
    (ozaki2_quantize_rows)."""
    torch = _torch or _load_torch()
    xtype = _type_of(X.dtype, "X")
    device = X.device
    if device.type != "cuda":
        raise TypeError("X must be on a GPU")
    X, ldx = _rows(X, "X")
    t, k = X.shape
    q = torch.empty((t, k), dtype=torch.int8, device=device)
    scale = torch.empty(t, dtype=torch.float32, device=device)
    _call(lib().ozaki2_quantize_rows, "ozaki2_quantize_rows", device, t, k, X.data_ptr(), ldx, xtype, q.data_ptr(),
          max(k, 1), scale.data_ptr())
    return q, scale


#: names of the activations, as enum ozaki2_activation numbers them
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError(f"activation must be one of {list(ACTIVATIONS)}, not {name!r}")
    return act


def _residual(residual, t, n, dtype, device):
    """A residual's tensor (a copy if its rows are not contiguous), pointer and pitch."""
    if residual is None:
        return None, None, 0
    if residual.dtype != dtype or residual.device != device or tuple(residual.shape) != (t, n):
        raise ValueError(f"residual must be a ({t}, {n}) {dtype} tensor on {device}")
    residual, ldr = _rows(residual, "residual")
    return residual, residual.data_ptr(), ldr


def i8gemm(A, B, a_scale, b_scale, bias=None, out_dtype=None, out=None, workspace=None, activation=None, residual=None):
    """C[t, n] = act((sum_k A[t, k] B[n, k]) * a_scale[t] * b_scale[n] + bias[n]) + residual[t, n] for int8 A (t, k) and
    B (n, k), the layout of a linear layer (ozaki2_i8gemm_ws; with an activation, a name from ACTIVATIONS, or a residual
    ozaki2_i8gemm_act_ws). The scales and the bias are float32; ``out_dtype`` is bfloat16 (default), float16 or
    float32; the residual has that dtype and shares no memory with ``out``, nor do A and B; ``workspace`` (optional) a tensor of
    ``ozaki2_i8gemm_workspace_size`` bytes (with an activation or a residual ``ozaki2_i8gemm_act_workspace_size`` bytes are faster
    for a few rows and a long k)."""
    torch = _torch or _load_torch()
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else torch.bfloat16
    ctype = _type_of(dt, "out_dtype")
    act = _activation(activation)
    device = A.device
    if A.dtype != torch.int8 or B.dtype != torch.int8 or device.type != "cuda" or B.device != device:
        raise TypeError("A and B must be int8 tensors on the same GPU")
    A, lda = _rows(A, "A")
    B, ldb = _rows(B, "B")
    t, k = A.shape
    n = B.shape[0]
    if B.shape[1] != k:
        raise ValueError("A and B must have the same number of columns")
    a_scale = _vector(a_scale, t, torch.float32, device, "a_scale")
    b_scale = _vector(b_scale, n, torch.float32, device, "b_scale")
    if bias is not None:
        bias = _vector(bias, n, torch.float32, device, "bias")
    C, ldc = _product_out(t, n, dt, out, device, A)
    L = lib()
    if act or residual is not None:
        ws, wp, wb = _workspace(L.ozaki2_i8gemm_act_workspace_size(t, n, k), workspace, device)
        residual, rp, ldr = _residual(residual, t, n, dt, device)
        _call(L.ozaki2_i8gemm_act_ws, "ozaki2_i8gemm_act_ws", device, t, n, k, A.data_ptr(), lda, a_scale.data_ptr(),
              B.data_ptr(), ldb, b_scale.data_ptr(), None if bias is None else bias.data_ptr(), act, rp, ldr, C.data_ptr(), ldc,
              ctype, wp, wb)
        return C
    ws, wp, wb = _workspace(L.ozaki2_i8gemm_workspace_size(t, n, k), workspace, device)
    _call(L.ozaki2_i8gemm_ws, "ozaki2_i8gemm_ws", device, t, n, k, A.data_ptr(), lda, a_scale.data_ptr(), B.data_ptr(),
          ldb, b_scale.data_ptr(), None if bias is None else bias.data_ptr(), C.data_ptr(), ldc, ctype, wp, wb)
    return C


def i8linear(X, B, b_scale, bias=None, out_dtype=None, out=None, workspace=None, activation=None, residual=None):
    """A linear layer with int8 weights B (n, k) and a scale per channel: the rows of X (t, k; bfloat16, float16 or
    float32) are quantised as quantize_rows does and multiplied as i8gemm does, bit for bit (ozaki2_i8linear_ws,
    ozaki2_i8linear_act_ws). The result has X's dtype unless ``out_dtype`` or ``out`` says otherwise, and so has the
    residual."""
    torch = _torch or _load_torch()
    xtype = _type_of(X.dtype, "X")
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else X.dtype
    ctype = _type_of(dt, "out_dtype")
    act = _activation(activation)
    device = X.device
    if B.dtype != torch.int8 or device.type != "cuda" or B.device != device:
        raise TypeError("X and int8 B must be on the same GPU")
    X, ldx = _rows(X, "X")
    B, ldb = _rows(B, "B")
    t, k = X.shape
    n = B.shape[0]
    if B.shape[1] != k:
        raise ValueError("X and B must have the same number of columns")
    b_scale = _vector(b_scale, n, torch.float32, device, "b_scale")
    if bias is not None:
        bias = _vector(bias, n, torch.float32, device, "bias")
    C, ldc = _product_out(t, n, dt, out, device, X)
    L = lib()
    if act or residual is not None:
        ws, wp, wb = _workspace(L.ozaki2_i8linear_act_workspace_size(t, n, k), workspace, device)
        residual, rp, ldr = _residual(residual, t, n, dt, device)
        _call(L.ozaki2_i8linear_act_ws, "ozaki2_i8linear_act_ws", device, t, n, k, X.data_ptr(), ldx, xtype, B.data_ptr(), ldb,
              b_scale.data_ptr(), None if bias is None else bias.data_ptr(), act, rp, ldr, C.data_ptr(), ldc, ctype, wp, wb)
        return C
    ws, wp, wb = _workspace(L.ozaki2_i8linear_workspace_size(t, n, k), workspace, device)
    _call(L.ozaki2_i8linear_ws, "ozaki2_i8linear_ws", device, t, n, k, X.data_ptr(), ldx, xtype, B.data_ptr(), ldb,
          b_scale.data_ptr(), None if bias is None else bias.data_ptr(), C.data_ptr(), ldc, ctype, wp, wb)
    return C


def rmsnorm_quantize(X, weight=None, residual=None, eps=1e-6, sum_out=None):
    """The root-mean-square norm in front of a quantised layer, with the residual's addition (ozaki2_rmsnorm_quantize):
    (q, scale, sum) with h = X + residual, y = h / sqrt(mean(h^2) + eps) * weight, and y as int8 with a float32 scale per
    row as quantize_rows gives it, the operands of i8gemm. ``weight`` is float32 (k,), ones if None. ``sum`` is h in X's
    dtype, or None without a residual; ``sum_out`` (optional) the tensor it is written to, which may be ``residual`` or
    ``X`` itself. Autograd does not see the call."""
    torch = _torch or _load_torch()
    xtype = _type_of(X.dtype, "X")
    device = X.device
    if device.type != "cuda":
        raise TypeError("X must be on a GPU")
    given_x, given_r = X, residual
    X, ldx = _rows(X, "X")
    t, k = X.shape
    if weight is not None:
        weight = _vector(weight, k, torch.float32, device, "weight")
    ldr = lds = 0
    if residual is not None:
        if residual.dtype != X.dtype or residual.device != device or residual.shape != X.shape:
            raise ValueError(f"residual must be a ({t}, {k}) {X.dtype} tensor on {device}")
        residual, ldr = _rows(residual, "residual")
    total = None
    if residual is not None or sum_out is not None:
        total, lds = _product_out(t, k, X.dtype, sum_out, device, X)
        if sum_out is not None:
            # element for element over an input, or apart from it (a row that stands for several cannot be written)
            for x in (given_x, given_r):
                if x is not None and _overlap(total, x) and (
                        total.data_ptr() != x.data_ptr()
                        or any(n > 1 and a != b for n, a, b in zip(x.shape, x.stride(), total.stride()))):
                    raise ValueError("sum_out must be X or residual itself or not overlap them")
    q = X.new_empty(t, k, dtype=torch.int8)
    scale = X.new_empty(t, dtype=torch.float32)
    _call(lib().ozaki2_rmsnorm_quantize, "ozaki2_rmsnorm_quantize", device, t, k, X.data_ptr(), ldx, xtype,
          None if residual is None else residual.data_ptr(), ldr, None if weight is None else weight.data_ptr(), eps,
          q.data_ptr(), max(k, 1), scale.data_ptr(), None if total is None else total.data_ptr(), lds)
    return q, scale, total


# ---- 16-bit layers -----------------------------------------------------------
def _layer_operands(X, W):
    torch = _torch or _load_torch()
    device = X.device
    if device.type != "cuda" or W.device != device:
        raise TypeError("X and W must be on the same GPU")
    kind = _xent_type(X, W)
    X, ldx = _rows(X, "X")
    W, ldw = _rows(W, "W")
    t, k = X.shape
    if W.shape[1] != k:
        raise ValueError("X and W must have the same number of columns")
    return device, kind, t, W.shape[0], k, X, ldx, W, ldw


def linear(X, W, bias=None, activation=None, residual=None, out_dtype=None, out=None, want_pre=False, workspace=None):
    """A linear layer with what follows it: (Y, Z) with Z = X @ W.T + bias and Y = act(Z) + residual (ozaki2_linear_ws).
    X (t, k) and W (n, k) are bfloat16 or float16, the bias float32 (n,), the activation a name from ACTIVATIONS. Y has
    X's dtype unless ``out_dtype`` or ``out`` says float32, and the residual (t, n) has Y's and shares no memory with
    ``out``, nor do X and W. Z, in X's dtype, is what linear_grad needs of a layer with an activation; it is None unless ``want_pre``.
    Autograd does not see the call."""
    torch = _torch or _load_torch()
    device, kind, t, n, k, X, ldx, W, ldw = _layer_operands(X, W)
    act = _activation(activation)
    dt = out_dtype if out_dtype is not None else out.dtype if out is not None else X.dtype
    if dt != X.dtype and dt != torch.float32:
        raise TypeError(f"the result must be {X.dtype} or float32, not {dt}")
    if bias is not None:
        bias = _vector(bias, n, torch.float32, device, "bias")
    residual, rp, ldr = _residual(residual, t, n, dt, device)
    Y, ldy = _product_out(t, n, dt, out, device, X)
    Z = X.new_empty(t, n) if want_pre else None
    L = lib()
    ws, wp, wb = _workspace(L.ozaki2_linear_workspace_size(t, n, k), workspace, device)
    _call(L.ozaki2_linear_ws, "ozaki2_linear_ws", device, t, n, k, X.data_ptr(), ldx, W.data_ptr(), ldw, kind,
          None if bias is None else bias.data_ptr(), act, rp, ldr, Y.data_ptr(), ldy, FP32 if dt == torch.float32 else kind,
          Z.data_ptr() if want_pre else None, max(n, 1), wp, wb)
    return Y, Z


def linear_grad(dY, X, W, Z=None, activation=None, want_dx=True, want_dw=True, want_dbias=True, workspace=None):
    """(dX, dW, dbias), the gradients of linear's layer from that of Y (ozaki2_linear_grad_ws); None for one that is not
    wanted. dY (t, n) has X's dtype, and so has Z, which linear returned with ``want_pre`` and which a layer without an
    activation does not need. dX and dW have X's dtype, dbias is float32; the residual's gradient is dY itself."""
    torch = _torch or _load_torch()
    device, kind, t, n, k, X, ldx, W, ldw = _layer_operands(X, W)
    act = _activation(activation)
    if act and Z is None:
        raise ValueError("a layer with an activation needs Z")
    for x, what in ((dY, "dY"), (Z if act else None, "Z")):
        if x is not None and (x.dtype != X.dtype or x.device != device or tuple(x.shape) != (t, n)):
            raise ValueError(f"{what} must be a ({t}, {n}) {X.dtype} tensor on {device}")
    dY, lddy = _rows(dY, "dY")
    zp = ldz = 0
    if act:
        Z, ldz = _rows(Z, "Z")
        zp = Z.data_ptr()
    dX = X.new_empty(t, k) if want_dx else None
    dW = X.new_empty(n, k) if want_dw else None
    dbias = X.new_empty(n, dtype=torch.float32) if want_dbias else None
    L = lib()
    size = L.ozaki2_linear_grad_workspace_size(t, n, k, 1 if want_dx else 0, 1 if want_dw else 0, 1 if want_dbias else 0)
    ws, wp, wb = _workspace(size, workspace, device)
    _call(L.ozaki2_linear_grad_ws, "ozaki2_linear_grad_ws", device, t, n, k, dY.data_ptr(), lddy, X.data_ptr(), ldx,
          W.data_ptr(), ldw, kind, act, zp, ldz, dX.data_ptr() if want_dx else None, max(k, 1),
          dW.data_ptr() if want_dw else None, max(k, 1), dbias.data_ptr() if want_dbias else None, wp, wb)
    return dX, dW, dbias


# ---- linear cross entropy ----------------------------------------------------
def _xent_operands(X, W, targets):
    torch = _torch or _load_torch()
    device = X.device
    if device.type != "cuda" or W.device != device or targets.device != device:
        raise TypeError("X, W and targets must be on the same GPU")
    if targets.dtype != torch.int64:
        raise TypeError("targets must be int64")
    X, ldx = _rows(X, "X")
    W, ldw = _rows(W, "W")
    t, d = X.shape
    v = W.shape[0]
    if W.shape[1] != d:
        raise ValueError("X and W must have the same number of columns")
    if targets.dim() != 1 or targets.shape[0] != t:
        raise ValueError(f"targets must have shape ({t},)")
    if t and not v:
        raise ValueError("W has no rows")
    return device, t, v, d, X, ldx, W, ldw, targets if targets.is_contiguous() else targets.contiguous()


def _xent_type(X, W):
    torch = _torch or _load_torch()
    if X.dtype not in (torch.bfloat16, torch.float16) or W.dtype != X.dtype:
        raise TypeError("X and W must both be bfloat16 or both float16")
    return BF16 if X.dtype == torch.bfloat16 else FP16


def xent(X, W, targets, ignore_index=-100, workspace=None):
    """Per token, the cross entropy of the logits X @ W.T against the target and their log-sum-exp, without storing
    the logits (ozaki2_xent_ws): (loss, lse), float32. X (t, d) and W (v, d) are bfloat16 or float16, targets (t,)
    int64. The loss is 0 where the target is ``ignore_index`` and NaN where it is out of range otherwise. Autograd does
    not see the call (the results require no gradient): xent_grad gives the gradients."""
    torch = _torch or _load_torch()
    kind = _xent_type(X, W)
    device, t, v, d, X, ldx, W, ldw, targets = _xent_operands(X, W, targets)
    loss = torch.empty(t, dtype=torch.float32, device=device)
    lse = torch.empty(t, dtype=torch.float32, device=device)
    L = lib()
    ws, wp, wb = _workspace(L.ozaki2_xent_workspace_size(t, v, d), workspace, device)
    _call(L.ozaki2_xent_ws, "ozaki2_xent_ws", device, t, v, d, X.data_ptr(), ldx, W.data_ptr(), ldw, kind,
          targets.data_ptr(), ignore_index, loss.data_ptr(), lse.data_ptr(), wp, wb)
    return loss, lse


def i8xent(A, B, a_scale, b_scale, targets, ignore_index=-100, workspace=None):
    """xent for quantised features A (t, k) and weights B (v, k), int8 with float32 scales per row: the logits are
    i8gemm's products in binary32, but with the sum times b_scale rounded first, so not always its bits
    (ozaki2_i8xent_ws). Returns (loss, lse)."""
    torch = _torch or _load_torch()
    if A.dtype != torch.int8 or B.dtype != torch.int8:
        raise TypeError("A and B must be int8")
    device, t, v, k, A, lda, B, ldb, targets = _xent_operands(A, B, targets)
    a_scale = _vector(a_scale, t, torch.float32, device, "a_scale")
    b_scale = _vector(b_scale, v, torch.float32, device, "b_scale")
    loss = torch.empty(t, dtype=torch.float32, device=device)
    lse = torch.empty(t, dtype=torch.float32, device=device)
    L = lib()
    ws, wp, wb = _workspace(L.ozaki2_i8xent_workspace_size(t, v, k), workspace, device)
    _call(L.ozaki2_i8xent_ws, "ozaki2_i8xent_ws", device, t, v, k, A.data_ptr(), lda, a_scale.data_ptr(), B.data_ptr(),
          ldb, b_scale.data_ptr(), targets.data_ptr(), ignore_index, loss.data_ptr(), lse.data_ptr(), wp, wb)
    return loss, lse


def xent_grad(X, W, targets, lse, grad_loss, ignore_index=-100, want_dx=True, want_dw=True, workspace=None):
    """(dX, dW), the gradients of sum(grad_loss * loss) for xent's loss, from the lse that xent returned
    (ozaki2_xent_grad_ws); None for one that is not wanted."""
    torch = _torch or _load_torch()
    kind = _xent_type(X, W)
    device, t, v, d, X, ldx, W, ldw, targets = _xent_operands(X, W, targets)
    lse = _vector(lse, t, torch.float32, device, "lse")
    grad_loss = _vector(grad_loss, t, torch.float32, device, "grad_loss")
    dX = torch.empty((t, d), dtype=X.dtype, device=device) if want_dx else None
    dW = torch.empty((v, d), dtype=X.dtype, device=device) if want_dw else None
    L = lib()
    ws, wp, wb = _workspace(L.ozaki2_xent_grad_workspace_size(t, v, d, 1 if want_dx else 0, 1 if want_dw else 0),
                            workspace, device)
    _call(L.ozaki2_xent_grad_ws, "ozaki2_xent_grad_ws", device, t, v, d, X.data_ptr(), ldx, W.data_ptr(), ldw, kind,
          targets.data_ptr(), ignore_index, lse.data_ptr(), grad_loss.data_ptr(),
          dX.data_ptr() if want_dx else None, max(d, 1), dW.data_ptr() if want_dw else None, max(d, 1), wp, wb)
    return dX, dW


# ---- the next token ------------------------------------------------------------
def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, workspace=None):
    """A token per row of logits (t, v; bfloat16, float16 or float32), and the logarithm of its probability among what the
    filters keep: (tokens int64, logprobs float32) (ozaki2_sample_ws). u (t,) holds float64 random numbers in [0, 1): the
    token is the first kept index whose running sum of probabilities exceeds u, so the same u gives the same token.
    ``temperature`` (0: the largest logit), ``top_k`` (0: off), ``top_p`` (1: off) and ``min_p`` (0: off) are numbers, or
    vectors (t,) with a value per row, float32 (top_k int32); include/ozaki2.h says what each keeps, in that order. A row
    without an entry to draw (all -inf, or NaN among them) gives -1 and NaN."""
    torch = _torch or _load_torch()
    kind = _type_of(logits.dtype, "logits")
    device = logits.device
    if device.type != "cuda":
        raise TypeError("logits must be on a GPU")
    logits, ldl = _rows(logits, "logits")
    t, v = logits.shape
    if t and not v:
        raise ValueError("logits have no columns")
    u = _vector(u, t, torch.float64, device, "u")

    def setting(x, dtype, what):
        """Its number and its vector, of which the call takes one."""
        if isinstance(x, torch.Tensor):
            x = _vector(x, t, dtype, device, what)
            return 0, x, x.data_ptr()
        return x, None, None

    temperature, temperatures, tp = setting(temperature, torch.float32, "temperature")
    top_k, top_ks, kp = setting(top_k, torch.int32, "top_k")
    top_p, top_ps, pp = setting(top_p, torch.float32, "top_p")
    min_p, min_ps, mp = setting(min_p, torch.float32, "min_p")
    tokens = logits.new_empty(t, dtype=torch.int64)
    logprobs = logits.new_empty(t, dtype=torch.float32)
    L = lib()
    ws, wp, wb = _workspace(L.ozaki2_sample_workspace_size(t, v), workspace, device)
    _call(L.ozaki2_sample_ws, "ozaki2_sample_ws", device, t, v, logits.data_ptr(), ldl, kind, u.data_ptr(), temperature, tp, top_k,
          kp, top_p, pp, min_p, mp, tokens.data_ptr(), logprobs.data_ptr(), wp, wb)
    return tokens, logprobs
