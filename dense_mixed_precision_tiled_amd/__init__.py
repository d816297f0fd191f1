"""Python binding of libgemm (tiled mixed-precision D = A x B + C on MI355X).

Argument marshalling only: every step of the multiply-accumulate runs in the
HIP kernels of ``lib/libgemm.so``.  The functions keep the C names and
argument order of ``include/libgemm.h``; pointers are passed as integers
(device addresses, e.g. ``tensor.data_ptr()``) and the stream as the integer
value of a ``hipStream_t`` (``torch.cuda.current_stream().cuda_stream``).

The library is loaded on first use.  When it is missing this raises: there
is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

# PyTorch-ROCm ships its own HIP runtime with the same soname as /opt/rocm's;
# importing torch first makes libgemm bind to that one runtime, so torch's
# streams and allocations are valid handles for libgemm.
import torch  # noqa: F401

__all__ = [
    "GEMM_ROW_MAJOR", "GEMM_COL_MAJOR", "GEMM_F32", "GEMM_F16", "GEMM_BF16", "GEMM_I8",
    "GEMM_I32", "GEMM_FP8_E4M3", "GEMM_FP8_E5M2",
    "GEMM_OK", "GemmError", "LIB_PATH", "library",
    "gemm_run", "gemm_run_noalloc", "gemm_run_config", "gemm_validate", "gemm_status_string",
    "gemm_num_configs", "gemm_config_name", "gemm_select_config",
    "GEMM_ACT_NONE", "GEMM_ACT_RELU", "GEMM_ACT_GELU", "GemmEpilogue",
    "gemm_run_ex", "gemm_run_ex_config", "gemm_validate_ex",
    "gemm_quantize_rows", "gemm_validate_quantize_rows",
    "gemm_run_scaled", "gemm_validate_scaled",
    "GEMM_ACT_SILU", "GemmMoe", "gemm_moe_run", "gemm_moe_workspace", "gemm_validate_moe",
    "gemm_moe_balance", "gemm_moe_balance_grad", "gemm_moe_balance_workspace",
    "gemm_validate_moe_balance", "gemm_validate_moe_balance_grad",
    "GemmLora", "gemm_lora_run", "gemm_lora_workspace", "gemm_validate_lora",
    "gemm_checkpoint_pack", "gemm_checkpoint_unpack", "gemm_checkpoint_act_grad",
    "gemm_checkpoint_wgrad", "gemm_checkpoint_wgrad_workspace", "gemm_validate_checkpoint_pack",
    "gemm_validate_checkpoint_unpack", "gemm_validate_checkpoint_act_grad",
    "gemm_validate_checkpoint_wgrad",
    "gemm_autotune", "gemm_autotune_lookup", "gemm_autotune_clear",
]

GEMM_ROW_MAJOR, GEMM_COL_MAJOR = 0, 1
GEMM_F32, GEMM_F16, GEMM_BF16, GEMM_I8, GEMM_I32 = 0, 1, 2, 3, 4
GEMM_FP8_E4M3, GEMM_FP8_E5M2 = 5, 6
GEMM_OK = 0
GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_SILU = 0, 1, 2, 3
STATUS_NAMES = {
    0: "GEMM_OK", -1: "GEMM_ERR_INVALID_DIM", -2: "GEMM_ERR_INVALID_LD",
    -3: "GEMM_ERR_NULL_PTR", -4: "GEMM_ERR_UNSUPPORTED", -5: "GEMM_ERR_INVALID_LAYOUT",
    -6: "GEMM_ERR_ALIASING", -7: "GEMM_ERR_HIP", -8: "GEMM_ERR_INVALID_CONFIG",
    -9: "GEMM_ERR_SCRATCH_TOO_SMALL",
}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libgemm.so")


class GemmEpilogue(ctypes.Structure):
    """gemm_epilogue_t: D = act(alpha * A x B + beta * C + bias), C/D layouts.

    ``bias`` is a device address (int) of N fp32 values, or 0 for none."""
    _fields_ = [("alpha", ctypes.c_float), ("beta", ctypes.c_float),
                ("bias", ctypes.c_void_p), ("activation", ctypes.c_int),
                ("layoutC", ctypes.c_int), ("layoutD", ctypes.c_int)]

    def __init__(self, alpha=1.0, beta=1.0, bias=0, activation=GEMM_ACT_NONE,
                 layoutC=GEMM_ROW_MAJOR, layoutD=GEMM_ROW_MAJOR):
        super().__init__(alpha, beta, bias or None, activation, layoutC, layoutD)


class GemmMoe(ctypes.Structure):
    """gemm_moe_t: a mixture-of-experts layer.

    ``W1``, ``W2`` and the scales of int8 weights are device addresses (int)."""
    _fields_ = [("H", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int64),
                ("topk", ctypes.c_int64), ("W1", ctypes.c_void_p), ("ld1", ctypes.c_int64),
                ("W2", ctypes.c_void_p), ("ld2", ctypes.c_int64), ("scale1", ctypes.c_void_p),
                ("scale2", ctypes.c_void_p), ("w_dtype", ctypes.c_int),
                ("activation", ctypes.c_int), ("renormalize", ctypes.c_int)]

    def __init__(self, H, I, E, topk, w_dtype, W1, ld1, W2, ld2, scale1=0, scale2=0,
                 activation=GEMM_ACT_SILU, renormalize=False):
        super().__init__(H, I, E, topk, W1 or None, ld1, W2 or None, ld2, scale1 or None,
                         scale2 or None, w_dtype, activation, int(renormalize))


class GemmLora(ctypes.Structure):
    """gemm_lora_t: the low-rank adapters of one projection.

    ``A``, ``B``, ``ranks`` and ``scales`` are device addresses (int); the last two may
    be 0 for none."""
    _fields_ = [("K", ctypes.c_int64), ("N", ctypes.c_int64), ("adapters", ctypes.c_int64),
                ("rank", ctypes.c_int64), ("A", ctypes.c_void_p), ("lda", ctypes.c_int64),
                ("B", ctypes.c_void_p), ("ldb", ctypes.c_int64), ("ranks", ctypes.c_void_p),
                ("scales", ctypes.c_void_p)]

    def __init__(self, K, N, adapters, rank, A, lda, B, ldb, ranks=0, scales=0):
        super().__init__(K, N, adapters, rank, A or None, lda, B or None, ldb, ranks or None,
                         scales or None)


# Exported symbols and their C signatures (mirrors include/libgemm.h).
_i64, _int, _vp, _cp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_char_p
_f32 = ctypes.c_float
_GEMM_ARGS = [_i64, _i64, _i64, _vp, _i64, _int, _vp, _i64, _int, _vp, _i64, _vp, _i64,
              _int, _int, _int, _int, _vp]
SIGNATURES = {
    "gemm_run": (_int, _GEMM_ARGS),
    "gemm_run_noalloc": (_int, _GEMM_ARGS),
    "gemm_run_config": (_int, [_int] + _GEMM_ARGS),
    "gemm_validate": (_int, [_i64, _i64, _i64, _vp, _i64, _int, _vp, _i64, _int, _vp, _i64,
                             _vp, _i64, _int, _int, _int]),
    "gemm_status_string": (_cp, [_int]),
    "gemm_num_configs": (_int, []),
    "gemm_config_name": (_cp, [_int]),
    "gemm_select_config": (_int, [_i64, _i64, _i64, _int, _int, _int, _int, _int]),
    "gemm_run_ex": (_int, _GEMM_ARGS[:-1] + [ctypes.POINTER(GemmEpilogue), _vp]),
    "gemm_run_ex_config": (_int, [_int] + _GEMM_ARGS[:-1] + [ctypes.POINTER(GemmEpilogue), _vp]),
    "gemm_validate_ex": (_int, [_i64, _i64, _i64, _vp, _i64, _int, _vp, _i64, _int, _vp, _i64,
                                _vp, _i64, _int, _int, _int, ctypes.POINTER(GemmEpilogue)]),
    "gemm_quantize_rows": (_int, [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _vp]),
    "gemm_validate_quantize_rows": (_int, [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp]),
    "gemm_run_scaled": (_int, _GEMM_ARGS[:9] + [_vp, _vp] + _GEMM_ARGS[9:-1] +
                        [ctypes.POINTER(GemmEpilogue), _vp]),
    "gemm_validate_scaled": (_int, _GEMM_ARGS[:9] + [_vp, _vp] + _GEMM_ARGS[9:-2] +
                             [ctypes.POINTER(GemmEpilogue)]),
    "gemm_moe_run": (_int, [_i64, ctypes.POINTER(GemmMoe), _vp, _i64, _vp, _i64, _vp, _i64, _int,
                            _vp, _i64, _vp]),
    "gemm_moe_workspace": (_i64, [_i64, ctypes.POINTER(GemmMoe)]),
    "gemm_validate_moe": (_int, [_i64, ctypes.POINTER(GemmMoe), _vp, _i64, _vp, _i64, _vp, _i64,
                                 _int, _vp, _i64]),
    "gemm_moe_balance": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _f32, _f32, _vp, _vp, _vp, _vp,
                                _i64, _vp]),
    "gemm_moe_balance_grad": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _f32, _f32, _vp, _vp, _vp,
                                     _vp, _i64, _int, _vp]),
    "gemm_moe_balance_workspace": (_i64, [_i64, _i64, _i64]),
    "gemm_validate_moe_balance": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _f32, _f32, _vp, _vp,
                                         _vp, _vp, _i64]),
    "gemm_validate_moe_balance_grad": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _f32, _f32, _vp,
                                              _vp, _vp, _vp, _i64, _int]),
    "gemm_lora_run": (_int, [_i64, ctypes.POINTER(GemmLora), _vp, _i64, _vp, _vp, _i64, _vp, _i64,
                             _int, _int, _vp, _i64, _vp]),
    "gemm_lora_workspace": (_i64, [_i64, ctypes.POINTER(GemmLora)]),
    "gemm_validate_lora": (_int, [_i64, ctypes.POINTER(GemmLora), _vp, _i64, _vp, _vp, _i64, _vp,
                                  _i64, _int, _int, _vp, _i64]),
    "gemm_checkpoint_pack": (_int, [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64, _vp]),
    "gemm_checkpoint_unpack": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp]),
    "gemm_checkpoint_act_grad": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int, _vp,
                                        _i64, _int, _vp]),
    "gemm_checkpoint_wgrad": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                     _vp, _i64, _int, _int, _vp, _i64, _vp]),
    "gemm_checkpoint_wgrad_workspace": (_i64, [_i64, _i64, _i64]),
    "gemm_validate_checkpoint_pack": (_int, [_i64, _i64, _vp, _i64, _int, _vp, _i64, _vp, _i64]),
    "gemm_validate_checkpoint_unpack": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int]),
    "gemm_validate_checkpoint_act_grad": (_int, [_i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _int,
                                                 _vp, _i64, _int]),
    "gemm_validate_checkpoint_wgrad": (_int, [_i64, _i64, _i64, _vp, _i64, _vp, _i64, _vp, _i64,
                                              _vp, _i64, _vp, _i64, _int, _int, _vp, _i64]),
    "gemm_autotune": (_int, _GEMM_ARGS[:-1] + [ctypes.POINTER(GemmEpilogue), _int,
                                              ctypes.POINTER(_int), _vp]),
    "gemm_autotune_lookup": (_int, [_i64, _i64, _i64, _int, _int, _int, _int, _int, _int]),
    "gemm_autotune_clear": (None, []),
}


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str = "gemm_run"):
        self.status = status
        super().__init__("%s failed: %s (%s)" % (where, STATUS_NAMES.get(status, status),
                                                gemm_status_string(status)))


_lib = None


def library() -> ctypes.CDLL:
    """Load lib/libgemm.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libgemm.so is not built (%s); run "
                "`python -m dense_mixed_precision_tiled_amd.build`" % LIB_PATH)
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def gemm_run(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
             in_dtype, acc_dtype, out_dtype, satf, stream) -> int:
    """Enqueue D = A x B + C; returns the gemm_status_t code."""
    return library().gemm_run(M, N, K, A, lda, layoutA, B, ldb, layoutB, C or None, ldc,
                              D, ldd, in_dtype, acc_dtype, out_dtype, int(satf), stream or None)


def gemm_run_noalloc(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                     in_dtype, acc_dtype, out_dtype, satf, stream) -> int:
    """gemm_run with no device allocation (split-K partial sums in the
    library's fixed 32 MiB scratch); returns the status code."""
    return library().gemm_run_noalloc(M, N, K, A, lda, layoutA, B, ldb, layoutB, C or None, ldc,
                                      D, ldd, in_dtype, acc_dtype, out_dtype, int(satf),
                                      stream or None)


def gemm_run_config(config_id, M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                    in_dtype, acc_dtype, out_dtype, satf, stream) -> int:
    """gemm_run with the tile-table entry forced; returns the status code."""
    return library().gemm_run_config(config_id, M, N, K, A, lda, layoutA, B, ldb, layoutB,
                                     C or None, ldc, D, ldd, in_dtype, acc_dtype, out_dtype,
                                     int(satf), stream or None)


def gemm_validate(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                  in_dtype, acc_dtype, out_dtype) -> int:
    """Host-only argument check (no device needed); returns the status code."""
    return library().gemm_validate(M, N, K, A or None, lda, layoutA, B or None, ldb, layoutB,
                                   C or None, ldc, D or None, ldd, in_dtype, acc_dtype,
                                   out_dtype)


def gemm_status_string(status: int) -> str:
    return library().gemm_status_string(status).decode()


def gemm_num_configs() -> int:
    return library().gemm_num_configs()


def gemm_config_name(config_id: int):
    s = library().gemm_config_name(config_id)
    return None if s is None else s.decode()


def gemm_select_config(M, N, K, layoutA, layoutB, in_dtype, acc_dtype, out_dtype) -> int:
    return library().gemm_select_config(M, N, K, layoutA, layoutB, in_dtype, acc_dtype,
                                        out_dtype)


def _epi_ref(epi):
    return None if epi is None else ctypes.byref(epi)


def gemm_run_ex(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                in_dtype, acc_dtype, out_dtype, satf, epi, stream) -> int:
    """Enqueue D = act(alpha * A x B + beta * C + bias) (``epi``: a GemmEpilogue
    or None for the plain gemm_run); returns the status code."""
    return library().gemm_run_ex(M, N, K, A, lda, layoutA, B, ldb, layoutB, C or None, ldc,
                                 D, ldd, in_dtype, acc_dtype, out_dtype, int(satf),
                                 _epi_ref(epi), stream or None)


def gemm_run_ex_config(config_id, M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                       in_dtype, acc_dtype, out_dtype, satf, epi, stream) -> int:
    """gemm_run_ex with the tile-table entry forced; returns the status code."""
    return library().gemm_run_ex_config(config_id, M, N, K, A, lda, layoutA, B, ldb, layoutB,
                                        C or None, ldc, D, ldd, in_dtype, acc_dtype, out_dtype,
                                        int(satf), _epi_ref(epi), stream or None)


def gemm_validate_ex(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                     in_dtype, acc_dtype, out_dtype, epi) -> int:
    """Host-only argument check of gemm_run_ex; returns the status code."""
    return library().gemm_validate_ex(M, N, K, A or None, lda, layoutA, B or None, ldb,
                                      layoutB, C or None, ldc, D or None, ldd, in_dtype,
                                      acc_dtype, out_dtype, _epi_ref(epi))


def gemm_quantize_rows(M, K, X, ldx, in_dtype, Q, ldq, scales, stream) -> int:
    """Enqueue the quantisation of X's rows to int8 ``Q`` with one fp32 scale
    for each row; returns the status code."""
    return library().gemm_quantize_rows(M, K, X or None, ldx, in_dtype, Q or None, ldq,
                                        scales or None, stream or None)


def gemm_validate_quantize_rows(M, K, X, ldx, in_dtype, Q, ldq, scales) -> int:
    """Host-only argument check of gemm_quantize_rows; returns the status code."""
    return library().gemm_validate_quantize_rows(M, K, X or None, ldx, in_dtype, Q or None, ldq,
                                                 scales or None)


def gemm_run_scaled(M, N, K, A, lda, layoutA, B, ldb, layoutB, scaleA, scaleB, C, ldc, D, ldd,
                    in_dtype, acc_dtype, out_dtype, satf, epi, stream) -> int:
    """Enqueue D = act(alpha * (A x B) * scaleA[i] * scaleB[j] + beta * C + bias)
    of int8 A and B (``epi``: a GemmEpilogue or None); returns the status code."""
    return library().gemm_run_scaled(M, N, K, A or None, lda, layoutA, B or None, ldb, layoutB,
                                     scaleA or None, scaleB or None, C or None, ldc, D or None,
                                     ldd, in_dtype, acc_dtype, out_dtype, int(satf),
                                     _epi_ref(epi), stream or None)


def gemm_validate_scaled(M, N, K, A, lda, layoutA, B, ldb, layoutB, scaleA, scaleB, C, ldc, D,
                         ldd, in_dtype, acc_dtype, out_dtype, epi) -> int:
    """Host-only argument check of gemm_run_scaled; returns the status code."""
    return library().gemm_validate_scaled(M, N, K, A or None, lda, layoutA, B or None, ldb,
                                          layoutB, scaleA or None, scaleB or None, C or None,
                                          ldc, D or None, ldd, in_dtype, acc_dtype, out_dtype,
                                          _epi_ref(epi))


def gemm_moe_run(T, layer, X, ldx, logits, ldl, D, ldd, in_dtype, workspace, workspace_bytes,
                 stream) -> int:
    """Enqueue the mixture-of-experts layer ``layer`` (a GemmMoe) on T tokens;
    returns the status code."""
    return library().gemm_moe_run(T, _epi_ref(layer), X or None, ldx, logits or None, ldl,
                                  D or None, ldd, in_dtype, workspace or None, workspace_bytes,
                                  stream or None)


def gemm_moe_workspace(T, layer) -> int:
    """Bytes of device workspace that gemm_moe_run needs, or a negative status code."""
    return library().gemm_moe_workspace(T, _epi_ref(layer))


def gemm_validate_moe(T, layer, X, ldx, logits, ldl, D, ldd, in_dtype, workspace,
                      workspace_bytes) -> int:
    """Host-only argument check of gemm_moe_run; returns the status code."""
    return library().gemm_validate_moe(T, _epi_ref(layer), X or None, ldx, logits or None, ldl,
                                       D or None, ldd, in_dtype, workspace or None,
                                       workspace_bytes)


def gemm_moe_balance(T, E, topk, logits, ldl, mask, balance, z, loss, counts, lse, workspace,
                     workspace_bytes, stream) -> int:
    """Enqueue the router's balance loss, its per-expert counts and the rows' log-sum-exps;
    returns the status code."""
    return library().gemm_moe_balance(T, E, topk, logits or None, ldl, mask or None, balance, z,
                                      loss or None, counts or None, lse or None,
                                      workspace or None, workspace_bytes, stream or None)


def gemm_moe_balance_grad(T, E, topk, logits, ldl, mask, balance, z, counts, lse, dloss, D, ldd,
                          out_dtype, stream) -> int:
    """Enqueue the gradient of gemm_moe_balance's loss with respect to the logits; returns
    the status code."""
    return library().gemm_moe_balance_grad(T, E, topk, logits or None, ldl, mask or None, balance,
                                           z, counts or None, lse or None, dloss or None,
                                           D or None, ldd, out_dtype, stream or None)


def gemm_moe_balance_workspace(T, E, topk) -> int:
    """Bytes of device workspace that gemm_moe_balance needs, or a negative status code."""
    return library().gemm_moe_balance_workspace(T, E, topk)


def gemm_validate_moe_balance(T, E, topk, logits, ldl, mask, balance, z, loss, counts, lse,
                              workspace, workspace_bytes) -> int:
    """Host-only argument check of gemm_moe_balance; returns the status code."""
    return library().gemm_validate_moe_balance(T, E, topk, logits or None, ldl, mask or None,
                                               balance, z, loss or None, counts or None,
                                               lse or None, workspace or None, workspace_bytes)


def gemm_validate_moe_balance_grad(T, E, topk, logits, ldl, mask, balance, z, counts, lse, dloss,
                                   D, ldd, out_dtype) -> int:
    """Host-only argument check of gemm_moe_balance_grad; returns the status code."""
    return library().gemm_validate_moe_balance_grad(T, E, topk, logits or None, ldl, mask or None,
                                                    balance, z, counts or None, lse or None,
                                                    dloss or None, D or None, ldd, out_dtype)


def gemm_lora_run(T, lora, X, ldx, ids, C, ldc, D, ldd, in_dtype, out_dtype, workspace,
                  workspace_bytes, stream) -> int:
    """Enqueue D = C + the low-rank adapters ``lora`` (a GemmLora), one for each of T
    tokens by ``ids``; returns the status code."""
    return library().gemm_lora_run(T, _epi_ref(lora), X or None, ldx, ids or None, C or None, ldc,
                                   D or None, ldd, in_dtype, out_dtype, workspace or None,
                                   workspace_bytes, stream or None)


def gemm_lora_workspace(T, lora) -> int:
    """Bytes of device workspace that gemm_lora_run needs, or a negative status code."""
    return library().gemm_lora_workspace(T, _epi_ref(lora))


def gemm_validate_lora(T, lora, X, ldx, ids, C, ldc, D, ldd, in_dtype, out_dtype, workspace,
                       workspace_bytes) -> int:
    """Host-only argument check of gemm_lora_run; returns the status code."""
    return library().gemm_validate_lora(T, _epi_ref(lora), X or None, ldx, ids or None, C or None,
                                        ldc, D or None, ldd, in_dtype, out_dtype,
                                        workspace or None, workspace_bytes)


def gemm_checkpoint_pack(M, K, X, ldx, in_dtype, Q, ldq, S, lds, stream) -> int:
    """Enqueue the packing of X to int8 ``Q`` with a power of two ``S`` for each 32 values
    of a row; returns the status code."""
    return library().gemm_checkpoint_pack(M, K, X or None, ldx, in_dtype, Q or None, ldq,
                                          S or None, lds, stream or None)


def gemm_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, out_dtype, stream) -> int:
    """Enqueue D = the values that Q and S stand for; returns the status code."""
    return library().gemm_checkpoint_unpack(M, K, Q or None, ldq, S or None, lds, D or None, ldd,
                                            out_dtype, stream or None)


def gemm_checkpoint_act_grad(M, K, Q, ldq, S, lds, G, ldg, activation, D, ldd, dtype,
                             stream) -> int:
    """Enqueue D = G * act'(the values that Q and S stand for); returns the status code."""
    return library().gemm_checkpoint_act_grad(M, K, Q or None, ldq, S or None, lds, G or None, ldg,
                                              activation, D or None, ldd, dtype, stream or None)


def gemm_checkpoint_wgrad(M, N, K, G, ldg, Q, ldq, S, lds, C, ldc, D, ldd, in_dtype, out_dtype,
                          workspace, workspace_bytes, stream) -> int:
    """Enqueue D = G^T x (the values that Q and S stand for) + C; returns the status code."""
    return library().gemm_checkpoint_wgrad(M, N, K, G or None, ldg, Q or None, ldq, S or None, lds,
                                           C or None, ldc, D or None, ldd, in_dtype, out_dtype,
                                           workspace or None, workspace_bytes, stream or None)


def gemm_checkpoint_wgrad_workspace(M, N, K) -> int:
    """Bytes of device workspace that gemm_checkpoint_wgrad needs (possibly 0), or a
    negative status code."""
    return library().gemm_checkpoint_wgrad_workspace(M, N, K)


def gemm_validate_checkpoint_pack(M, K, X, ldx, in_dtype, Q, ldq, S, lds) -> int:
    """Host-only argument check of gemm_checkpoint_pack; returns the status code."""
    return library().gemm_validate_checkpoint_pack(M, K, X or None, ldx, in_dtype, Q or None, ldq,
                                                   S or None, lds)


def gemm_validate_checkpoint_unpack(M, K, Q, ldq, S, lds, D, ldd, out_dtype) -> int:
    """Host-only argument check of gemm_checkpoint_unpack; returns the status code."""
    return library().gemm_validate_checkpoint_unpack(M, K, Q or None, ldq, S or None, lds,
                                                     D or None, ldd, out_dtype)


def gemm_validate_checkpoint_act_grad(M, K, Q, ldq, S, lds, G, ldg, activation, D, ldd,
                                      dtype) -> int:
    """Host-only argument check of gemm_checkpoint_act_grad; returns the status code."""
    return library().gemm_validate_checkpoint_act_grad(M, K, Q or None, ldq, S or None, lds,
                                                       G or None, ldg, activation, D or None, ldd,
                                                       dtype)


def gemm_validate_checkpoint_wgrad(M, N, K, G, ldg, Q, ldq, S, lds, C, ldc, D, ldd, in_dtype,
                                   out_dtype, workspace, workspace_bytes) -> int:
    """Host-only argument check of gemm_checkpoint_wgrad; returns the status code."""
    return library().gemm_validate_checkpoint_wgrad(M, N, K, G or None, ldg, Q or None, ldq,
                                                    S or None, lds, C or None, ldc, D or None, ldd,
                                                    in_dtype, out_dtype, workspace or None,
                                                    workspace_bytes)


def gemm_autotune(M, N, K, A, lda, layoutA, B, ldb, layoutB, C, ldc, D, ldd,
                  in_dtype, acc_dtype, out_dtype, satf, epi, reps, stream):
    """Time every table entry on this call, record the fastest for the
    signature; returns (status, chosen entry).  Synchronises the stream."""
    out = ctypes.c_int(-1)
    st = library().gemm_autotune(M, N, K, A, lda, layoutA, B, ldb, layoutB, C or None, ldc,
                                 D, ldd, in_dtype, acc_dtype, out_dtype, int(satf),
                                 _epi_ref(epi), int(reps), ctypes.byref(out), stream or None)
    return st, out.value


def gemm_autotune_lookup(M, N, K, layoutA, layoutB, in_dtype, acc_dtype, out_dtype,
                         layoutD=GEMM_ROW_MAJOR) -> int:
    """The recorded entry for this signature, or -1."""
    return library().gemm_autotune_lookup(M, N, K, layoutA, layoutB, in_dtype, acc_dtype,
                                          out_dtype, layoutD)


def gemm_autotune_clear() -> None:
    library().gemm_autotune_clear()
