"""ctypes loader for libpuro.so. The library must have been built (see build.py); there is no
fallback of any kind: a missing or unloadable library raises."""
from __future__ import annotations

import ctypes
import os
import threading

from .build import LIB_PATH

_lock = threading.Lock()
_lib = None

# Every symbol declared in include/puro.h, with its ctypes signature.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
W_GROUP_MAX = 8  # PURO_W_GROUP_MAX


class PuroWItem(ctypes.Structure):
    """puro_w_item: one weight matrix of a grouped 128x128 quantisation."""
    _fields_ = [("w", ctypes.c_void_p), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("q", ctypes.c_void_p), ("s", ctypes.c_void_p)]

class PuroAdamWParams(ctypes.Structure):
    """puro_adamw_params: AdamW hyperparameters of one step."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float),
                ("step", ctypes.c_int64)]


class PuroBlockNorm(ctypes.Structure):
    """puro_block_norm: one forward block norm."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("rows", "cols")]
                + [(k, ctypes.c_int) for k in ("residual_type", "gate_kind", "pow2")]
                + [(k, ctypes.c_float) for k in ("alpha", "beta", "eps")]
                + [(k, ctypes.c_void_p) for k in
                   ("y", "r", "w_post", "w_pre", "gate", "r_out", "n", "nq", "ns", "rstd_y",
                    "rstd_r", "yq", "ys", "rq", "rs")])


class PuroBlockNormGrad(ctypes.Structure):
    """puro_block_norm_grad: one backward block norm."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("rows", "cols")]
                + [(k, ctypes.c_int) for k in ("residual_type", "gate_kind", "accumulate")]
                + [(k, ctypes.c_float) for k in ("alpha", "beta")]
                + [(k, ctypes.c_void_p) for k in
                   ("dr_out", "dn", "y", "yq", "ys", "r", "rq", "rs", "rstd_y", "rstd_r",
                    "w_post", "w_pre", "gate", "dr", "dy", "dw_post", "dw_pre", "dgate")])


class PuroNsItem(ctypes.Structure):
    """puro_ns_item: one matrix of a grouped orthogonalisation."""
    _fields_ = [(k, ctypes.c_void_p) for k in ("g", "m", "m_out", "u")]


class PuroNewtonSchulzParams(ctypes.Structure):
    """puro_newton_schulz_params."""
    _fields_ = [("steps", ctypes.c_int), ("nesterov", ctypes.c_int), ("beta", ctypes.c_float),
                ("scale", ctypes.c_float), ("coefficients", ctypes.c_float * 3)]


class PuroLinearXent(ctypes.Structure):
    """puro_linear_xent: one forward cross entropy."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("tokens", "d", "vocab", "ldh", "ldw")]
                + [(k, ctypes.c_void_p) for k in ("h", "w", "targets", "loss", "lse")])


class PuroLinearXentGrad(ctypes.Structure):
    """puro_linear_xent_grad: one backward cross entropy."""
    _fields_ = ([(k, ctypes.c_int64) for k in ("tokens", "d", "vocab", "ldh", "ldw")]
                + [(k, ctypes.c_int) for k in ("dw_type", "accumulate")]
                + [(k, ctypes.c_void_p) for k in
                   ("h", "w", "targets", "lse", "dloss", "dlse", "dh", "dw")])


TYPE_BF16, TYPE_FP32 = 0, 1                                     # PURO_TYPE_*
GATE_NONE, GATE_CHANNEL, GATE_TOKEN, GATE_FULL = 0, 1, 2, 3     # PURO_GATE_*
NORM_MAX_COLS = 16384                                           # PURO_NORM_MAX_COLS
NS_GROUP_MAX = 64                                               # PURO_NS_GROUP_MAX

OPT_MAX_BLOCKS = 2048  # PURO_OPT_MAX_BLOCKS
OPT_WORKSPACE_BYTES = 8 * OPT_MAX_BLOCKS + 256  # PURO_OPT_WORKSPACE_BYTES

SIGNATURES = {
    "puro_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "puro_abi_version": ([], ctypes.c_int),
    "puro_set_debug": ([ctypes.c_int], None),
    "puro_debug_level": ([], ctypes.c_int),
    "puro_quant_act_1x128": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "puro_quant_w_128x128": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "puro_quant_transpose": ([_P, _I64, _I64, _P, _P, _P], ctypes.c_int),
    "puro_quant_dual_1x128": ([_P, _I64, _I64, _P, _P, _P, _P, _P], ctypes.c_int),
    "puro_quant_w_128x128_group": ([ctypes.POINTER(PuroWItem), ctypes.c_int, _P], ctypes.c_int),
    "puro_fp8_gemm_fwd": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "puro_fp8_gemm_dgrad": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "puro_fp8_gemm_wgrad": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P],
                            ctypes.c_int),
    "puro_gemm_kernel_name": ([ctypes.c_int, _I64, _I64, _I64, ctypes.c_int], ctypes.c_char_p),
}
SIGNATURES.update({
    "puro_frobenius_norm": ([_P, _I64, _P, _P, _P], ctypes.c_int),
    "puro_hyperball_step": ([_P, _P, _I64, ctypes.c_float, _P, _P, _P, _P], ctypes.c_int),
    "puro_hyperball_step_noalloc": ([_P, _P, _I64, ctypes.c_float, _P, _P, _P], ctypes.c_int),
    "puro_hyperball_step_u16": ([_P, _P, _I64, ctypes.c_float, _P, _P, _P, _P], ctypes.c_int),
    "puro_newton_schulz_workspace": ([_I64, _I64, _I64], _I64),
    "puro_newton_schulz": ([ctypes.POINTER(PuroNsItem), ctypes.c_int, _I64, _I64,
                            ctypes.POINTER(PuroNewtonSchulzParams), _P, _P], ctypes.c_int),
    "puro_linear_xent_fwd_workspace": ([ctypes.POINTER(PuroLinearXent)], _I64),
    "puro_linear_xent_fwd": ([ctypes.POINTER(PuroLinearXent), _P, _P], ctypes.c_int),
    "puro_linear_xent_bwd_workspace": ([ctypes.POINTER(PuroLinearXentGrad)], _I64),
    "puro_linear_xent_bwd": ([ctypes.POINTER(PuroLinearXentGrad), _P, _P], ctypes.c_int),
    "puro_adamw_step": ([_P, _P, _P, _P, _I64, ctypes.POINTER(PuroAdamWParams), _P, _P],
                        ctypes.c_int),
})
_INT = ctypes.c_int
SIGNATURES.update({
    "puro_ckpt_pack": ([_P, _INT, _I64, _I64, _I64, _INT, _P, _P, _P], _INT),
    "puro_ckpt_unpack": ([_P, _P, _I64, _I64, _P, _INT, _I64, _P], _INT),
    "puro_ckpt_transpose": ([_P, _P, _I64, _I64, _INT, _P, _P, _P], _INT),
    # (the structures as bytes, or by reference)
    "puro_block_norm_fwd": ([_P, _P], _INT),
    "puro_block_norm_workspace": ([_I64, _I64], _I64),
    "puro_block_norm_bwd": ([_P, _P, _P], _INT),
    "puro_swiglu_fwd": ([_P, _I64, _I64, _P, _P, _P, _P, _P, _INT, _P], _INT),
    "puro_swiglu_bwd": ([_P, _P, _P, _P, _I64, _I64, _P, _P], _INT),
    "puro_swiglu_bwd_fp8": ([_P, _P, _P, _P, _I64, _I64, _INT] + [_P] * 7, _INT),
})
# The power-of-two-scale variants take the same arguments as their standard counterparts.
POW2_BASES = ("puro_quant_act_1x128", "puro_quant_w_128x128", "puro_quant_w_128x128_group",
              "puro_quant_transpose", "puro_quant_dual_1x128", "puro_fp8_gemm_fwd",
              "puro_fp8_gemm_dgrad", "puro_fp8_gemm_wgrad")
SIGNATURES.update({b + "_pow2": SIGNATURES[b] for b in POW2_BASES})


class PuroError(RuntimeError):
    """A libpuro call returned a nonzero status (or the library is unavailable)."""


def lib() -> ctypes.CDLL:
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise PuroError(
                    "libpuro.so is not built (%s); run `python -m "
                    "blockwise_fp8_gemm_x128_amd.build`" % LIB_PATH)
            try:  # make torch's HIP runtime the one libpuro binds to (one runtime per process)
                import torch  # noqa: F401
            except ImportError:  # pragma: no cover
                pass
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def check(status: int) -> None:
    if status != 0:
        raise PuroError(lib().puro_status_string(status).decode())
