"""ctypes binding to libpwq.so -- argument marshalling only.

Every step of the quantization runs in the library's HIP kernels; torch only
supplies device memory (outputs and workspaces) and the current HIP stream.
There is no fallback: without the built library every call raises.
"""
import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpwq.so")

PWQ_OK, PWQ_ERR_INVALID_ARG, PWQ_ERR_UNSUPPORTED, PWQ_ERR_WORKSPACE, PWQ_ERR_HIP = range(5)
PWQ_F32, PWQ_BF16, PWQ_F64 = 0, 1, 2
PWQ_I8 = 3                    # 8-bit integers (include/pwq_serve.h)
PWQ_X_TOKEN_MAJOR = 0x100     # X stored ntok x n (one row per token)
GRID_KINDS = {"sym": 0, "asym": 1, "colspacing": 2}
ORDERS = {"back_to_front": 0, "front_to_back": 1, "perm": 2, "act_order": 3, "min_pivot": 4}

# every symbol include/pwq.h declares
EXPORTS = [
    "pwq_status_string", "pwq_last_error",
    "pwq_hessian_workspace_size", "pwq_hessian_accum",
    "pwq_cholesky_workspace_size", "pwq_damp_cholesky", "pwq_damp_cholesky_static",
    "pwq_grid_steps",
    "pwq_sweep_workspace_size", "pwq_babai_sweep",
    "pwq_quant_layer_workspace_size", "pwq_quant_layer",
    "pwq_rate_workspace_size", "pwq_column_entropy",
    "pwq_kernel_timer_attach", "pwq_kernel_timer_count",
    "pwq_overflow_workspace_size", "pwq_overflow_entries",
    "pwq_ssqr_workspace_size", "pwq_ssqr_quant_layer",
    "pwq_min_pivot_workspace_size", "pwq_min_pivot_order",
    "pwq_oaem_workspace_size", "pwq_oaem_init",
]
# and include/pwq_serve.h (packed layers)
SERVE_EXPORTS = [
    "pwq_packed_row_bytes", "pwq_pack_tiles", "pwq_pack_codes", "pwq_pack_overflow",
    "pwq_rms_norm", "pwq_packed_linear_workspace_size", "pwq_packed_linear",
]
PWQ_TIMER_HESSIAN_TILES, PWQ_TIMER_LAZY_UPDATE, PWQ_TIMER_SWEEP_BLOCK = 0, 1, 2
TIMED_KERNELS = {"hessian_tiles": PWQ_TIMER_HESSIAN_TILES, "lazy_update": PWQ_TIMER_LAZY_UPDATE,
                 "sweep_block": PWQ_TIMER_SWEEP_BLOCK}


class PwqGrid(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("bits", ctypes.c_int32),
                ("group_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("c", ctypes.c_double), ("kappa", ctypes.c_double)]


RESULT_BYTES = 64          # sizeof(pwq_result) = 56, padded
_RESULT_FMT = "<dddddii8x"  # loss, loss_damped, bound, delta_sq, lambda, info, ndead


class PwqError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{status}: {msg}")
        self.status = status


_lib = None

_vp, _i32, _i64, _f64, _sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64,
                              ctypes.c_double, ctypes.c_size_t)
_SIGS = {
    "pwq_status_string": (ctypes.c_char_p, [_i32]),
    "pwq_last_error": (ctypes.c_char_p, []),
    "pwq_hessian_workspace_size": (_sz, [_i64, _i64]),
    "pwq_hessian_accum": (_i32, [_vp, _i64, _vp, _i32, _i64, _i64, _i32, _vp, _sz, _vp]),
    "pwq_cholesky_workspace_size": (_sz, [_i64, _i32]),
    "pwq_damp_cholesky": (_i32, [_vp, _i64, _f64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_damp_cholesky_static": (_i32, [_vp, _i64, _f64, _i32, _vp, _vp, _vp, _vp]),
    "pwq_grid_steps": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, ctypes.POINTER(PwqGrid),
                              _vp, _vp, _vp]),
    "pwq_sweep_workspace_size": (_sz, [_i64, _i64, _i32, _i32]),
    "pwq_babai_sweep": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _vp,
                               ctypes.POINTER(PwqGrid), _vp, _vp, _i32, _vp, _vp, _vp, _sz,
                               _vp]),
    "pwq_quant_layer_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32, _i32, _i32]),
    "pwq_quant_layer": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64, _i64, _vp,
                               ctypes.POINTER(PwqGrid), _i32, _vp, _f64, _i32, _i32, _vp,
                               _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_rate_workspace_size": (_sz, [_i64]),
    "pwq_column_entropy": (_i32, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_overflow_workspace_size": (_sz, [_i64]),
    "pwq_overflow_entries": (_i32, [_vp, _i64, _i64, _i64, ctypes.POINTER(PwqGrid), _vp, _vp,
                                    _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_oaem_workspace_size": (_sz, [_i64, _i64, _i32, _i32]),
    "pwq_oaem_init": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, ctypes.c_double, _i32, _i32,
                             _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_min_pivot_workspace_size": (_sz, [_i64]),
    "pwq_min_pivot_order": (_i32, [_vp, _i64, ctypes.c_double, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pwq_ssqr_workspace_size": (_sz, [_i64, _i64, _i64, _i32, _i32, _i32]),
    "pwq_ssqr_quant_layer": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i32, _i64, _i64, _vp,
                                    ctypes.POINTER(PwqGrid), _f64, _i32, _i32, _f64, _i32, _f64,
                                    _vp, _vp, _vp, _vp, _i64, _vp, _vp, _vp,
                                    ctypes.POINTER(ctypes.c_int64),
                                    ctypes.POINTER(ctypes.c_double), _vp, _sz, _vp]),
    "pwq_packed_row_bytes": (_i64, [_i64]),
    "pwq_pack_tiles": (_i64, [_i64, _i64]),
    "pwq_pack_codes": (_i32, [_vp, _i64, _i64, _i64, ctypes.POINTER(PwqGrid), _vp, _vp, _vp, _vp,
                              _vp, _vp]),
    "pwq_pack_overflow": (_i32, [_vp, _i64, _i64, _i64, ctypes.POINTER(PwqGrid), _vp, _vp, _i64,
                                 _vp]),
    "pwq_rms_norm": (_i32, [_vp, _i32, _i64, _i64, _i64, _vp, _i64, _vp, _i32, _f64, _vp, _i64,
                            _vp, _i32, _i64, _vp, _vp]),
    "pwq_packed_linear_workspace_size": (_sz, [_vp, _i32, _i64, _i64, _i64, _i64, _i32, _i64]),
    "pwq_packed_linear": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _i32,
                                 _vp, _vp, _i64, _vp, _i32, _i64, _vp, _sz, _vp]),
    "pwq_kernel_timer_attach": (_i32, [_i32, _vp, _vp, _i64]),
    "pwq_kernel_timer_count": (_i64, [_i32]),
}


def lib():
    """Load libpwq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libpwq.so is not built; run `python -m post_weight_quantization_19_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def check(status):
    if status != PWQ_OK:
        L = lib()
        raise PwqError(L.pwq_status_string(status).decode(), L.pwq_last_error().decode())


def make_grid(kind="sym", bits=4, group=0, c=0.0, kappa=0.0):
    return PwqGrid(GRID_KINDS[kind], int(bits), int(group), 0, float(c), float(kappa))


def parse_result(raw: bytes):
    loss, loss_d, bound, dsq, lam, info, ndead = struct.unpack(_RESULT_FMT, raw[:56])
    return {"loss": loss, "loss_damped": loss_d, "bound": bound, "delta_sq": dsq,
            "lambda": lam, "info": info, "ndead": ndead}
