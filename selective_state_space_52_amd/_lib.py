"""ctypes view of libmssm.so (include/mssm.h).  Argument marshalling only."""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmssm.so")

MSSM_F32 = 0
MSSM_BF16 = 1
MSSM_FLAG_LOAD_STATE = 1
MSSM_FLAG_LAYOUT_BLD = 2
MSSM_FLAG_BC_STATE_MAJOR = 4
MSSM_FLAG_STATE_STREAM = 8

STATUS = {
    0: "MSSM_OK", -1: "MSSM_ERR_NULL", -2: "MSSM_ERR_DIMS",
    -3: "MSSM_ERR_UNSUPPORTED", -4: "MSSM_ERR_ALIGN", -5: "MSSM_ERR_ALIAS",
    -6: "MSSM_ERR_HIP", -7: "MSSM_ERR_WORKSPACE",
}

MSSM_OP_SCAN_FWD = 0
MSSM_OP_SCAN_FWD_CONV = 1
MSSM_OP_SCAN_BWD = 2
MSSM_OP_MAMBA2_FWD = 3

# every symbol include/mssm.h declares
EXPORTS = ("mssm_selective_scan_fwd", "mssm_selective_scan_bwd",
           "mssm_selective_scan_fwd_conv", "mssm_causal_conv1d_fwd",
           "mssm_selective_state_update", "mssm_mamba2_scan_fwd",
           "mssm_selective_scan_fwd_plan", "mssm_set_scan_timing_events",
           "mssm_status_string", "mssm_last_error", "mssm_abi_version",
           "mssm_selective_scan_fwd_ws", "mssm_selective_scan_fwd_conv_ws",
           "mssm_selective_scan_bwd_ws", "mssm_mamba2_scan_fwd_ws",
           "mssm_workspace_size", "mssm_selective_scan_fwd_noalloc",
           "mssm_valu_probe", "mssm_causal_conv1d_bwd",
           "mssm_rms_norm_fwd", "mssm_rms_norm_fwd_fp8", "mssm_rms_norm_bwd",
           "mssm_rms_norm_bwd_workspace", "mssm_quantize_fp8", "mssm_fp8_matmul",
           "mssm_sample", "mssm_mamba2_state_update",
           "mssm_mamba2_state_update_workspace",
           "mssm_embedding_fwd", "mssm_embedding_bwd", "mssm_embedding_bwd_workspace",
           "mssm_token_logprobs_fwd", "mssm_token_logprobs_workspace",
           "mssm_token_logprobs_bwd", "mssm_policy_loss",
           "mssm_preference_loss", "mssm_adamw")


class Dims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("dstate", ctypes.c_int64), ("seqlen", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("time_segments", ctypes.c_int32), ("ngroups", ctypes.c_int32)]


class Plan(ctypes.Structure):
    _fields_ = [("groups", ctypes.c_int32), ("whole_groups", ctypes.c_int32),
                ("split_groups", ctypes.c_int32), ("segments", ctypes.c_int32),
                ("segment_len", ctypes.c_int64),
                ("waves_per_group", ctypes.c_int32), ("kernels", ctypes.c_int32),
                ("workspace_bytes", ctypes.c_int64),
                ("vector_path", ctypes.c_int32), ("reserved", ctypes.c_int32)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("res_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class QuantDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("x_stride", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("block_rows", ctypes.c_int32), ("transpose", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class MatmulDims(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("out_dtype", ctypes.c_int32), ("b_block_rows", ctypes.c_int32)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("logits_stride", ctypes.c_int64), ("noise_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("temperature", ctypes.c_float), ("top_p", ctypes.c_float),
                ("min_p", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("temperature_row", ctypes.c_void_p), ("top_k_row", ctypes.c_void_p),
                ("top_p_row", ctypes.c_void_p), ("min_p_row", ctypes.c_void_p)]


class StepDims(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("cache", ctypes.c_int64),
                ("nheads", ctypes.c_int64), ("headdim", ctypes.c_int64),
                ("ngroups", ctypes.c_int64), ("dstate", ctypes.c_int64),
                ("xbc_stride", ctypes.c_int64), ("dt_stride", ctypes.c_int64),
                ("z_stride", ctypes.c_int64), ("width", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32)]


class EmbedDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64), ("dim", ctypes.c_int64),
                ("io_stride", ctypes.c_int64), ("table_dtype", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("scale", ctypes.c_float), ("add", ctypes.c_int32)]


class LogprobDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("logits_stride", ctypes.c_int64), ("grad_stride", ctypes.c_int64),
                ("io_dtype", ctypes.c_int32), ("temperature", ctypes.c_float)]


class PolicyArgs(ctypes.Structure):
    _fields_ = [("dims", LogprobDims), ("clip_low", ctypes.c_float),
                ("clip_high", ctypes.c_float), ("kl_coef", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class PreferenceArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("pairs", ctypes.c_int64), ("beta", ctypes.c_float),
                ("label_smoothing", ctypes.c_float)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("size", ctypes.c_int64), ("weight_decay", ctypes.c_float),
                ("grad_dtype", ctypes.c_int32)]


class AdamwArgs(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("grad_scale", ctypes.c_double),
                ("step", ctypes.c_int64), ("seed", ctypes.c_uint64),
                ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("lr_value", ctypes.c_void_p), ("grad_scale_value", ctypes.c_void_p),
                ("step_value", ctypes.c_void_p)]


_lib = None


def lib():
    """The loaded library; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libmssm.so is not built (%s); run "
                "`python -m selective_state_space_52_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, fp, i = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int
        L.mssm_selective_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                              vp, fp, ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_fwd.restype = i
        L.mssm_selective_scan_bwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                              fp, vp, fp, vp, vp, fp, fp, fp,
                                              fp, vp, fp, fp,
                                              ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_bwd.restype = i
        L.mssm_selective_scan_fwd_conv.argtypes = [vp, fp, fp, vp, vp, fp, vp, vp,
                                                   fp, vp, fp, i, vp, fp, vp,
                                                   ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_fwd_conv.restype = i
        L.mssm_causal_conv1d_fwd.argtypes = [vp, fp, fp, vp, i, i, vp,
                                             ctypes.POINTER(Dims), vp]
        L.mssm_causal_conv1d_fwd.restype = i
        L.mssm_selective_state_update.argtypes = [fp, vp, vp, fp, vp, vp, fp, vp,
                                                  fp, i, vp, ctypes.POINTER(Dims), vp]
        L.mssm_selective_state_update.restype = i
        L.mssm_mamba2_scan_fwd.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                           ctypes.c_int64, vp, fp,
                                           ctypes.POINTER(Dims), vp]
        L.mssm_mamba2_scan_fwd.restype = i
        i64 = ctypes.c_int64
        L.mssm_selective_scan_fwd_ws.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                                 vp, fp, vp, i64, ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_fwd_ws.restype = i
        L.mssm_selective_scan_fwd_conv_ws.argtypes = [vp, fp, fp, vp, vp, fp, vp, vp,
                                                      fp, vp, fp, i, vp, fp, vp, vp, i64,
                                                      ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_fwd_conv_ws.restype = i
        L.mssm_selective_scan_bwd_ws.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                                 fp, vp, fp, vp, vp, fp, fp, fp,
                                                 fp, vp, fp, fp, vp, i64,
                                                 ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_bwd_ws.restype = i
        L.mssm_mamba2_scan_fwd_ws.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                              i64, vp, fp, vp, i64,
                                              ctypes.POINTER(Dims), vp]
        L.mssm_mamba2_scan_fwd_ws.restype = i
        L.mssm_selective_scan_fwd_noalloc.argtypes = [vp, vp, fp, vp, vp, fp, vp, fp, i,
                                                      vp, fp, ctypes.POINTER(Dims), vp]
        L.mssm_selective_scan_fwd_noalloc.restype = i
        L.mssm_workspace_size.argtypes = [i, ctypes.POINTER(Dims), i64,
                                          ctypes.POINTER(i64)]
        L.mssm_workspace_size.restype = i
        L.mssm_selective_scan_fwd_plan.argtypes = [ctypes.POINTER(Dims),
                                                   ctypes.POINTER(Plan)]
        L.mssm_selective_scan_fwd_plan.restype = i
        L.mssm_status_string.argtypes = [i]
        L.mssm_status_string.restype = ctypes.c_char_p
        L.mssm_last_error.argtypes = []
        L.mssm_last_error.restype = ctypes.c_char_p
        L.mssm_set_scan_timing_events.argtypes = [vp, vp]
        L.mssm_set_scan_timing_events.restype = i
        L.mssm_abi_version.argtypes = []
        L.mssm_abi_version.restype = i
        L.mssm_causal_conv1d_bwd.argtypes = [vp, fp, fp, vp, i, i, vp, vp, fp, fp, vp,
                                             ctypes.POINTER(Dims), vp]
        L.mssm_causal_conv1d_bwd.restype = i
        L.mssm_valu_probe.argtypes = [i, i, i, vp, vp]
        L.mssm_valu_probe.restype = i
        def sig(name, args):
            f = getattr(L, name)
            f.argtypes, f.restype = args, i
        nd, out64 = ctypes.POINTER(NormDims), ctypes.POINTER(i64)
        sd = ctypes.POINTER(StepDims)
        sig("mssm_rms_norm_fwd", [vp] * 6 + [nd, vp])
        sig("mssm_rms_norm_fwd_fp8", [vp] * 7 + [nd, vp])
        sig("mssm_rms_norm_bwd", [vp] * 9 + [i64, nd, i, vp])
        sig("mssm_rms_norm_bwd_workspace", [nd, out64])
        sig("mssm_quantize_fp8", [vp] * 3 + [ctypes.POINTER(QuantDims), vp])
        sig("mssm_fp8_matmul", [vp] * 5 + [ctypes.POINTER(MatmulDims), vp])
        sig("mssm_sample", [vp] * 4 + [ctypes.POINTER(SampleArgs), vp])
        sig("mssm_mamba2_state_update", [vp] * 10 + [i] + [vp] * 3 + [i64, sd, vp])
        sig("mssm_mamba2_state_update_workspace", [sd, out64])
        ed, ld = ctypes.POINTER(EmbedDims), ctypes.POINTER(LogprobDims)
        sig("mssm_embedding_fwd", [vp] * 3 + [ed, vp])
        sig("mssm_embedding_bwd", [vp] * 4 + [i64, ed, vp])
        sig("mssm_embedding_bwd_workspace", [ed, out64])
        sig("mssm_token_logprobs_fwd", [vp] * 5 + [i64, ld, vp])
        sig("mssm_token_logprobs_workspace", [ld, out64])
        sig("mssm_token_logprobs_bwd", [vp] * 5 + [ld, vp])
        sig("mssm_policy_loss", [vp] * 10 + [i64, ctypes.POINTER(PolicyArgs), vp])
        sig("mssm_preference_loss", [vp] * 6 + [ctypes.POINTER(PreferenceArgs), vp])
        sig("mssm_adamw", [vp, i64] + [vp] * 4 + [ctypes.POINTER(AdamwArgs), vp])
        _lib = L
    return _lib


class MssmError(RuntimeError):
    def __init__(self, code: int):
        L = lib()
        msg = L.mssm_status_string(code).decode()
        if code in (-6, -7):
            msg += ": " + L.mssm_last_error().decode()
        super().__init__("%s (%d): %s" % (STATUS.get(code, "?"), code, msg))
        self.code = code


def check(code: int) -> None:
    if code != 0:
        raise MssmError(code)
