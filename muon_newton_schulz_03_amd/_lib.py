"""ctypes view of the C ABI declared in include/muon.h (argument marshalling only)."""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon_mi355x.so")

MUON_OK = 0
MUON_E_INVAL = -1
MUON_E_UNSUPPORTED = -2
MUON_E_MISMATCH = -3
MUON_E_WORKSPACE = -4
MUON_SCRATCH_BYTES = 64 << 20
MUON_E_HIP = -5

MUON_DTYPE_F32 = 0
MUON_DTYPE_BF16 = 1
MUON_PATH_BF16 = 0
MUON_PATH_F32 = 1

KIND_MOMENTUM, KIND_GRAM, KIND_POLY, KIND_UPDATE, KIND_APPLY, KIND_NORM, KIND_FUSED = range(7)
KIND_COUNT = 7
KIND_NAMES = ("momentum", "gram", "poly", "update", "apply", "norm", "fused")

EXPORTS = ("muon_version", "muon_workspace_size", "muon_init", "muon_step", "muon_step_schedule", "muon_destroy",
           "muon_last_error", "muon_describe", "muon_profile_enable", "muon_profile_select", "muon_profile_read",
           "muon_step_scratch", "muon_check", "muon_fused_limits",
           "muon_layernorm_forward", "muon_layernorm_workspace_size", "muon_layernorm_backward",
           "muon_attention_forward", "muon_attention_workspace_size", "muon_attention_backward",
           "muon_qk_norm_forward", "muon_qk_norm_workspace_size", "muon_qk_norm_backward",
           "muon_embedding_forward", "muon_embedding_workspace_size", "muon_embedding_backward")

ATTENTION_ZERO_OUT, ATTENTION_ZERO_LSE = 1, 2
ATTENTION_ZERO_DQ, ATTENTION_ZERO_DK, ATTENTION_ZERO_DV = 1, 2, 4
MUON_INDEX_I32, MUON_INDEX_I64 = 0, 1
PAIRS_HALVES, PAIRS_NEIGHBOURS = 0, 1
QK_ZERO_Q, QK_ZERO_K = 1, 2
EMBEDDING_ACCUMULATE = 1


class MatrixDesc(ctypes.Structure):
    _fields_ = [("weight", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("momentum", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_w", ctypes.c_int64),
                ("ld_g", ctypes.c_int64), ("w_dtype", ctypes.c_int32), ("g_dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class Options(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("x_master_iters", ctypes.c_int32),
                ("zero_momentum", ctypes.c_int32), ("max_T", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("fused", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("workspace_bytes", ctypes.c_int64), ("n_matrices", ctypes.c_int32), ("tile", ctypes.c_int32),
                ("blocks", ctypes.c_int32 * KIND_COUNT), ("x_master_iters", ctypes.c_int32),
                ("path", ctypes.c_int32), ("n_f32_matrices", ctypes.c_int32), ("n_groups", ctypes.c_int32),
                ("bf16_tile_rows", ctypes.c_int32), ("bf16_tile_cols", ctypes.c_int32), ("fused", ctypes.c_int32)]


class LayerNormDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld_x", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("ld_dx", ctypes.c_int64), ("x_dtype", ctypes.c_int32),
                ("p_dtype", ctypes.c_int32), ("eps", ctypes.c_float), ("reserved", ctypes.c_int32)]


class AttentionDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("seqs", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("reserved", ctypes.c_int32)]


class Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class QkNormDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("seqs", ctypes.c_int32), ("q_heads", ctypes.c_int32),
                ("k_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("p_dtype", ctypes.c_int32), ("position_dtype", ctypes.c_int32), ("eps", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class RotationDesc(ctypes.Structure):
    _fields_ = [("frequencies", ctypes.POINTER(ctypes.c_double)), ("dim", ctypes.c_int32), ("pairs", ctypes.c_int32)]


class EmbeddingDesc(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("vocab", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("ld_table", ctypes.c_int64), ("ld_out", ctypes.c_int64), ("table_dtype", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("id_dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class MuonError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"muon error {code}: {msg}")
        self.code = code


_lib = None


def load() -> ctypes.CDLL:
    """Load the in-tree build of the library (fails loudly if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = LIB_PATH
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m muon_newton_schulz_03_amd.build`")
    lib = ctypes.CDLL(path)
    P = ctypes.POINTER
    lib.muon_version.restype = ctypes.c_char_p
    lib.muon_version.argtypes = []
    lib.muon_last_error.restype = ctypes.c_char_p
    lib.muon_last_error.argtypes = []
    lib.muon_workspace_size.restype = ctypes.c_size_t
    lib.muon_workspace_size.argtypes = [P(MatrixDesc), ctypes.c_int, P(Options)]
    lib.muon_init.restype = ctypes.c_int
    lib.muon_init.argtypes = [P(MatrixDesc), ctypes.c_int, P(Options), ctypes.c_void_p, ctypes.c_size_t,
                              ctypes.c_void_p, P(ctypes.c_void_p)]
    lib.muon_step.restype = ctypes.c_int
    lib.muon_step.argtypes = [ctypes.c_void_p, P(MatrixDesc), ctypes.c_int, ctypes.c_float, ctypes.c_float,
                              ctypes.c_float, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_float,
                              ctypes.c_void_p]
    lib.muon_step_schedule.restype = ctypes.c_int
    lib.muon_step_schedule.argtypes = [ctypes.c_void_p, P(MatrixDesc), ctypes.c_int, P(ctypes.c_float), ctypes.c_int,
                                       ctypes.c_float, ctypes.c_int, ctypes.c_float, ctypes.c_void_p]
    lib.muon_step_scratch.restype = ctypes.c_int
    lib.muon_step_scratch.argtypes = [P(MatrixDesc), ctypes.c_int, P(Options), ctypes.c_float, ctypes.c_float,
                                      ctypes.c_float, ctypes.c_int, ctypes.c_float, ctypes.c_int, ctypes.c_float,
                                      ctypes.c_void_p]
    lib.muon_destroy.restype = ctypes.c_int
    lib.muon_destroy.argtypes = [ctypes.c_void_p]
    lib.muon_describe.restype = ctypes.c_int
    lib.muon_describe.argtypes = [P(MatrixDesc), ctypes.c_int, P(Options), P(PlanInfo), ctypes.c_int,
                                  P(ctypes.c_int32), ctypes.c_int, P(ctypes.c_int32)]
    lib.muon_profile_enable.restype = ctypes.c_int
    lib.muon_profile_enable.argtypes = [ctypes.c_void_p, ctypes.c_int]
    lib.muon_profile_select.restype = ctypes.c_int
    lib.muon_profile_select.argtypes = [ctypes.c_void_p, ctypes.c_uint32]
    lib.muon_profile_read.restype = ctypes.c_int
    lib.muon_profile_read.argtypes = [ctypes.c_void_p, P(ctypes.c_double), P(ctypes.c_int64)]
    lib.muon_check.restype = ctypes.c_int
    lib.muon_check.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    lib.muon_fused_limits.restype = ctypes.c_int
    lib.muon_fused_limits.argtypes = [ctypes.c_void_p, ctypes.c_int32, ctypes.c_int32]
    vp, hp = ctypes.c_void_p, P(Heads)
    lib.muon_layernorm_forward.restype = ctypes.c_int
    lib.muon_layernorm_forward.argtypes = [P(LayerNormDesc)] + [vp] * 7
    lib.muon_layernorm_workspace_size.restype = ctypes.c_size_t
    lib.muon_layernorm_workspace_size.argtypes = [P(LayerNormDesc)]
    lib.muon_layernorm_backward.restype = ctypes.c_int
    lib.muon_layernorm_backward.argtypes = [P(LayerNormDesc)] + [vp] * 9 + [ctypes.c_size_t, vp]
    lib.muon_attention_forward.restype = ctypes.c_int
    lib.muon_attention_forward.argtypes = [P(AttentionDesc), vp, hp, hp, hp, hp, vp, ctypes.c_uint32, vp]
    lib.muon_attention_workspace_size.restype = ctypes.c_size_t
    lib.muon_attention_workspace_size.argtypes = [P(AttentionDesc)]
    lib.muon_attention_backward.restype = ctypes.c_int
    lib.muon_attention_backward.argtypes = ([P(AttentionDesc), vp] + [hp] * 5 + [vp] + [hp] * 3 +
                                            [ctypes.c_uint32, vp, ctypes.c_size_t, vp])
    rp = P(RotationDesc)
    lib.muon_qk_norm_forward.restype = ctypes.c_int
    lib.muon_qk_norm_forward.argtypes = [P(QkNormDesc), rp, vp, vp, hp, hp, vp, vp, hp, hp, ctypes.c_uint32, vp]
    lib.muon_qk_norm_workspace_size.restype = ctypes.c_size_t
    lib.muon_qk_norm_workspace_size.argtypes = [P(QkNormDesc)]
    lib.muon_qk_norm_backward.restype = ctypes.c_int
    lib.muon_qk_norm_backward.argtypes = ([P(QkNormDesc), rp, vp, vp, hp, hp, hp, hp, vp, vp, hp, hp, vp, vp,
                                           ctypes.c_uint32, vp, ctypes.c_size_t, vp])
    lib.muon_embedding_forward.restype = ctypes.c_int
    lib.muon_embedding_forward.argtypes = [P(EmbeddingDesc)] + [vp] * 4
    lib.muon_embedding_workspace_size.restype = ctypes.c_size_t
    lib.muon_embedding_workspace_size.argtypes = [P(EmbeddingDesc)]
    lib.muon_embedding_backward.restype = ctypes.c_int
    lib.muon_embedding_backward.argtypes = [P(EmbeddingDesc), vp, vp, vp, ctypes.c_uint32, vp, ctypes.c_size_t, vp]
    _lib = lib
    return lib


def check(code: int) -> None:
    if code != MUON_OK:
        raise MuonError(code, load().muon_last_error().decode())


def last_error() -> str:
    return load().muon_last_error().decode()
