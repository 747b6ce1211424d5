"""ctypes declarations of libmuon.so (include/muon.h).  Loaded on first use.

There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmuon.so")

MUON_OK = 0
MUON_ERR_INVALID_ARGUMENT = 1
MUON_ERR_INVALID_SHAPE = 2
MUON_ERR_UNSUPPORTED_DTYPE = 3
MUON_ERR_WORKSPACE_TOO_SMALL = 4
MUON_ERR_HIP = 5

MUON_DTYPE_F32 = 0
MUON_DTYPE_BF16 = 1
MUON_VARIANT_MUON = 0
MUON_VARIANT_MUONGS = 1
MUON_VARIANT_MUONH = 2
MUON_VARIANT_NORMUON = 3
MUON_VARIANT_MEQMUON = 4
MUON_SCALE_KELLER = 0x100
MUON_STATS_PER_MATRIX = 5
MUON_MAX_DIM = 32768
MUON_MAX_NS_STEPS = 100
MUON_GROUPS_PER_LAUNCH = 8
MUON_ADAMW_MAX_ELEMENTS = 1 << 40
MUON_ADAMW_TENSORS_PER_LAUNCH = 32
MUON_ADAMW8_MAX_ELEMENTS = 1 << 35
MUON_ADAMW8_TENSORS_PER_LAUNCH = 56
MUON_NOALLOC_WORKSPACE_BYTES = 64 << 20
MUON_MAX_TOKENS = 1 << 30
MUON_CKPT_BLOCK = 32
MUON_CKPT_E4M3 = 0
MUON_CKPT_INT8 = 1
MUON_LINEAR_MAX_COUNT = 1024
MUON_LINEAR_FEW, MUON_LINEAR_TILES_64, MUON_LINEAR_TILES_128 = 0, 1, 2
MUON_LINEAR_STREAM_128, MUON_LINEAR_STREAM_256 = 3, 4
MUON_WEIGHT_BLOCK = 128

# Every symbol include/muon.h declares.
EXPORTS = (
    "muon_workspace_bytes", "muon_workspace_bytes_grouped", "muon_step",
    "muon_step_batched", "muon_step_grouped", "muon_status_string", "muon_last_hip_error",
    "muon_profile_enable", "muon_profile_read", "muon_phase_name",
    "muon_adamw_step", "muon_adamw_step_grouped", "muon_step_grouped_noalloc",
    "muon_checkpoint_save", "muon_checkpoint_restore", "muon_layernorm_forward",
    "muon_layernorm_workspace_bytes", "muon_layernorm_backward",
    "muon_weight_grad_workspace_bytes", "muon_weight_grad_tile", "muon_weight_grad",
    "muon_adamw_byte_step_grouped", "muon_adamw_byte_moments",
    "muon_linear_forward", "muon_linear_input_grad", "muon_weight_quantize",
    "muon_linear_forward_quantized", "muon_linear_input_grad_quantized", "muon_linear_kernel",
)
MUON_NUM_PHASES = 10


class MuonGroup(ctypes.Structure):
    _fields_ = [
        ("count", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("W_table", ctypes.c_void_p),
        ("G_table", ctypes.c_void_p),
        ("M_table", ctypes.c_void_p),
        ("W", ctypes.c_void_p),
        ("G", ctypes.c_void_p),
        ("M", ctypes.c_void_p),
    ]


class AdamwTensor(ctypes.Structure):
    _fields_ = [
        ("P", ctypes.c_void_p),
        ("G", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("n", ctypes.c_int64),
        ("lr", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
    ]


class Adamw8State(ctypes.Structure):
    _fields_ = [
        ("m_q", ctypes.c_void_p),
        ("m_scale", ctypes.c_void_p),
        ("r_q", ctypes.c_void_p),
        ("r_scale", ctypes.c_void_p),
        ("n", ctypes.c_int64),
    ]


class Adamw8Tensor(ctypes.Structure):
    _fields_ = [
        ("P", ctypes.c_void_p),
        ("G", ctypes.c_void_p),
        ("state", Adamw8State),
        ("lr", ctypes.c_double),
        ("weight_decay", ctypes.c_double),
        ("seed", ctypes.c_uint32),
    ]


class Ckpt(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("tokens", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("format", ctypes.c_int),
    ]


class Weight8(ctypes.Structure):
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("q_t", ctypes.c_void_p),
        ("scale", ctypes.c_void_p),
        ("count", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
    ]


def weight_pitch(n: int) -> int:
    """Bytes per row of an 8-bit weight's q (MUON_WEIGHT_PITCH)."""
    return (n + 127) // 128 * 128


def ckpt_q_pitch(cols: int) -> int:
    """Bytes per row of a checkpoint's q (MUON_CKPT_Q_PITCH)."""
    return (cols + 31) // 32 * 32


def ckpt_scale_pitch(cols: int) -> int:
    """Bytes per row of a checkpoint's scales (MUON_CKPT_SCALE_PITCH)."""
    return (cols + 127) // 128 * 4


_lib = None

_STEP_SCALARS = [ctypes.c_int, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_int,
                 ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_int,
                 ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p]


def lib():
    """The loaded library; raises RuntimeError if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m muon_step_03_amd.build` "
            "(or __graft_entry__.build()); the Muon step has no non-HIP implementation")
    L = ctypes.CDLL(LIB_PATH)
    L.muon_workspace_bytes.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    L.muon_workspace_bytes.restype = ctypes.c_size_t
    L.muon_workspace_bytes_grouped.argtypes = [ctypes.POINTER(MuonGroup), ctypes.c_int, ctypes.c_int]
    L.muon_workspace_bytes_grouped.restype = ctypes.c_size_t
    L.muon_step.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                            ctypes.c_int64, ctypes.c_int64] + _STEP_SCALARS
    L.muon_step.restype = ctypes.c_int
    L.muon_step_batched.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_int64, ctypes.c_int64, ctypes.c_int64] + _STEP_SCALARS
    L.muon_step_batched.restype = ctypes.c_int
    L.muon_step_grouped.argtypes = [ctypes.POINTER(MuonGroup), ctypes.c_int] + _STEP_SCALARS
    L.muon_step_grouped.restype = ctypes.c_int
    L.muon_step_grouped_noalloc.argtypes = ([ctypes.POINTER(MuonGroup), ctypes.c_int]
                                            + _STEP_SCALARS[:9] + [ctypes.c_void_p, ctypes.c_void_p])
    L.muon_step_grouped_noalloc.restype = ctypes.c_int
    L.muon_status_string.argtypes = [ctypes.c_int]
    L.muon_status_string.restype = ctypes.c_char_p
    L.muon_last_hip_error.argtypes = []
    L.muon_last_hip_error.restype = ctypes.c_int
    L.muon_profile_enable.argtypes = [ctypes.c_int]
    L.muon_profile_enable.restype = ctypes.c_int
    L.muon_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64),
                                    ctypes.c_int]
    L.muon_profile_read.restype = ctypes.c_int
    L.muon_adamw_step.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                  ctypes.c_double, ctypes.c_int64, ctypes.c_void_p]
    L.muon_adamw_step.restype = ctypes.c_int
    L.muon_adamw_step_grouped.argtypes = [ctypes.POINTER(AdamwTensor), ctypes.c_int64, ctypes.c_int,
                                          ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                          ctypes.c_int64, ctypes.c_void_p]
    L.muon_adamw_step_grouped.restype = ctypes.c_int
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.muon_adamw_byte_step_grouped.argtypes = [ctypes.POINTER(Adamw8Tensor), i64, i32, ctypes.c_double,
                                           ctypes.c_double, ctypes.c_double, i64, p]
    L.muon_adamw_byte_step_grouped.restype = i32
    L.muon_adamw_byte_moments.argtypes = [ctypes.POINTER(Adamw8State), i64, p, p, i32, p]
    L.muon_adamw_byte_moments.restype = i32
    ck = ctypes.POINTER(Ckpt)
    w8 = ctypes.POINTER(Weight8)
    for fn in (L.muon_linear_forward, L.muon_linear_input_grad):
        fn.argtypes = [p, i64, i32, p, p, i64, i64, i64, i64, p, p]
        fn.restype = i32
    for fn in (L.muon_linear_forward_quantized, L.muon_linear_input_grad_quantized):
        fn.argtypes = [ck, w8, p, p, i32, p]
        fn.restype = i32
    L.muon_linear_kernel.argtypes = [i32, i32, i64, i64, i64, i64, i32]
    L.muon_linear_kernel.restype = i32
    L.muon_weight_quantize.argtypes = [p, i32, w8, p]
    L.muon_weight_quantize.restype = i32
    L.muon_checkpoint_save.argtypes = [p, i64, i32, ck, p]
    L.muon_checkpoint_save.restype = i32
    L.muon_checkpoint_restore.argtypes = [ck, p, i32, p]
    L.muon_checkpoint_restore.restype = i32
    L.muon_layernorm_forward.argtypes = [p, i64, p, p, i64, i64, i32, i32, ctypes.c_double,
                                         p, p, p, ck, ck, p]
    L.muon_layernorm_forward.restype = i32
    L.muon_layernorm_workspace_bytes.argtypes = [i64, i64]
    L.muon_layernorm_workspace_bytes.restype = ctypes.c_size_t
    L.muon_layernorm_backward.argtypes = [p, i64, p, i64, ck, p, p, p, i64, i64, i32, i32,
                                          p, p, p, i32, p, ctypes.c_size_t, p]
    L.muon_layernorm_backward.restype = i32
    L.muon_weight_grad_workspace_bytes.argtypes = [i64, i32, i64, i64, i64, i32]
    L.muon_weight_grad_workspace_bytes.restype = ctypes.c_size_t
    L.muon_weight_grad_tile.argtypes = [i64, i32, i64, i64, i64, i32]
    L.muon_weight_grad_tile.restype = i32
    L.muon_weight_grad.argtypes = [p, i64, i32, ck, p, i64, i64, p, i32, i32, p,
                                   ctypes.c_size_t, p]
    L.muon_weight_grad.restype = i32
    L.muon_phase_name.argtypes = [ctypes.c_int]
    L.muon_phase_name.restype = ctypes.c_char_p
    _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().muon_status_string(int(status)).decode()
