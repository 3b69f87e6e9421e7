"""Loads libqstate.so and declares the C ABI of include/qstate.h for ctypes.

There is no fallback: if the library is missing or does not load, this
raises, and nothing in the package computes the step any other way."""

from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (loads the HIP runtime the library links against first)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqstate.so")

QSTATE_OK = 0
QSTATE_E_INVALID = -1
QSTATE_E_UNSUPPORTED = -2
QSTATE_E_LAUNCH = -3
QSTATE_E_NOMEM = -4

GDN, GLA, SCALAR, KDA = 0, 1, 2, 3
RTN, SR, BDR = 0, 1, 2
VALUE_AXIS, KEY_AXIS = 0, 1

EXPORTS = (
    "qstate_state_bytes", "qstate_create", "qstate_load_fp32", "qstate_step",
    "qstate_readout", "qstate_store_fp32", "qstate_get_step", "qstate_set_step",
    "qstate_destroy", "qstate_strerror", "qstate_bits_by_decay",
)
# include/qstate_ceiling.h: bandwidth-ceiling kernels (measurement support)
CEILING_EXPORTS = ("qstate_ceiling_copy", "qstate_ceiling_rmw")
# include/qstate_scan.h: the recurrences over whole sequences and their gradients
SCAN_EXPORTS = ("qstate_scan_workspace", "qstate_scan", "qstate_scan_backward")

# include/qstate_norm.h: the norms around the mixer block and their gradients
NORM_EXPORTS = ("qstate_norm", "qstate_norm_workspace", "qstate_norm_backward")

# include/qstate_draft.h: drafted tokens over the stored state
DRAFT_EXPORTS = ("qstate_verify", "qstate_accept")

# include/qstate_group_norm.h: the group norm of the readout and its gradients
GROUP_NORM_EXPORTS = ("qstate_group_norm", "qstate_group_norm_workspace",
                      "qstate_group_norm_backward")

# include/qstate_linear.h: products with 4-bit weights
LINEAR_EXPORTS = ("qstate_linear", "qstate_linear_bytes", "qstate_linear_pack",
                  "qstate_linear_quantize")


class QStateConfig(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("dk", ctypes.c_int32),
        ("dv", ctypes.c_int32), ("group", ctypes.c_int32), ("mixer", ctypes.c_int32),
        ("rounding", ctypes.c_int32), ("fp32_state", ctypes.c_int32),
        ("head_bits", ctypes.POINTER(ctypes.c_uint8)), ("seed", ctypes.c_uint64),
        ("layer", ctypes.c_uint32), ("group_axis", ctypes.c_int32),
        ("channel_bits", ctypes.POINTER(ctypes.c_uint8)), ("window", ctypes.c_int32),
        ("window_merge", ctypes.c_int32), ("lrb_threshold", ctypes.c_float),
    ]


class ScanConfigC(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("batch", "heads", "heads_qk", "dk", "dv", "mixer",
                                               "dtype", "pad")]
                + [(n, ctypes.c_int64) for n in ("tokens", "q_stride", "k_stride", "v_stride",
                                                 "o_stride")])


class NormConfigC(ctypes.Structure):
    _fields_ = ([("tokens", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("groups", "width", "dtype", "act",
                                                 "weight_groups")]
                + [("eps", ctypes.c_float)]
                + [(n, ctypes.c_int64) for n in ("x_stride", "gate_stride", "residual_stride")])


class DraftConfigC(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("tokens", "heads_qk", "dtype", "pad")]
                + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "v_stride")])


class GroupNormConfigC(ctypes.Structure):
    _fields_ = ([("tokens", ctypes.c_int64)]
                + [(n, ctypes.c_int32) for n in ("groups", "width", "dtype", "act", "mode", "center")]
                + [("eps", ctypes.c_float), ("shared", ctypes.c_int32)]
                + [(n, ctypes.c_int64) for n in ("x_stride", "gate_stride")])


class LinearConfigC(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("inputs", "outputs", "group", "dtype")]
                + [(n, ctypes.c_int64) for n in ("rows", "x_stride")])


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run "
                          "python -m bit_recurrent_state_amd.build")
    from . import build
    if all(os.path.exists(f) for f in build.SOURCES + build.HEADERS) and build.stale():
        raise ImportError(f"{LIB_PATH} was built from other sources or flags than those in "
                          "the package: run python -m bit_recurrent_state_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    P, c_int, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    cfgp = ctypes.POINTER(QStateConfig)
    sigs = {
        "qstate_state_bytes": (c_int, [cfgp, ctypes.POINTER(sz), ctypes.POINTER(sz)]),
        "qstate_create": (c_int, [cfgp, P, P, ctypes.POINTER(P)]),
        "qstate_load_fp32": (c_int, [P, P, P]),
        "qstate_step": (c_int, [P, P, P, P, P, P, P, P]),
        "qstate_readout": (c_int, [P, P, P, P]),
        "qstate_store_fp32": (c_int, [P, P, P]),
        "qstate_get_step": (c_int, [P, ctypes.POINTER(ctypes.c_uint64)]),
        "qstate_set_step": (c_int, [P, ctypes.c_uint64]),
        "qstate_destroy": (c_int, [P]),
        "qstate_strerror": (ctypes.c_char_p, [c_int]),
        "qstate_bits_by_decay": (c_int, [P, c_int, c_int, ctypes.c_float, ctypes.c_uint8,
                                         ctypes.c_uint8, P]),
        "qstate_ceiling_copy": (c_int, [P, P, sz, c_int, P]),
        "qstate_ceiling_rmw": (c_int, [P, sz, ctypes.c_uint32, c_int, P]),
        "qstate_scan_workspace": (c_int, [ctypes.POINTER(ScanConfigC), c_int, ctypes.POINTER(sz)]),
        "qstate_scan": (c_int, [ctypes.POINTER(ScanConfigC)] + [P] * 10 + [sz, P]),
        "qstate_norm": (c_int, [ctypes.POINTER(NormConfigC)] + [P] * 9),
        "qstate_norm_workspace": (c_int, [ctypes.POINTER(NormConfigC), ctypes.POINTER(sz)]),
        "qstate_norm_backward": (c_int, [ctypes.POINTER(NormConfigC)] + [P] * 6 + [c_int]
                                 + [P] * 9 + [sz, P]),
        "qstate_scan_backward": (c_int, [ctypes.POINTER(ScanConfigC)] + [P] * 16 + [sz, P]),
        "qstate_group_norm": (c_int, [ctypes.POINTER(GroupNormConfigC)] + [P] * 6),
        "qstate_group_norm_workspace": (c_int, [ctypes.POINTER(GroupNormConfigC),
                                                ctypes.POINTER(sz)]),
        "qstate_group_norm_backward": (c_int, [ctypes.POINTER(GroupNormConfigC)] + [P] * 10
                                       + [sz, P]),
        "qstate_linear": (c_int, [ctypes.POINTER(LinearConfigC)] + [P] * 6),
        "qstate_linear_bytes": (c_int, [ctypes.POINTER(LinearConfigC), ctypes.POINTER(sz),
                                        ctypes.POINTER(sz)]),
        "qstate_linear_pack": (c_int, [ctypes.POINTER(LinearConfigC)] + [P] * 5),
        "qstate_linear_quantize": (c_int, [ctypes.POINTER(LinearConfigC)] + [P] * 4),
        "qstate_verify": (c_int, [cfgp, ctypes.POINTER(DraftConfigC)] + [P] * 11),
        "qstate_accept": (c_int, [cfgp, ctypes.POINTER(DraftConfigC), ctypes.c_uint64] + [P] * 8),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype, fn.argtypes = res, args
    _lib = L
    return L


class QStateError(RuntimeError):
    def __init__(self, call: str, status: int):
        msg = lib().qstate_strerror(status).decode()
        super().__init__(f"{call} failed with status {status}: {msg}")
        self.status = status


def check(call: str, status: int) -> None:
    if status != QSTATE_OK:
        raise QStateError(call, status)
