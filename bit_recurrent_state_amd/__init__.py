"""Quantized recurrent-state decode step for MI355X (gfx950).

The C ABI (include/qstate.h, qstate_scan.h, qstate_norm.h, qstate_draft.h,
qstate_group_norm.h, qstate_linear.h) is implemented by libqstate.so, built from
csrc/ with hipcc; this package is its thin Python binding."""

from .qstate import (BDR, GDN, GLA, KDA, KEY_AXIS, RTN, SCALAR, SR, VALUE_AXIS, Config, QState, ReadoutNorm,  # noqa
                     qstate_bits_by_decay,
                     qstate_create, qstate_destroy, qstate_get_step, qstate_load_fp32,
                     qstate_readout, qstate_set_step, qstate_state_bytes, qstate_step,
                     qstate_store_fp32)
from .draft import Draft, DraftConfig, qstate_accept, qstate_verify  # noqa
from .group_norm import (ACTIVATE, GATE, GATE_FIRST, PLAIN, GroupNormConfig, group_norm,  # noqa
                         qstate_group_norm, qstate_group_norm_backward, qstate_group_norm_workspace)
from .linear import (LinearConfig, Weight4, linear4, qstate_linear, qstate_linear_bytes,  # noqa
                     qstate_linear_pack, qstate_linear_quantize)
from .norm import (SIGMOID, SILU, NormConfig, block_norm, qstate_norm, qstate_norm_backward,  # noqa
                   qstate_norm_workspace)
from .sequence import ScanConfig, qstate_scan, qstate_scan_backward, qstate_scan_workspace, scan  # noqa
