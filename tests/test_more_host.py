"""Host side of include/qstate_group_norm.h and qstate_linear.h (no GPU): exports
and argument checks before any launch."""

import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED = 0, -1, -2


@pytest.fixture(scope="module")
def L():
    from bit_recurrent_state_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    from bit_recurrent_state_amd._lib import lib
    return lib()


@pytest.mark.parametrize("header,listed", [("qstate_group_norm.h", "GROUP_NORM_EXPORTS"),
                                           ("qstate_linear.h", "LINEAR_EXPORTS")])
def test_exports_every_declared_symbol(L, header, listed):
    from bit_recurrent_state_amd import _lib
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"^int\s+(qstate_\w+)\s*\(", text, re.M)))
    assert names == sorted(getattr(_lib, listed))
    for n in names:
        assert hasattr(L, n), n


def _norm(**kw):
    from bit_recurrent_state_amd._lib import GroupNormConfigC
    base = dict(tokens=5, groups=4, width=128, dtype=1, act=0, mode=0, center=1, eps=1e-5, shared=0)
    base.update(kw)
    return GroupNormConfigC(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(tokens=0), OK), (dict(width=1), OK), (dict(width=16384), OK),
    (dict(x_stride=512), OK), (dict(shared=1), OK), (dict(tokens=-1), INVALID),
    (dict(groups=0), INVALID), (dict(width=0), INVALID), (dict(dtype=3), INVALID),
    (dict(act=2), INVALID), (dict(mode=4), INVALID), (dict(mode=-1), INVALID),
    (dict(center=2), INVALID), (dict(shared=2), INVALID), (dict(eps=0.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(gate_stride=511), INVALID), (dict(x_stride=-1), INVALID),
    (dict(width=16385), UNSUPPORTED), (dict(groups=65536), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED), (dict(x_stride=(1 << 40) + 8), UNSUPPORTED),
])
def test_norm_configs(L, kw, status):
    n = ctypes.c_size_t(7)
    assert L.qstate_group_norm_workspace(_norm(**kw), ctypes.byref(n)) == status
    assert (n.value != 7) == (status == OK)


def test_norm_refuses_before_any_launch(L):
    a = P(4096)
    n = ctypes.c_size_t()

    def fwd(c, x=a, w=a, b=a, z=None, y=a):
        return L.qstate_group_norm(c, x, w, b, z, y, None)

    assert L.qstate_group_norm_workspace(None, ctypes.byref(n)) == INVALID
    assert L.qstate_group_norm_workspace(_norm(), None) == INVALID
    assert fwd(_norm(tokens=0), x=None, y=None) == OK
    for kw in (dict(x=None), dict(y=None), dict(z=a), dict(x=P(4097)), dict(w=P(4098)), dict(b=P(4098)),
               dict(y=P(4097))):
        assert fwd(_norm(), **kw) == INVALID, kw
    for mode in (1, 2):
        assert fwd(_norm(mode=mode)) == INVALID
        assert fwd(_norm(mode=mode), z=P(4097)) == INVALID

    def bwd(c, x=a, z=None, dy=a, dx=a, dz=None, dw=a, db=a, ws=a, nws=1 << 40):
        return L.qstate_group_norm_backward(c, x, a, a, z, dy, dx, dz, dw, db, ws, nws, None)

    for kw in (dict(x=None), dict(dy=None), dict(dz=a), dict(z=a), dict(ws=None), dict(ws=P(4096 + 128)),
               dict(dx=P(4097)), dict(dw=P(4098))):
        assert bwd(_norm(), **kw) == INVALID, kw
    assert L.qstate_group_norm_workspace(_norm(), ctypes.byref(n)) == OK
    assert bwd(_norm(), nws=n.value - 1) == INVALID
    assert bwd(_norm(tokens=0), x=None, dy=None, dw=None, db=None, ws=None) == OK


def _linear(**kw):
    from bit_recurrent_state_amd._lib import LinearConfigC
    base = dict(inputs=256, outputs=100, group=64, dtype=1, rows=3, x_stride=0)
    base.update(kw)
    return LinearConfigC(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(rows=0), OK), (dict(outputs=1), OK), (dict(inputs=1 << 20, outputs=1), OK),
    (dict(outputs=1 << 20, inputs=128), OK), (dict(x_stride=256), OK), (dict(rows=1 << 19), OK),
    (dict(inputs=0), INVALID), (dict(outputs=0), INVALID), (dict(rows=-1), INVALID),
    (dict(group=0), INVALID), (dict(inputs=96, group=64), INVALID), (dict(dtype=3), INVALID),
    (dict(x_stride=255), INVALID), (dict(x_stride=-1), INVALID), (dict(group=16), UNSUPPORTED),
    (dict(group=256), UNSUPPORTED), (dict(inputs=1 << 21), UNSUPPORTED),
    (dict(outputs=(1 << 20) + 1), UNSUPPORTED), (dict(rows=(1 << 19) + 1), UNSUPPORTED),
    (dict(inputs=1 << 20, outputs=1 << 15), UNSUPPORTED),
])
def test_linear_configs(L, kw, status):
    a, b = ctypes.c_size_t(7), ctypes.c_size_t(7)
    assert L.qstate_linear_bytes(_linear(**kw), ctypes.byref(a), ctypes.byref(b)) == status
    assert (a.value != 7) == (status == OK)


def test_linear_sizes(L):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.qstate_linear_bytes(_linear(outputs=17, inputs=192), ctypes.byref(a), ctypes.byref(b)) == OK
    assert a.value == 4 * 1024 and b.value == 4 * 16 * 2 * 4
    assert L.qstate_linear_bytes(_linear(), None, ctypes.byref(b)) == INVALID


def test_linear_refuses_before_any_launch(L):
    a = P(4096)

    def mul(c, x=a, w=a, s=a, b=None, y=a):
        return L.qstate_linear(c, x, w, s, b, y, None)

    assert mul(None) == INVALID
    assert mul(_linear(rows=0), x=None, y=None) == OK
    for kw in (dict(x=None), dict(w=None), dict(s=None), dict(y=None), dict(x=P(4104)), dict(w=P(4104)),
               dict(s=P(4100)), dict(b=P(4098)), dict(y=P(4097))):
        assert mul(_linear(), **kw) == INVALID, kw
    assert mul(_linear(x_stride=257)) == INVALID

    def pack(c, codes=a, gs=a, w=a, s=a):
        return L.qstate_linear_pack(c, codes, gs, w, s, None)

    for kw in (dict(codes=None), dict(gs=None), dict(w=None), dict(s=None), dict(gs=P(4098)),
               dict(w=P(4104)), dict(s=P(4104))):
        assert pack(_linear(), **kw) == INVALID, kw

    def quantize(c, v=a, w=a, s=a):
        return L.qstate_linear_quantize(c, v, w, s, None)

    for kw in (dict(v=None), dict(w=None), dict(s=None), dict(v=P(4097)), dict(w=P(4104)),
               dict(s=P(4104))):
        assert quantize(_linear(), **kw) == INVALID, kw


def test_python_refuses_host_tensors(L):
    from bit_recurrent_state_amd import (GroupNormConfig, LinearConfig, Weight4, group_norm,
                                         qstate_group_norm, qstate_linear_quantize)
    x = torch.zeros(2, 128)
    with pytest.raises(TypeError):
        group_norm(x, 2)
    with pytest.raises(TypeError):
        qstate_group_norm(GroupNormConfig(2, 2, 64), x, y=x)
    with pytest.raises(TypeError):
        Weight4.quantize(x)
    with pytest.raises(TypeError):
        qstate_linear_quantize(LinearConfig(128, 2), x, x, x)
    for c in (GroupNormConfig(2, 2, 64, torch.float64), LinearConfig(128, 2, dtype=torch.int8)):
        with pytest.raises(ValueError):
            c.to_c()
