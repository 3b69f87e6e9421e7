"""Host side of include/qstate_draft.h (no GPU): exports, argument checks before
any launch, the 64-bit reference against the recurrence token by token."""

import ctypes
import os
import re

import pytest
import torch

from draft_reference import GDN, GLA, KDA, MIXERS, accept64, inputs, node_mask, verify64

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


def test_exports_every_declared_symbol(L):
    from bit_recurrent_state_amd import _lib
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qstate_draft.h")).read(),
                  flags=re.S)
    names = sorted(set(re.findall(r"^int\s+(qstate_\w+)\s*\(", text, re.M)))
    assert names == sorted(_lib.DRAFT_EXPORTS)
    for n in names:
        assert hasattr(L, n), n


def _state(**kw):
    from bit_recurrent_state_amd import Config
    base = dict(batch=2, heads=4, dk=128, dv=64, group=32, mixer=GDN)
    base.update(kw)
    return Config(**base).to_c()


def _draft(**kw):
    from bit_recurrent_state_amd._lib import DraftConfigC
    base = dict(tokens=8, heads_qk=2, dtype=1, pad=0)
    base.update(kw)
    return DraftConfigC(**base)


def _calls(L, state, draft, skip=(), **kw):
    """Statuses of verify and accept with pointers that are not memory (never reached: every call
    below fails on its arguments)."""
    c, _keep = state
    a = dict(codes=P(4096), scales=P(8192), q=P(4096), k=P(4096), v=P(4096), g=P(4096), b=P(4096),
             parents=None, o=P(4096), writes=P(4096), last=P(4096))
    a.update(kw)
    v = L.qstate_verify(ctypes.byref(c) if c else None, draft, a["codes"], a["scales"], a["q"], a["k"],
                        a["v"], a["g"], a["b"], a["parents"], a["o"], a["writes"], None) \
        if "verify" not in skip else None
    w = L.qstate_accept(ctypes.byref(c) if c else None, draft, 0, a["codes"], a["scales"], a["k"],
                        a["g"], a["parents"], a["writes"], a["last"], None) \
        if "accept" not in skip else None
    return v, w


@pytest.mark.parametrize("state,draft,status", [
    (dict(batch=0), {}, INVALID), (dict(dk=96), {}, UNSUPPORTED), (dict(mixer=4), {}, INVALID),
    (dict(group=24), {}, INVALID), (dict(window=4), {}, UNSUPPORTED),
    (dict(group_axis=1), {}, UNSUPPORTED), (dict(heads=300), {}, UNSUPPORTED),
    (dict(batch=1 << 23), {}, UNSUPPORTED),
    ({}, dict(tokens=0), INVALID), ({}, dict(tokens=-1), INVALID), ({}, dict(tokens=65), UNSUPPORTED),
    (dict(dk=256), dict(tokens=33), UNSUPPORTED), ({}, dict(heads_qk=0), INVALID),
    ({}, dict(heads_qk=3), INVALID), ({}, dict(dtype=3), INVALID), ({}, dict(dtype=-1), INVALID),
    ({}, dict(pad=1), INVALID), ({}, dict(q_stride=255), INVALID), ({}, dict(k_stride=-1), INVALID),
    ({}, dict(v_stride=255), INVALID), ({}, dict(q_stride=(1 << 22) + 8), UNSUPPORTED),
    ({}, dict(v_stride=(1 << 22) + 8), UNSUPPORTED),
])
def test_configs(L, state, draft, status):
    assert _calls(L, _state(**state), _draft(**draft)) == (status, status)


def test_refuses_before_any_launch(L):
    both = (INVALID, INVALID)
    assert _calls(L, (None, None), _draft()) == both
    assert _calls(L, _state(), None) == both
    for name in ("codes", "scales", "k", "g"):
        assert _calls(L, _state(), _draft(), **{name: None}) == both, name
    for name, by in (("codes", 8), ("scales", 4), ("k", 8), ("g", 4), ("writes", 8), ("parents", 2)):
        assert _calls(L, _state(), _draft(), **{name: P(4096 + by)}) == both, name
    for name in ("q", "v", "b"):
        assert _calls(L, _state(), _draft(), skip=("accept",), **{name: None})[0] == INVALID, name
    for name, by in (("q", 8), ("v", 1), ("o", 1), ("b", 2)):
        assert _calls(L, _state(), _draft(), skip=("accept",), **{name: P(4096 + by)})[0] == INVALID
    assert _calls(L, _state(), _draft(), skip=("accept",), o=None, writes=None)[0] == INVALID
    for name in ("writes", "last"):
        assert _calls(L, _state(), _draft(), skip=("verify",), **{name: None})[1] == INVALID
    assert _calls(L, _state(), _draft(), skip=("verify",), last=P(4098))[1] == INVALID


def test_python_refuses_host_tensors():
    from bit_recurrent_state_amd import Config, DraftConfig, qstate_accept, qstate_verify
    x, S = inputs(GDN, 2, 3, "tree", 2, 2, 64, 16, torch.float32, "cpu")
    cfg = Config(2, 2, 64, 16, mixer=GDN, fp32_state=True)
    with pytest.raises(TypeError):
        qstate_verify(cfg, DraftConfig(3, 2), S.flatten(), None, x["q"], x["k"], x["v"],
                      x["log_alpha"], x["beta"], x["parents"], x["v"].clone())
    with pytest.raises(TypeError):
        qstate_accept(cfg, DraftConfig(3, 2), 0, S.flatten(), None, x["k"], x["log_alpha"],
                      x["parents"], x["v"], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        DraftConfig(3, 2, torch.float64).to_c()


@pytest.mark.parametrize("mixer", MIXERS)
def test_reference_of_a_chain(mixer):
    """The tree's definition on a chain is the recurrence of the packed scan."""
    from scan_reference import scan64
    m = MIXERS[mixer]
    x, S = inputs(m, 2, 5, "chain", 2, 1, 64, 8, torch.float64, "cpu")
    o, writes, states = verify64(x, S, m)
    y = {n: None if x[n] is None else x[n].flatten(0, 1) for n in ("q", "k", "v", "log_alpha", "beta")}
    y.update(initial_state=S, offsets=torch.tensor([0, 5, 10]))
    o2, S2, _ = scan64(y, m, 2)
    assert torch.allclose(o.flatten(0, 1), o2, rtol=1e-12, atol=1e-14)
    assert torch.allclose(accept64(x, S, states, torch.tensor([4, 4])), S2, rtol=1e-12, atol=1e-14)
    assert torch.equal(accept64(x, S, states, torch.tensor([-1, 7])), S.double())


def test_reference_of_branches():
    """Two children of one node do not see each other, and padding is no node."""
    x, S = inputs(KDA, 1, 4, "chain", 1, 1, 64, 4, torch.float64, "cpu")
    x["parents"] = torch.tensor([[-1, 0, 0, -2]], dtype=torch.int32)
    assert node_mask(x["parents"]).tolist() == [[True, True, True, False]]
    o, w, _ = verify64(x, S, KDA)
    y = {n: None if t is None else t[:, [0, 2]].contiguous() for n, t in x.items()}
    y["parents"] = torch.tensor([[-1, 0]], dtype=torch.int32)
    o2, w2, _ = verify64(y, S, KDA)
    assert torch.equal(o[:, [0, 2]], o2) and torch.equal(w[:, [0, 2]], w2)
    assert not o[:, 3].any() and not w[:, 3].any()
    assert GLA != KDA


def test_a_handle_keeps_its_configuration(monkeypatch):
    """A configuration that is changed for the next handle: the first one's calls still go by the sizes
    of its memory, and refuse others before the library is reached."""
    from bit_recurrent_state_amd import Config, Draft, QState, draft, qstate
    calls = []
    monkeypatch.setattr(qstate, "qstate_create", lambda *a: None)
    monkeypatch.setattr(qstate, "qstate_get_step", lambda h: 0)
    monkeypatch.setattr(qstate, "qstate_set_step", lambda h, s: None)
    monkeypatch.setattr(draft, "_on_device", lambda *a: None)
    monkeypatch.setattr(draft, "_stream", lambda *a: None)
    monkeypatch.setattr(draft, "_call", lambda *a: calls.append(a) or 0)
    bits = [8, 4]
    cfg = Config(4, 2, 64, 16, mixer=GDN, head_bits=bits)
    st = QState(cfg, device="cpu")
    cfg.batch, cfg.heads, cfg.dv = 2, 1, 8
    bits[0] = 4
    few, _ = inputs(GDN, 2, 3, "chain", 1, 1, 64, 8, torch.float32, "cpu")
    names = ("q", "k", "v", "log_alpha", "beta")
    with pytest.raises(ValueError):
        st.verify(*(few[n] for n in names))
    last = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        st.accept(Draft(few["k"], few["log_alpha"], None, few["v"]), last)
    assert not calls
    x, _ = inputs(GDN, 4, 3, "chain", 2, 2, 64, 16, torch.float32, "cpu")
    _, d = st.verify(*(x[n] for n in names))
    st.accept(d, torch.zeros(4, dtype=torch.int32))
    assert len(calls) == 2
    assert st.cfg.bits().tolist() == [[8] * 4, [4] * 4]
