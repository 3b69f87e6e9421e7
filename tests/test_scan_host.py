"""Host side of include/qstate_scan.h and qstate_norm.h (no GPU): exports,
argument checks before any launch, workspace sizes, the 64-bit reference
against differences."""

import ctypes
import os
import re

import pytest
import torch

from scan_reference import GDN, GLA, KDA, SCALAR, inputs, norm64, scan64

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


@pytest.mark.parametrize("header,listed", [("qstate_scan.h", "SCAN_EXPORTS"),
                                           ("qstate_norm.h", "NORM_EXPORTS")])
def test_exports_every_declared_symbol(L, header, listed):
    from bit_recurrent_state_amd import _lib
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = sorted(set(re.findall(r"^int\s+(qstate_\w+)\s*\(", text, re.M)))
    assert names == sorted(getattr(_lib, listed)) and len(names) == 3
    for n in names:
        assert hasattr(L, n), n


def _scan(**kw):
    from bit_recurrent_state_amd._lib import ScanConfigC
    base = dict(batch=2, heads=4, heads_qk=2, dk=128, dv=64, mixer=GDN, dtype=1, pad=0, tokens=128)
    base.update(kw)
    return ScanConfigC(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(tokens=0), OK), (dict(dv=1), OK), (dict(dv=4096, heads=256, heads_qk=1), OK),
    (dict(q_stride=256), OK), (dict(v_stride=1 << 22), OK),
    (dict(batch=0), INVALID), (dict(heads=0), INVALID), (dict(heads_qk=3), INVALID),
    (dict(heads_qk=0), INVALID), (dict(dv=0), INVALID), (dict(mixer=4), INVALID),
    (dict(dtype=3), INVALID), (dict(dtype=-1), INVALID), (dict(pad=1), INVALID),
    (dict(tokens=-1), INVALID), (dict(q_stride=255), INVALID), (dict(v_stride=-1), INVALID),
    (dict(dk=96), UNSUPPORTED), (dict(dk=512), UNSUPPORTED), (dict(heads=300, heads_qk=1), UNSUPPORTED),
    (dict(dv=4097), UNSUPPORTED), (dict(tokens=1 << 31), UNSUPPORTED),
    (dict(tokens=1 << 28), OK), (dict(tokens=1 << 29), UNSUPPORTED),
    (dict(batch=500000, tokens=0, dv=32), OK), (dict(batch=1100000, tokens=0, dv=32), UNSUPPORTED),
    (dict(o_stride=(1 << 22) + 8), UNSUPPORTED),
    (dict(tokens=1 << 28, heads_qk=4), UNSUPPORTED), (dict(tokens=1 << 26, heads_qk=4), OK),
])
def test_scan_configs(L, kw, status):
    n = ctypes.c_size_t(7)
    for backward in (0, 1):
        assert L.qstate_scan_workspace(_scan(**kw), backward, ctypes.byref(n)) == status
    assert (n.value > 7) == (status == OK)


def test_scan_refuses_before_any_launch(L):
    """Every call fails on its arguments: the pointers are not memory."""
    a = [P(4096 * (i + 1)) for i in range(16)]
    n = ctypes.c_size_t()

    def fwd(c, q=a[0], k=a[1], v=a[2], g=a[3], b=a[4], off=None, s0=None, o=a[5], s1=a[6], ws=a[7],
            nws=1 << 40):
        return L.qstate_scan(c, q, k, v, g, b, off, s0, o, s1, ws, nws, None)

    assert L.qstate_scan_workspace(None, 0, ctypes.byref(n)) == INVALID
    assert L.qstate_scan_workspace(_scan(), 2, ctypes.byref(n)) == INVALID
    assert L.qstate_scan_workspace(_scan(), 0, None) == INVALID
    assert fwd(_scan(batch=0)) == INVALID and fwd(_scan(dk=96)) == UNSUPPORTED
    for name in ("q", "k", "v", "g", "b", "ws"):
        assert fwd(_scan(), **{name: None}) == INVALID, name
    assert fwd(_scan(), o=None, s1=None) == INVALID
    assert fwd(_scan(tokens=127)) == INVALID  # not a multiple of the batch, and no offsets
    for name, by in (("q", 8), ("k", 8), ("v", 1), ("g", 4), ("b", 4), ("off", 4), ("s0", 4),
                     ("o", 1), ("s1", 8), ("ws", 16)):
        assert fwd(_scan(), **{name: P(4096 + by)}) == INVALID, name
    assert L.qstate_scan_workspace(_scan(), 0, ctypes.byref(n)) == OK
    assert fwd(_scan(), nws=n.value - 1) == INVALID

    def bwd(c, do=a[5], ds1=None, dq=a[6], dk=a[7], dv=a[8], dg=a[9], db=a[10], ds0=None, ws=a[11],
            nws=1 << 40):
        return L.qstate_scan_backward(c, a[0], a[1], a[2], a[3], a[4], None, None, do, ds1, dq, dk,
                                      dv, dg, db, ds0, ws, nws, None)

    for name in ("do", "dq", "dk", "dv", "dg", "db", "ws"):
        assert bwd(_scan(), **{name: None}) == INVALID, name
    for name, by in (("do", 8), ("ds1", 8), ("dq", 1), ("dv", 1), ("dg", 2), ("db", 2), ("ds0", 4),
                     ("ws", 128)):
        assert bwd(_scan(), **{name: P(4096 + by)}) == INVALID, name
    assert L.qstate_scan_workspace(_scan(), 1, ctypes.byref(n)) == OK
    assert bwd(_scan(), nws=n.value - 1) == INVALID


def _norm(**kw):
    from bit_recurrent_state_amd._lib import NormConfigC
    base = dict(tokens=5, groups=4, width=128, dtype=1, act=0, weight_groups=0, eps=1e-6)
    base.update(kw)
    return NormConfigC(**base)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(tokens=0), OK), (dict(width=1), OK), (dict(width=16384), OK),
    (dict(x_stride=512), OK), (dict(tokens=-1), INVALID), (dict(groups=0), INVALID),
    (dict(width=0), INVALID), (dict(dtype=3), INVALID), (dict(act=2), INVALID),
    (dict(weight_groups=2), INVALID), (dict(eps=0.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(gate_stride=511), INVALID),
    (dict(width=16385), UNSUPPORTED), (dict(groups=65536), UNSUPPORTED),
    (dict(tokens=1 << 31), UNSUPPORTED),
])
def test_norm_configs(L, kw, status):
    n = ctypes.c_size_t()
    assert L.qstate_norm_workspace(_norm(**kw), ctypes.byref(n)) == status


def test_norm_refuses_before_any_launch(L):
    a = [P(4096 * (i + 1)) for i in range(16)]

    def fwd(x=a[0], w=a[1], z=None, res=None, sc=None, nw=a[2], r=a[3], h=a[4], c=None):
        return L.qstate_norm(c or _norm(), x, w, z, res, sc, nw, r, h, None)

    assert fwd(x=None) == INVALID and fwd(r=None, h=None, nw=None) == INVALID
    assert fwd(h=None) == INVALID  # next_weight without h
    for name, by in (("x", 1), ("w", 2), ("z", 1), ("res", 1), ("sc", 2), ("nw", 2), ("r", 1), ("h", 1)):
        assert fwd(**{name: P(4096 + by)}) == INVALID, name
    assert fwd(c=_norm(tokens=0)) == OK  # nothing to do

    def bwd(x=a[0], z=None, nw=None, has_h=0, dr=a[1], dh=None, dx=a[2], dz=None, dw=a[3], dnw=None,
            ws=a[4], nws=1 << 40):
        return L.qstate_norm_backward(_norm(), x, None, z, None, None, nw, has_h, dr, dh, dx, dz, None,
                                      dw, None, dnw, ws, nws, None)

    assert bwd(x=None) == INVALID and bwd(has_h=2) == INVALID
    assert bwd(dz=a[5]) == INVALID  # a gate's gradient without a gate
    assert bwd(dh=a[5]) == INVALID and bwd(nw=a[5]) == INVALID and bwd(dnw=a[5]) == INVALID
    assert bwd(ws=None) == INVALID and bwd(nws=16) == INVALID and bwd(ws=P(4096 + 64)) == INVALID


def test_python_refuses_host_tensors():
    from bit_recurrent_state_amd import block_norm, scan
    x = inputs(GDN, 1, [3], 2, 2, 64, 8, torch.float32, "cpu")
    with pytest.raises(TypeError):
        scan(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], mixer=GDN, offsets=x["offsets"])
    with pytest.raises(TypeError):
        block_norm(torch.zeros(2, 8))


@pytest.mark.parametrize("mixer", [GDN, GLA, SCALAR, KDA])
def test_reference_gradients_against_differences(mixer):
    """The 64-bit reference that the GPU tests use, along random directions."""
    x = inputs(mixer, 2, [5, 3], 2, 1, 64, 3, torch.float64, "cpu")
    x = {n: t.double() if t is not None and n != "offsets" else t for n, t in x.items()}
    g = torch.Generator().manual_seed(1)
    co = torch.randn(x["v"].shape, generator=g, dtype=torch.float64)

    def loss(y, grad=False):
        o, S, leaf = scan64(y, mixer, 2, grad)
        return (o * co).sum() + 0.1 * S.sum(), leaf

    value, leaf = loss(x, True)
    value.backward()
    h = 1e-6
    for n, t in leaf.items():
        if t is None:
            continue
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        up, down = ({**x, n: x[n] + s * h * d} for s in (1, -1))
        diff = float(loss(up)[0] - loss(down)[0]) / (2 * h)
        assert abs(diff - float((t.grad * d).sum())) <= 1e-7 * (1.0 + abs(diff)), n


def test_norm_reference_gradients_against_differences():
    g = torch.Generator().manual_seed(2)
    args = [torch.randn(3, 4, 16, generator=g, dtype=torch.float64) for _ in range(3)]
    args = [args[0], torch.randn(16, generator=g, dtype=torch.float64), args[1], args[2],
            torch.randn(16, generator=g, dtype=torch.float64),
            torch.randn(16, generator=g, dtype=torch.float64)]
    leaves = [t.clone().requires_grad_(True) for t in args]

    def loss(a):
        r, h = norm64(*a, 1e-6, 0)
        return (r.sin() + h.cos()).sum()

    loss(leaves).backward()
    for i, t in enumerate(args):
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        up, down = ([a + s * 1e-6 * d if j == i else a for j, a in enumerate(args)] for s in (1, -1))
        diff = float(loss(up) - loss(down)) / 2e-6
        assert abs(diff - float((leaves[i].grad * d).sum())) <= 1e-7 * (1.0 + abs(diff)), i


def test_captured_backward_beside_an_eager_graph_is_refused(monkeypatch):
    """The rule itself, on the CPU: another stream's live graph of the same leaf, and only that."""
    import gc

    from bit_recurrent_state_amd import sequence

    class Twice(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, stream):
            sequence._alive[ctx] = stream
            return 2 * x

        @staticmethod
        def backward(ctx, d):
            sequence._refuse_capture(ctx, None)
            return 2 * d, None

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    monkeypatch.setattr(sequence, "_stream", lambda stream, device: 7)
    x, other = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    capturing = False
    eager, y = Twice.apply(x, 1), Twice.apply(x, 7)
    far = Twice.apply(other, 1)
    torch.autograd.grad(y.sum(), x, retain_graph=True)
    capturing = True
    with pytest.raises(RuntimeError, match="drop the results"):
        torch.autograd.grad(y.sum(), x, retain_graph=True)
    del eager
    gc.collect()
    (d,) = torch.autograd.grad(y.sum(), x)
    assert torch.equal(d, torch.full((3,), 2.0)) and far.requires_grad
    n = len(sequence._alive)
    del y, far
    gc.collect()
    assert len(sequence._alive) == n - 2


def test_readout_norm_shapes(L):
    """Right sizes in wrong shapes are refused, whatever the device."""
    from bit_recurrent_state_amd import ReadoutNorm
    shape, heads, dv = (6, 4, 32), 4, 32

    def config(o_shape=None, **kw):
        return ReadoutNorm(**kw).config(shape, torch.float32, torch.device("cpu"), o_shape)

    for kw in (dict(weight=torch.ones(dv, heads)), dict(weight=torch.ones(heads * dv)),
               dict(weight=torch.ones(dv + 1)), dict(weight=torch.tensor(1.0)),
               dict(gate=torch.ones(4, 6, 32)), dict(gate=torch.ones(6, 32, 4)),
               dict(gate=torch.ones(2, 3, 4, 32)), dict(gate=torch.ones(3, 2, 4, 32), o_shape=(2, 3, 4, 32))):
        with pytest.raises(ValueError):
            config(**kw)
    for kw in (dict(weight=torch.ones(dv)), dict(weight=torch.ones(heads, dv)), dict(gate=torch.ones(shape)),
               dict(gate=torch.ones(6 * 4 * 32)), dict(gate=torch.ones(2, 3, 4, 32), o_shape=(2, 3, 4, 32))):
        with pytest.raises(TypeError, match="device tensor"):  # the next check: the shapes passed
            config(**kw)


def _noted(monkeypatch, capturing):
    """A stand-in for the operators: noted and checked as they are, on the CPU."""
    from bit_recurrent_state_amd import sequence

    class Noted(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, stream):
            with sequence._alive_lock:
                sequence._alive[ctx] = stream
            return 2 * x

        @staticmethod
        def backward(ctx, d):
            sequence._refuse_capture(ctx, None)
            return 2 * d, None

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(sequence, "_stream", lambda stream, device: 7)
    return Noted.apply


@pytest.mark.parametrize("through", ["projection", "views", "both operators"])
def test_captured_backward_sees_leaves_behind_other_operations(monkeypatch, through):
    """The shared leaf is a weight whose product enters the operators, as in a layer."""
    import gc
    capturing = [False]
    op = _noted(monkeypatch, capturing)
    x, W = torch.ones(4, 3), torch.ones(3, 3, requires_grad=True)
    W2 = torch.ones(3, 3, requires_grad=True)

    def call(W, stream):
        if through == "views":
            return op(W.view(9)[1:].unflatten(0, (2, 4)).transpose(0, 1), stream)
        y = op(torch.relu(x @ W), stream)
        return op(y @ W2.detach(), stream) if through == "both operators" else y

    eager, mine = call(W, 1), call(W, 7)
    capturing[0] = True
    with pytest.raises(RuntimeError, match="drop the results"):
        torch.autograd.grad(mine.sum(), W, retain_graph=True)
    other = call(W2, 1)  # another leaf's graph does not matter
    del eager
    gc.collect()
    torch.autograd.grad(mine.sum(), W)
    assert other.requires_grad


def test_captured_backward_while_other_threads_begin_calls(monkeypatch):
    """The list of live calls is read while other threads add to it and drop from it."""
    import threading
    capturing = [True]
    op = _noted(monkeypatch, capturing)
    x, other = torch.ones(3, requires_grad=True), torch.ones(3, requires_grad=True)
    stop, failed = threading.Event(), []

    def begin():
        try:
            kept = []
            while not stop.is_set():
                kept.append(op(other, 1))
                del kept[:-50]
        except Exception as e:  # noqa
            failed.append(e)

    threads = [threading.Thread(target=begin) for _ in range(3)]
    for t in threads:
        t.start()
    try:
        for _ in range(300):
            torch.autograd.grad(op(x, 7).sum(), x)
    finally:
        stop.set()
        for t in threads:
            t.join()
    assert not failed


def test_tracing_is_refused_and_forward_mode_goes_through_autograd():
    from torch.autograd import forward_ad
    from torch.fx.experimental.proxy_tensor import make_fx

    from bit_recurrent_state_amd import block_norm, scan
    from bit_recurrent_state_amd.sequence import _through_autograd
    x, s = torch.randn(3, 8), inputs(GDN, 1, [3], 2, 2, 64, 8, torch.float32, "cpu")

    def call(v):
        return scan(s["q"], s["k"], v, s["log_alpha"], s["beta"], mixer=GDN, offsets=s["offsets"])[0]

    for f, a in ((lambda x: block_norm(x), x), (call, s["v"])):
        with pytest.raises(RuntimeError, match="traced"):
            make_fx(f)(a)
        with pytest.raises(RuntimeError, match="traced"):
            torch.jit.trace(f, a)
        with pytest.raises(TypeError, match="device tensor"):  # and no longer after it
            f(a)
    assert not _through_autograd((x, None))
    with forward_ad.dual_level():
        assert _through_autograd((x, None))
        with torch.no_grad():
            assert _through_autograd((forward_ad.make_dual(x, x),))
    assert _through_autograd((x.clone().requires_grad_(True),)) and not _through_autograd((x,))
