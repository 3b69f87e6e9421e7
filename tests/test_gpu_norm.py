"""The block norm and its gradients against 64 bits (GPU)."""

import itertools

import pytest
import torch

from scan_reference import norm64, rel

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = ("x", "weight", "gate", "residual", "scale", "next_weight")

# FP32 between inputs and outputs: a row's sums of w squares err by at most
# (2 + log2 of the terms a thread and a tree add) roundings, the elementwise
# parts by some ten more: 32 * 2^-24 of the norm.  Weights' gradients are sums
# over rows of such terms of either sign, whose norm is about sqrt(rows) of the
# terms' against sums of up to 128 rows a team in FP32: twice that.
BASE = 32 * 2.0 ** -24


def tol(dtype):
    return BASE if dtype == torch.float32 else torch.finfo(dtype).eps / 2 + BASE


def make(rows, groups, width, dtype, gate, residual, scale, each, nxt, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (rows, groups, width) if groups else (rows, width)

    def normal(*s):
        return torch.randn(s, generator=g)

    x = {"x": normal(*shape).to(dtype), "weight": 1 + 0.1 * normal(*(shape[1:] if each else shape[-1:])),
         "gate": 2 * normal(*shape), "residual": normal(*shape), "scale": 0.5 + 0.1 * normal(width),
         "next_weight": 1 + 0.1 * normal(width)}
    for n, on in (("gate", gate), ("residual", residual), ("scale", scale), ("next_weight", nxt)):
        x[n] = x[n].to(dtype if n in ("gate", "residual") else torch.float32) if on else None
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def run(x, act=0, eps=1e-6, **kw):
    from bit_recurrent_state_amd import block_norm
    y = block_norm(x["x"], act=act, eps=eps, **{n: x[n] for n in NAMES[1:]}, **kw)
    return y if isinstance(y, tuple) else (y,)


def check(x, act=0, eps=1e-6, seeds=None):
    dt = x["x"].dtype
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items() if t is not None}
    out = run({**x, **leaves}, act, eps)
    l64 = {n: t.double().requires_grad_(True) for n, t in x.items() if t is not None}
    want = norm64(*(l64.get(n) for n in NAMES), eps, act)
    assert len(out) == len(want)
    for a, b in zip(out, want):
        assert a.dtype == dt and a.shape == x["x"].shape
        assert rel(a, b) <= tol(dt)
    g = torch.Generator().manual_seed(9)
    seeds = [torch.randn(a.shape, generator=g).to(dt).cuda() for a in out]
    got = torch.autograd.grad(out, list(leaves.values()), seeds)
    exact = torch.autograd.grad(want, list(l64.values()), [s.double() for s in seeds])
    for n, a, b in zip(leaves, got, exact):
        assert a.dtype == x[n].dtype and a.shape == x[n].shape
        sums = n in ("weight", "scale", "next_weight")
        assert rel(a, b) <= (2 * BASE if sums else tol(a.dtype)), n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,groups,width", [(1, 0, 8), (37, 3, 64), (5, 0, 513), (3, 2, 100),
                                               (2, 0, 1), (300, 4, 128), (9, 0, 2048), (4, 0, 4096),
                                               (3, 0, 5000), (2, 0, 8192), (2, 0, 16384), (2, 0, 9999)])
def test_widths(dtype, rows, groups, width):
    """With width 1, n is x / |x|: its own gradient is a difference of equal numbers and not checked."""
    x = make(rows, groups, width, TYPES[dtype], True, True, True, False, True)
    if width > 1:
        check(x)
    else:
        out = run(x)
        want = norm64(*(None if x[n] is None else x[n].double() for n in NAMES), 1e-6, 0)
        assert all(rel(a, b) <= tol(TYPES[dtype]) for a, b in zip(out, want))


@pytest.mark.parametrize("gate,residual,scale,each,nxt", itertools.product([0, 1], repeat=5))
def test_parts(gate, residual, scale, each, nxt):
    for dtype, width in ((torch.bfloat16, 64), (torch.float32, 700)):
        check(make(19, 3, width, dtype, gate, residual, scale, each, nxt), act=gate and each)


def test_without_weight():
    x = make(40, 2, 128, torch.float32, True, False, False, False, True)
    x["weight"] = None
    check(x)


def test_many_rows():
    """More rows than teams: every team sums several rows into the weights' gradients."""
    check(make(9000, 4, 64, torch.bfloat16, True, True, True, False, True))
    check(make(3000, 7, 64, torch.float32, True, False, False, True, False))
    check(make(1500, 0, 1030, torch.float16, True, True, False, False, True))


def test_strides_views_and_places():
    """Gate and x as parts of wider rows; in place over x and over the residual."""
    from bit_recurrent_state_amd import NormConfig, qstate_norm
    x = make(50, 4, 64, torch.bfloat16, True, True, True, False, True)
    want = run(x)
    wide = torch.cat([x["x"].flatten(1), x["gate"].flatten(1), x["residual"].flatten(1)[:, :3]], 1)
    for off in (0, 3):
        w = torch.cat([wide[:, :off], wide], 1)
        part = {"x": w[:, off:off + 256].view(50, 4, 64), "gate": w[:, off + 256:off + 512].view(50, 4, 64)}
        got = run({**x, **part})
        assert all(rel(a, b) <= tol(torch.bfloat16) for a, b in zip(got, want))
    t = {n: x[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("x", "gate", "residual")}
    assert all(torch.equal(a, b) for a, b in zip(run({**x, **t}), want))
    c = NormConfig(50, 4, 64, torch.bfloat16)
    r, h = x["residual"].clone(), x["x"].clone()
    qstate_norm(c, h, x["weight"], x["gate"], r, x["scale"], x["next_weight"], r, h)
    assert torch.equal(r, want[0]) and torch.equal(h, want[1])
    only = torch.empty_like(h)
    qstate_norm(c, x["x"], x["weight"], x["gate"], x["residual"], x["scale"], x["next_weight"], None, only)
    assert torch.equal(only, want[1])


def test_extremes():
    """Rows of zeros, huge and tiny values, gates at both ends; NaN and infinity stay in their row."""
    x = make(8, 0, 256, torch.float32, True, True, False, False, True)
    x["x"][0] = 0
    x["x"][1] *= 1e15
    x["x"][2] *= 1e-15
    x["gate"][3] = 80.0
    x["gate"][4] = -80.0
    out = run(x)
    want = norm64(*(None if x[n] is None else x[n].double() for n in NAMES), 1e-6, 0)
    for a, b in zip(out, want):
        assert all(rel(a[i], b[i]) <= BASE for i in range(8))
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["x"][5, 17] = float("nan")
    y["gate"][6, 3] = float("inf")
    bad = run(y)
    for a, b in zip(bad, out):
        keep = [0, 1, 2, 3, 4, 7]
        assert torch.equal(a[keep], b[keep])
        assert a[5].isnan().all() if a is bad[1] else a[5].isnan().any()
    z = make(4, 0, 64, torch.float32, True, False, False, False, False)
    z["gate"][0] = float("inf")
    z["gate"][1] = -float("inf")
    z["gate"][2, 5] = float("nan")
    (s,) = run(z, act=1)
    n = norm64(z["x"].double(), z["weight"].double(), None, None, None, None, 1e-6, 0)[0]
    assert rel(s[0], n[0]) <= BASE and not s[1].abs().gt(1e-30).any()
    assert s[2].isnan().sum() == 1 and s[2, 5].isnan()


def test_empty_and_partial_gradients():
    from bit_recurrent_state_amd import block_norm
    x = torch.zeros(0, 4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    y = block_norm(x, weight=w)
    y.sum().backward()
    assert y.shape == x.shape and x.grad.shape == x.shape and not w.grad.any()
    x = make(30, 0, 128, torch.float32, True, True, True, False, True)
    for which in (0, 1):  # a loss of r alone, of h alone
        leaves = {n: t.clone().requires_grad_(n in ("gate", "scale")) for n, t in x.items()}
        run({**x, **leaves})[which].sum().backward()
        l64 = {n: t.double().requires_grad_(True) for n, t in x.items()}
        norm64(*(l64[n] for n in NAMES), 1e-6, 0)[which].sum().backward()
        for n in NAMES:
            if n in ("gate", "scale"):
                assert rel(leaves[n].grad, l64[n].grad) <= 2 * BASE
            else:
                assert leaves[n].grad is None


def test_same_bits_streams_and_graph():
    from bit_recurrent_state_amd import NormConfig, qstate_norm, qstate_norm_backward, qstate_norm_workspace
    xs = [make(700, 4, 64, torch.bfloat16, True, True, True, False, True, seed=s) for s in range(3)]
    c = NormConfig(700, 4, 64, torch.bfloat16)
    x = {n: t.clone() for n, t in xs[0].items()}
    dr, dh = (torch.randn(700, 4, 64, device="cuda").bfloat16() for _ in range(2))

    def go(x, out, ws):
        args = [x[n] for n in NAMES]
        qstate_norm(c, *args, out[0], out[1])
        qstate_norm_backward(c, *args, True, dr, dh, *out[2:], workspace=ws)

    def new():
        return ([torch.empty_like(dr) for _ in range(5)]
                + [torch.empty(64, device="cuda") for _ in range(3)])

    out, ws = new(), torch.empty(qstate_norm_workspace(c), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        go(x, out, ws)
    for i in (1, 2, 0, 1):
        for n in NAMES:
            x[n].copy_(xs[i][n])
        graph.replay()
        torch.cuda.synchronize()
        eager = new()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            go(xs[i], eager, torch.empty_like(ws))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))


def test_refusals():
    from bit_recurrent_state_amd import block_norm
    x = make(4, 2, 64, torch.float32, True, True, True, False, True)
    for change in (dict(gate=x["gate"].bfloat16()), dict(gate=x["gate"][:2]), dict(weight=x["weight"][:5]),
                   dict(weight=x["weight"].double()), dict(scale=x["scale"][None]),
                   dict(residual=x["residual"].cpu()), dict(x=x["x"].double()), dict(act=3),
                   dict(weight=torch.ones(3, 64, device="cuda"))):
        y = {**x, **change}
        act = y.pop("act", 0)
        with pytest.raises((ValueError, TypeError)):
            run(y, act=act)
    from bit_recurrent_state_amd._lib import QStateError
    with pytest.raises(QStateError):
        block_norm(torch.zeros(2, 64, device="cuda"), eps=0.0)


def test_many_rows_before_the_last_dimension():
    """[1, rows, width] with more rows than a token may have, also as part of wider rows."""
    x = make(70000, 0, 16, torch.float32, True, False, False, False, False)
    want = run(x)[0]
    wide = torch.cat([x["x"], x["gate"]], 1)[None]
    for a, z in ((x["x"][None], x["gate"][None]), (wide[..., :16], wide[..., 16:])):
        got = run({**x, "x": a, "gate": z})[0]
        assert got.shape == a.shape and torch.equal(got[0], want)


def test_rows_beyond_32_bits():
    """Rows behind 2^31 elements: the same bits as alone (about 35 GB)."""
    from bit_recurrent_state_amd import NormConfig, qstate_norm, qstate_norm_backward
    n, width = 70, 2048
    before = (1 << 31) // width
    x = make(n, 0, width, torch.bfloat16, True, True, True, False, True)
    want = run(x)
    dr, dh = (torch.randn(n, width, device="cuda").bfloat16() for _ in range(2))
    small = NormConfig(n, 1, width, torch.bfloat16)
    big = NormConfig(before + n, 1, width, torch.bfloat16)
    vectors = [x[k] for k in ("weight", "scale", "next_weight")]

    def go(c, xx, gate, res, dr, dh):
        view = lambda t: t.view(c.tokens, 1, width)
        r, h, dx, dz, dy = (torch.empty_like(view(xx)) for _ in range(5))
        a = (view(xx), vectors[0], view(gate), view(res), vectors[1], vectors[2])
        qstate_norm(c, *a, r, h)
        qstate_norm_backward(c, *a, True, view(dr), view(dh), dx, dz, dy)
        return [t.view(-1, width) for t in (r, h, dx, dz, dy)]

    def behind(t):
        b = torch.zeros(before + n, width, dtype=t.dtype, device="cuda")
        b[before:] = t
        return b

    alone = go(small, x["x"], x["gate"], x["residual"], dr, dh)
    assert torch.equal(alone[0], want[0]) and torch.equal(alone[1], want[1])
    got = go(big, *(behind(t) for t in (x["x"], x["gate"], x["residual"], dr, dh)))
    for a, b in zip(got, alone):
        assert torch.equal(a[before:], b)
    del got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", TYPES)
def test_silu_over_the_types_range(dtype):
    """Gates from the type's lowest to its largest value, forward and backward, element by element:
    far below zero SiLU and its slope are zero, far above the gate itself and one; at minus infinity
    the limit.  Relative to each element: half a step of the type and 32 roundings, as for a row."""
    dt = TYPES[dtype]
    end = torch.finfo(dt).max
    values = [-end, -end / 4, -1e4, -200.0, -100.0, -88.0, -80.0, 0.0, 80.0, 90.0, 200.0, 1e4, end / 4, end]
    x = make(len(values), 0, 64, dt, True, False, False, False, False)
    x["gate"] = torch.tensor(values).to(dt).cuda()[:, None].repeat(1, 64)
    x["x"] = x["x"].abs().clamp(0.25, 0.5)  # products with the largest gates stay in the type's range
    x["weight"].fill_(0.5)
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items() if t is not None}
    (out,) = run({**x, **leaves})
    l64 = {n: t.double().requires_grad_(True) for n, t in x.items() if t is not None}
    (want,) = norm64(*(l64.get(n) for n in NAMES), 1e-6, 0)
    # seeds that keep the gradients of the largest gates in range
    d = torch.where(x["gate"].abs() > 100, torch.finfo(dt).tiny * 16, 1.0).to(dt)
    got = torch.autograd.grad(out, [leaves["x"], leaves["gate"]], d)
    exact = torch.autograd.grad(want, [l64["x"], l64["gate"]], d.double())
    step = torch.finfo(dt).eps / 2
    for a, b in zip((out, got[1]), (want, exact[1])):
        # results below the type's normal numbers are rounded to its smallest step
        bound = (step + BASE) * b.abs() + torch.finfo(dt).tiny * (step * 2 + 2.0 ** -20) + 1e-34
        assert ((a.double() - b).abs() <= bound).all(), (a[:, 0], b[:, 0])
    # dx is a difference of terms; zero where the gate is far below zero
    low = x["gate"][:, 0].float() < -99
    assert got[0][low].abs().max() <= 1e-34
    z = {**x, "gate": torch.full_like(x["gate"], -float("inf"))}
    leaves = {n: t.clone().requires_grad_(True) for n, t in z.items() if t is not None}
    (out,) = run({**z, **leaves})
    grads = torch.autograd.grad(out, [leaves["x"], leaves["gate"]], torch.ones_like(out))
    for t in (out, *grads):
        assert t.abs().max() <= 1e-34


def test_rows_of_zeros_with_a_tiny_eps():
    """eps may be any positive number: a row of zeros has finite gradients where the formula's are."""
    x = make(6, 0, 128, torch.float32, False, True, False, False, True)
    x["x"][1] = 0
    x["residual"][1] = 0
    for eps in (1e-6, 1e-20, 1e-30):
        leaves = {n: t.clone().requires_grad_(True) for n, t in x.items() if t is not None}
        out = run({**x, **leaves}, eps=eps)
        l64 = {n: t.double().requires_grad_(True) for n, t in x.items() if t is not None}
        want = norm64(*(l64.get(n) for n in NAMES), eps, 0)
        seeds = [torch.full_like(t, 1e-3) for t in out]
        got = torch.autograd.grad(out, [leaves["residual"]], seeds)[0]
        exact = torch.autograd.grad(want, [l64["residual"]], [s.double() for s in seeds])[0]
        for i in range(6):
            assert rel(got[i], exact[i]) <= tol(torch.float32), (eps, i)


def test_forward_mode_and_tracing_are_refused():
    """Neither has a rule here: an error, and not a result without a tangent or an empty trace."""
    from torch.autograd import forward_ad
    from torch.fx.experimental.proxy_tensor import make_fx

    from bit_recurrent_state_amd import block_norm, scan
    from scan_reference import GDN, inputs
    x = torch.randn(3, 64, device="cuda")
    s = inputs(GDN, 1, [12], 1, 1, 64, 8, torch.float32, "cuda")

    def go(x, v):
        o, _ = scan(s["q"], s["k"], v, s["log_alpha"], s["beta"], mixer=GDN, offsets=s["offsets"])
        return block_norm(x), o

    want = go(x, s["v"])
    with forward_ad.dual_level():
        again = go(x, s["v"])  # no tangents: as ever
        assert all(torch.equal(a, b) for a, b in zip(want, again))
        with pytest.raises(NotImplementedError):
            block_norm(forward_ad.make_dual(x, torch.ones_like(x)))
        with pytest.raises(NotImplementedError):
            go(x, forward_ad.make_dual(s["v"], torch.ones_like(s["v"])))
    for f, a in ((lambda x: block_norm(x), x), (lambda v: go(x, v)[1], s["v"])):
        with pytest.raises(RuntimeError, match="trac"):
            make_fx(f)(a)
        with pytest.raises(RuntimeError, match="trac"):
            torch.jit.trace(f, a)
    assert all(torch.equal(a, b) for a, b in zip(want, go(x, s["v"])))
