"""The group norm and its gradients against 64 bits (GPU)."""

import itertools

import pytest
import torch

from scan_reference import rel

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MODES = ("plain", "gate", "gate_first", "activate")

# FP32 between inputs and outputs: a row's two sums (mean, squares) err by at most 2 + log2 of the
# terms a thread and a tree add roundings each, the elementwise parts by some sixteen more: 48 * 2^-24
# of the norm.  Gradients go through two such sums more.  Weights' gradients are sums over rows of such
# terms of either sign, whose norm is about sqrt(rows) of the terms' against sums of up to 128 rows a
# team in FP32: twice that.
BASE = 48 * 2.0 ** -24


def tol(dtype, times=1):
    return times * BASE + (0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2)


def norm64(x, groups, weight, bias, gate, mode, center, eps, act):
    def activate(z):
        return z * torch.sigmoid(z) if act == 0 else torch.sigmoid(z)

    u = x * activate(gate) if mode == "gate_first" else x
    u = u.unflatten(-1, (groups, -1))
    if center:
        u = u - u.mean(-1, keepdim=True)
    n = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        n = n * weight.view(-1, n.shape[-1])
    if bias is not None:
        n = n + bias.view(-1, n.shape[-1])
    n = n.flatten(-2)
    return n * activate(gate) if mode == "gate" else activate(n) if mode == "activate" else n


def make(rows, groups, width, dtype, mode, shared=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    C = groups * width

    def normal(*s):
        return torch.randn(s, generator=g)

    x = {"x": (normal(rows, C) + 0.5).to(dtype), "weight": 1 + 0.1 * normal(width if shared else C),
         "bias": 0.1 * normal(width if shared else C),
         "gate": (2 * normal(rows, C)).to(dtype) if mode in ("gate", "gate_first") else None}
    return {n: None if t is None else t.cuda() for n, t in x.items()}


def call(x, groups, mode, center=True, eps=1e-5, act=0):
    from bit_recurrent_state_amd import group_norm
    return group_norm(x["x"], groups, weight=x["weight"], bias=x["bias"], gate=x["gate"],
                      gate_first=mode == "gate_first", activate=mode == "activate", center=center,
                      eps=eps, act=act)


def check(x, groups, mode, center=True, eps=1e-5, act=0):
    dt = x["x"].dtype
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items() if t is not None}
    y = call({**x, **leaves}, groups, mode, center, eps, act)
    l64 = {n: t.double().requires_grad_(True) for n, t in x.items() if t is not None}
    want = norm64(l64["x"], groups, *(l64.get(n) for n in ("weight", "bias", "gate")), mode, center,
                  eps, act)
    assert y.dtype == dt and y.shape == x["x"].shape
    assert rel(y, want) <= tol(dt)
    dy = torch.randn(y.shape, generator=torch.Generator().manual_seed(9)).to(dt).cuda()
    got = torch.autograd.grad(y, list(leaves.values()), dy)
    exact = torch.autograd.grad(want, list(l64.values()), dy.double())
    for n, a, b in zip(leaves, got, exact):
        assert a.dtype == x[n].dtype and a.shape == x[n].shape
        assert rel(a, b) <= tol(a.dtype, 4 if n in ("weight", "bias") else 2), n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rows,groups,width", [(1, 1, 8), (37, 3, 64), (5, 1, 513), (3, 2, 100), (300, 4, 128),
                                               (9, 2, 1024), (4, 1, 4096), (3, 3, 1030), (2, 1, 9999),
                                               (2, 1, 16384), (11, 70, 12)])
def test_widths(dtype, mode, rows, groups, width):
    check(make(rows, groups, width, TYPES[dtype], mode), groups, mode)


@pytest.mark.parametrize("mode,center,shared,act", itertools.product(MODES, [0, 1], [0, 1], [0, 1]))
def test_forms(mode, center, shared, act):
    for dtype, groups, width in ((torch.bfloat16, 3, 64), (torch.float32, 2, 700), (torch.float32, 5, 7)):
        check(make(19, groups, width, dtype, mode, shared), groups, mode, center, act=act)


@pytest.mark.parametrize("without", ["weight", "bias", "both"])
def test_without_weight_or_bias(without):
    for mode in MODES:
        x = make(40, 2, 128, torch.float32, mode)
        for n in ("weight", "bias"):
            if without in (n, "both"):
                x[n] = None
        check(x, 2, mode)


def test_many_rows():
    """More rows than teams: every team sums several rows into the weights' gradients."""
    check(make(9000, 4, 64, torch.bfloat16, "gate"), 4, "gate")
    check(make(3000, 7, 64, torch.float32, "activate", True), 7, "activate")
    check(make(40000, 1, 16, torch.float32, "plain"), 1, "plain")
    check(make(1500, 2, 1030, torch.float16, "gate_first"), 2, "gate_first", False)


def test_one_channel():
    """A centered group of one channel is its own mean: nothing but the bias is left."""
    x = make(9, 4, 1, torch.float32, "plain")
    assert torch.equal(call(x, 4, "plain"), x["bias"].expand(9, 4))


def test_large_mean():
    """The variance is taken from centered values: a mean 4096 times the deviation costs no more than
    the inputs' own rounding of the mean, 2^-24 * 4096 of a deviation, over and over."""
    x = make(50, 2, 256, torch.float32, "plain")
    x["x"] = (x["x"] + 4096.0)
    want = norm64(x["x"].double(), 2, x["weight"].double(), x["bias"].double(), None, "plain", True, 1e-5, 0)
    # mean: (2 + log2 256) roundings of sums of 4096; differences are exact to that
    assert rel(call(x, 2, "plain"), want) <= 4096 * 10 * 2.0 ** -24 + BASE


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("mode", ["gate", "activate"])
def test_weights_gradients_hold_to_fp32(dtype, act, mode):
    """dweight and dbias are FP32 whatever x's type is, also where the activation is small.

    One token, so that a value is one term, and x of 1 and -1, so that normalised values are off by the
    root's 3 roundings.  sigmoid: the exponential's ulp (2 roundings), what its argument is off by (4 at
    -86), its product, the sum, the reciprocal's ulp (2): 10.  silu's slope: 1 - s off by 4, which adding 1
    makes 6 where |z| is 4 or more, and two products; the term's product: 22 * 2^-24 in all."""
    g = torch.Generator().manual_seed(4)
    C = 256
    x = torch.where(torch.rand(1, C, generator=g) < 0.5, -1.0, 1.0)
    z = torch.empty(1, C).uniform_(-86.0, -4.0, generator=g)
    dt = TYPES[dtype]
    leaves = {"x": x.to(dt), "weight": torch.ones(C) if mode == "gate" else torch.zeros(C),
              "bias": torch.zeros(C) if mode == "gate" else z[0].clone(),
              "gate": z.to(dt) if mode == "gate" else None}
    leaves = {n: None if t is None else t.cuda() for n, t in leaves.items()}
    own = {n: None if t is None else t.clone().requires_grad_(True) for n, t in leaves.items()}
    l64 = {n: None if t is None else t.double().requires_grad_(True) for n, t in leaves.items()}
    y = call(own, 2, mode, False, 1e-12, act)
    want = norm64(l64["x"], 2, l64["weight"], l64["bias"], l64["gate"], mode, False, 1e-12, act)
    sums = ("weight", "bias")
    got = torch.autograd.grad(y, [own[n] for n in sums], torch.ones_like(y))
    exact = torch.autograd.grad(want, [l64[n] for n in sums], torch.ones_like(want))
    for n, a, b in zip(sums, got, exact):
        off = ((a.double() - b) / b).abs()
        assert bool((off <= 22 * 2.0 ** -24).all()), (n, float(off.max()))


def test_equal_values_and_zeros():
    """Rows without variance: the bias alone, finite gradients."""
    x = make(6, 2, 64, torch.float32, "plain")
    x["x"][:3] = 0.0
    x["x"][3:] = 2.0
    leaf = x["x"].clone().requires_grad_(True)
    y = call({**x, "x": leaf}, 2, "plain")
    assert torch.equal(y.detach(), x["bias"].expand(6, 128))
    d, = torch.autograd.grad(y, leaf, torch.randn_like(y))
    assert bool(torch.isfinite(d).all())


@pytest.mark.parametrize("mode", ["gate", "gate_first"])
def test_masked_gates(mode):
    """Gates at the type's lowest value and at minus infinity let nothing through: silu holds its
    argument at -87 there, 87 e^-87 = 1.5e-36, which a normalised value of at most sqrt(64) and a
    weight below 2 (in front: a value below 8, and 1 / sqrt(eps) = 317) multiply."""
    least = 1.5e-36 * (16.0 if mode == "gate" else 16.0 * 317.0)
    for dtype in TYPES.values():
        x = make(8, 2, 64, dtype, mode)
        x["bias"] = None
        x["gate"][2] = torch.finfo(dtype).min
        x["gate"][5, :64] = -float("inf")
        y = call(x, 2, mode)
        assert bool(torch.isfinite(y).all())
        assert float(y[2].abs().max()) <= least and float(y[5, :64].abs().max()) <= least
        leaf = x["gate"].clone().requires_grad_(True)
        d, = torch.autograd.grad(call({**x, "gate": leaf}, 2, mode), leaf, torch.ones_like(y))
        assert bool(torch.isfinite(d).all())


def test_nan_stays_in_its_group():
    x = make(10, 4, 32, torch.bfloat16, "gate")
    want = call(x, 4, "gate")
    x["x"][3, 40] = float("nan")
    x["x"][7, 0] = float("inf")
    y = call(x, 4, "gate")
    assert bool(torch.isnan(y[3, 32:64]).all()) and bool(torch.isnan(y[7, :32]).any())
    y[3, 32:64], y[7, :32] = want[3, 32:64], want[7, :32]
    assert torch.equal(y, want)


def test_strides_views_and_places():
    from bit_recurrent_state_amd import GATE, GroupNormConfig, qstate_group_norm
    x = make(50, 4, 64, torch.bfloat16, "gate")
    want = call(x, 4, "gate")
    wide = torch.cat([x["x"], x["gate"], x["x"][:, :3]], 1)
    for off in (0, 3):
        w = torch.cat([wide[:, :off], wide], 1)
        got = call({**x, "x": w[:, off:off + 256], "gate": w[:, off + 256:off + 512]}, 4, "gate")
        assert rel(got, want) <= tol(torch.bfloat16)
    t = {n: x[n].t().contiguous().t() for n in ("x", "gate")}
    assert torch.equal(call({**x, **t}, 4, "gate"), want)
    three = {n: x[n].view(5, 10, 256) for n in ("x", "gate")}
    assert torch.equal(call({**x, **three}, 4, "gate").view(50, 256), want)
    c = GroupNormConfig(50, 4, 64, torch.bfloat16, mode=GATE)
    for place in ("x", "gate"):
        y = {n: x[n].clone() for n in ("x", "gate")}
        qstate_group_norm(c, y["x"], x["weight"], x["bias"], y["gate"], y[place])
        assert torch.equal(y[place], want)


def test_no_rows():
    x = make(0, 4, 64, torch.float32, "gate")
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items()}
    y = call(leaves, 4, "gate")
    assert y.shape == (0, 256)
    g = torch.autograd.grad(y, list(leaves.values()), y.detach())
    assert all(t.shape == l.shape and not t.any() for t, l in zip(g, leaves.values()))


def test_gradients_against_differences():
    x = {n: t.double() if t is not None else None for n, t in make(2, 2, 16, torch.float32, "gate_first").items()}
    leaves = {n: x[n].float().requires_grad_(True) for n in x}
    dy = torch.randn(2, 32, generator=torch.Generator().manual_seed(1)).cuda()
    got = dict(zip(leaves, torch.autograd.grad(call(leaves, 2, "gate_first"), list(leaves.values()), dy)))

    def loss(v):
        return float((norm64(v["x"], 2, v["weight"], v["bias"], v["gate"], "gate_first", True, 1e-5, 0)
                      * dy.double()).sum())

    h = 1e-6
    for n in x:
        for at in (0, 5, 17):
            d = torch.zeros_like(x[n])
            d.view(-1)[at] = h
            slope = (loss({**x, n: x[n] + d}) - loss({**x, n: x[n] - d})) / (2 * h)
            # differences in 64 bits err by 1e-9 or so, the gradient by its tolerance of its norm
            assert abs(slope - float(got[n].view(-1)[at])) <= 1e-6 + 4 * BASE * float(got[n].norm())


def test_streams_and_graphs():
    """On another stream; a training step captured and replayed with new values in place."""
    from bit_recurrent_state_amd import GroupNormConfig, qstate_group_norm
    x = make(300, 4, 64, torch.float32, "activate")
    want = call(x, 4, "activate")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want)
    qstate_group_norm(GroupNormConfig(300, 4, 64, mode=3), x["x"], x["weight"], x["bias"], None, y,
                      stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    leaves = {n: t.clone().requires_grad_(True) for n, t in x.items() if t is not None}
    dy = torch.randn_like(want)

    def step():
        out = call({**leaves, "gate": None}, 4, "activate")
        return [out.detach()] + list(torch.autograd.grad(out, list(leaves.values()), dy))

    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        held = step()
    for i in range(3):
        with torch.no_grad():
            leaves["x"].copy_(x["x"] * (1.0 + i))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_capture_beside_an_eager_graph_is_refused(monkeypatch):
    """The check stands before any launch; no capture is made here."""
    x = make(30, 4, 64, torch.float32, "plain")
    leaf = x["x"].clone().requires_grad_(True)
    alive = call({**x, "x": leaf}, 4, "plain")
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        y = call({**x, "x": leaf}, 4, "plain")
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        with pytest.raises(RuntimeError, match="drop the results"):
            torch.autograd.grad(y.sum(), leaf, retain_graph=True)
        del alive
        torch.autograd.grad(y.sum(), leaf)
    torch.cuda.synchronize()


def test_readout_norm_forms():
    """The forms of the readout's norm on the decode path: step, prefill and verify."""
    from bit_recurrent_state_amd import GDN, Config, QState, ReadoutNorm
    B, H, dk, dv = 3, 2, 64, 32
    g = torch.Generator().manual_seed(2)

    def normal(*s):
        return torch.randn(s, generator=g).cuda()

    q, k, v = normal(B, 4, H, dk), normal(B, 4, H, dk) / 8, normal(B, 4, H, dv)
    la, beta, z = -0.1 * normal(B, 4, H).abs(), torch.sigmoid(normal(B, 4, H)), normal(B, 4, H, dv)
    each = 1 + 0.1 * normal(H, dv), 0.1 * normal(H, dv)
    shared = 1 + 0.1 * normal(dv), 0.1 * normal(dv)
    S = 0.3 * normal(B, H, dv, dk)
    for w, b, first, center in ((*each, False, True), (*shared, True, False), (shared[0], None, True, True),
                                (None, None, False, True)):
        st = QState(Config(B, H, dk, dv, mixer=GDN, fp32_state=True))

        def want(o, z):
            w2, b2 = (None if t is None else t.double().expand(H, dv).reshape(-1) for t in (w, b))
            y = norm64(o.double().flatten(-2), H, w2, b2, z.double().flatten(-2),
                       "gate_first" if first else "gate", center, 1e-6, 0)
            return y.view(o.shape)

        def norm(z):
            return ReadoutNorm(w, z.contiguous(), bias=b, gate_first=first, center=center)

        st.load_fp32(S)
        plain, _ = st.verify(q, k, v, la, beta)
        o, _ = st.verify(q, k, v, la, beta, norm=norm(z))
        assert rel(o, want(plain, z)) <= tol(torch.float32)
        st.load_fp32(S)
        plain = st.prefill(q, k, v, la, beta)
        st.load_fp32(S)
        assert rel(st.prefill(q, k, v, la, beta, norm=norm(z)), want(plain, z)) <= tol(torch.float32)
        one = [t[:, 0].contiguous() for t in (q, k, v, la.exp(), beta)]
        a, b1 = torch.empty(B, H, dv, device="cuda"), torch.empty(B, H, dv, device="cuda")
        st.load_fp32(S)
        st.step(*one, a)
        st.load_fp32(S)
        st.step(*one, b1, norm=norm(z[:, 0]))
        assert rel(b1, want(a, z[:, 0])) <= tol(torch.float32)


def test_refusals():
    from bit_recurrent_state_amd import ReadoutNorm, group_norm
    from bit_recurrent_state_amd._lib import QStateError
    x = make(5, 2, 64, torch.float32, "gate")
    X = x["x"]
    for kw in (dict(groups=3), dict(groups=0), dict(weight=x["weight"][:5]), dict(act=2),
               dict(weight=x["weight"].double()), dict(gate=x["gate"][:3]), dict(gate_first=True),
               dict(gate=x["gate"], activate=True), dict(gate=x["gate"].half()),
               dict(weight=x["weight"], bias=x["bias"][:64])):
        kw = {"groups": 2, **kw}
        with pytest.raises(ValueError):
            group_norm(X, **kw)
    with pytest.raises(ValueError):
        group_norm(X.double(), 2)
    with pytest.raises(TypeError):
        group_norm(X.cpu(), 2)
    for eps in (0.0, float("nan"), float("inf")):
        with pytest.raises(QStateError):
            group_norm(X, 2, eps=eps)
    with pytest.raises(ValueError):
        ReadoutNorm(gate_first=True).config((5, 2, 64), torch.float32, X.device)
    with pytest.raises(ValueError):
        ReadoutNorm(x["weight"].view(2, 64), bias=x["bias"][:64]).config((5, 2, 64), torch.float32, X.device)
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: group_norm(t, 2), (X,), check_trace=False)
    import torch.autograd.forward_ad as fwd
    with fwd.dual_level(), pytest.raises(RuntimeError):
        group_norm(fwd.make_dual(X, X), 2)
