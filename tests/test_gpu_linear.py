"""Products with 4-bit weights against 64 bits (GPU)."""

import pytest
import torch

from scan_reference import rel

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def close(y, x, codes, scales, bias=None):
    """Products with whole numbers are exact (FP32 inputs: to 2^-24 of each).  A sum goes through at most
    24 matrix instructions in a group (4 of 32 columns times 6 pairs of terms), an addition for each
    group of a wave's tiles (an eighth of all), 8 of the waves' sums, and 4 more of scale, split and
    bias.  Each rounds by at most 2^-24 of a partial sum, which is at most the sum of the terms'
    magnitudes; y is then rounded once, by at most half a step."""
    x, W = x.double(), values(codes, scales)
    K, G = W.shape[1], W.shape[1] // scales.shape[1]
    want, size = torch.matmul(x, W.T), torch.matmul(x.abs(), W.abs().T)
    if bias is not None:
        want, size = want + bias.double(), size + bias.double().abs()
    n = 24 + -(-K // 1024) * (128 // G) + 8 + 4
    half = 0.0 if y.dtype == torch.float32 else torch.finfo(y.dtype).eps / 2
    # a 16-bit result among the subnormal numbers is rounded by half their step
    least = 0.0 if y.dtype == torch.float32 else torch.finfo(y.dtype).smallest_normal * half
    off = (y.double() - want).abs()
    return bool((off <= half * want.abs() + (1 + half) * n * 2.0 ** -24 * size + least).all())


def weights(outputs, inputs, group, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-7, 8, (outputs, inputs), generator=g, dtype=torch.int8).cuda()
    scales = (0.5 + torch.rand(outputs, inputs // group, generator=g)).cuda() / inputs ** 0.5
    return codes, scales


def values(codes, scales):
    return (codes.double().unflatten(-1, (scales.shape[1], -1)) * scales.double().unsqueeze(-1)).flatten(-2)


def check(rows, inputs, outputs, group, dtype, bias=False):
    from bit_recurrent_state_amd import Weight4, linear4
    codes, scales = weights(outputs, inputs, group)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(rows, inputs, generator=g).to(dtype).cuda()
    b = torch.randn(outputs, generator=g).cuda() if bias else None
    y = linear4(x, Weight4.from_codes(codes, scales), b)
    assert y.shape == (rows, outputs) and y.dtype == dtype
    assert close(y, x, codes, scales, b)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,tiles,outputs", [(1, 1, 1), (1, 5, 16), (2, 3, 17), (15, 32, 100),
                                                (16, 9, 1000), (17, 2, 64), (32, 1, 33), (33, 4, 50),
                                                (64, 7, 31), (65, 3, 40), (200, 2, 129)])
def test_sizes(dtype, group, rows, tiles, outputs):
    check(rows, group * tiles, outputs, group, TYPES[dtype], bias=outputs % 2 == 1)


@pytest.mark.parametrize("dtype", TYPES)
def test_model_sizes(dtype):
    check(1, 4096, 4096, 64, TYPES[dtype])
    check(16, 4096, 6144, 128, TYPES[dtype])
    check(61, 2080, 4100, 32, TYPES[dtype], True)


def test_single_codes():
    """Every place of a tile and every code: unit rows of x pick out single weights, exactly."""
    from bit_recurrent_state_amd import Weight4, linear4
    codes, scales = weights(37, 256, 32, 3)
    w = Weight4.from_codes(codes, scales)
    for dtype in TYPES.values():
        y = linear4(torch.eye(256, dtype=dtype, device="cuda"), w)
        assert torch.equal(y.t(), (codes.float() * scales.repeat_interleave(32, 1)).to(dtype))


def test_nibbles():
    from bit_recurrent_state_amd import Weight4
    codes, scales = weights(20, 192, 64)
    u = codes.view(torch.uint8)
    w = Weight4.from_nibbles((u[:, 0::2] & 15) | (u[:, 1::2] << 4), scales)
    v = Weight4.from_codes(codes, scales)
    assert torch.equal(w.packed, v.packed) and torch.equal(w.scales, v.scales)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize(dtype, group):
    """Each weight within half a step of its group's largest / 7; a group of zeros stays zero."""
    from bit_recurrent_state_amd import Weight4, linear4
    dt = TYPES[dtype]
    W = torch.randn(50, 384, generator=torch.Generator().manual_seed(4)).cuda()
    W[7, :group] = 0.0
    W[8] *= 1e-6
    W = W.to(dt)
    w = Weight4.quantize(W, group)
    got = linear4(torch.eye(384, device="cuda"), w).t().double()
    big = W.double().unflatten(-1, (-1, group)).abs().amax(-1, keepdim=True).expand(-1, -1, group).flatten(-2)
    assert bool(((got - W.double()).abs() <= big / 7 * (0.5 + 2.0 ** -20)).all())
    assert not got[7, :group].any()
    again = Weight4.quantize(got.float(), group)  # values on the grid stay where they are
    assert rel(linear4(torch.eye(384, device="cuda"), again).t(), got) <= 2.0 ** -22


def test_rows_do_not_mix():
    """A NaN or an infinity in a row of x spoils that row, and each row gives what it gives alone."""
    from bit_recurrent_state_amd import Weight4, linear4
    codes, scales = weights(70, 512, 64)
    w = Weight4.from_codes(codes, scales)
    for dtype in TYPES.values():
        x = torch.randn(20, 512, device="cuda").to(dtype)
        want = linear4(x, w)
        x[3, 9] = float("nan")
        x[17, 0] = float("inf")
        y = linear4(x, w)
        keep = [i for i in range(20) if i not in (3, 17)]
        assert torch.equal(y[keep], want[keep]) and bool(torch.isnan(y[3]).all())
        assert not bool(torch.isfinite(y[17][codes[:, 0] != 0]).any())
        assert torch.equal(linear4(x[5:6], w), want[5:6])


def test_strides_and_shapes():
    from bit_recurrent_state_amd import LinearConfig, Weight4, linear4, qstate_linear
    codes, scales = weights(40, 128, 64)
    w = Weight4.from_codes(codes, scales)
    x = torch.randn(6, 128, device="cuda").bfloat16()
    want = linear4(x, w)
    for pad in (1, 8):
        wide = torch.cat([x[:, :pad], x, x[:, :pad]], 1)
        assert torch.equal(linear4(wide[:, pad:pad + 128], w), want)
    assert torch.equal(linear4(x.view(2, 3, 128), w), want.view(2, 3, 40))
    assert torch.equal(linear4(x.t().contiguous().t(), w), want)
    assert torch.equal(linear4(x[0], w), want[0])
    assert linear4(x[:0], w).shape == (0, 40)
    wide = torch.cat([x, x], 1)
    y = torch.empty_like(want)
    qstate_linear(LinearConfig(128, 40, 64, torch.bfloat16, 6, 256), wide[:, 128:], w.packed, w.scales, None, y)
    assert torch.equal(y, want)


def test_streams_and_graphs():
    from bit_recurrent_state_amd import LinearConfig, Weight4, linear4, qstate_linear
    codes, scales = weights(300, 1024, 128)
    w = Weight4.from_codes(codes, scales)
    x = torch.randn(5, 1024, device="cuda")
    want = linear4(x, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y = torch.empty_like(want)
    qstate_linear(LinearConfig(1024, 300, 128, rows=5), x, w.packed, w.scales, None, y, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = linear4(x, w)
    for i in range(3):
        x.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, linear4(x, w))


def _layer():
    from bit_recurrent_state_amd import GDN, Config, QState, ReadoutNorm, Weight4
    from draft_reference import inputs
    x, S = inputs(GDN, 3, 5, "tree", 4, 2, 64, 32, torch.bfloat16, "cuda")
    st = QState(Config(3, 4, 64, 32, 32, GDN, head_bits=[8, 4, 4, 4]))
    st.load_fp32(S)
    W = torch.randn(96, 128, device="cuda") / 11
    g = torch.randn(3, 5, 4, 32, device="cuda").bfloat16()
    return st, x, S, Weight4.quantize(W, 64), ReadoutNorm(gate=g, center=True)


def test_a_layer_of_drafted_tokens():
    """Readout, group norm with its gate and output projection in one call give what the operators give
    one by one; the accepted path and the next token after it."""
    from bit_recurrent_state_amd import ReadoutNorm, group_norm, linear4
    st, x, S, w, norm = _layer()
    args = (x["q"], x["k"], x["v"], x["log_alpha"], x["beta"])
    y, draft = st.verify(*args, parents=x["parents"], norm=norm, project=w)
    o, _ = st.verify(*args, parents=x["parents"])
    by_hand = group_norm(o.flatten(-2), 4, gate=norm.gate.flatten(-2), eps=norm.eps)
    assert y.shape == (3, 5, 96) and torch.equal(y, linear4(by_hand, w))
    st.accept(draft, torch.tensor([4, 1, 2], dtype=torch.int32, device="cuda"))
    codes, scales, counter = st.codes.clone(), st.scales.clone(), st.step_counter
    f32 = torch.float32
    one = [torch.randn(3, 4, d, device="cuda") for d in (64, 64, 32)]
    gates = torch.rand(3, 4, device="cuda"), torch.rand(3, 4, device="cuda")
    a, b = torch.empty(3, 4, 32, device="cuda"), torch.empty(3, 4, 32, device="cuda")
    gate = ReadoutNorm(gate=norm.gate[:, 0].to(f32).contiguous())
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = st.step(*one, *gates, a, norm=gate, project=w, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    st.codes.copy_(codes)
    st.scales.copy_(scales)
    st.step_counter = counter
    st.step(*one, *gates, b, norm=gate)
    assert torch.equal(a, b) and torch.equal(got, linear4(b.view(3, 128), w))
    st.load_fp32(S)
    p = st.prefill(*args, norm=norm, project=w)
    st.load_fp32(S)
    assert torch.equal(p, linear4(st.prefill(*args, norm=norm).flatten(-2), w))


def test_projections_that_do_not_fit_leave_the_state():
    from bit_recurrent_state_amd import Weight4
    st, x, S, w, _ = _layer()
    codes, counter = st.codes.clone(), st.step_counter
    args = (x["q"], x["k"], x["v"], x["log_alpha"], x["beta"])
    other = Weight4.quantize(torch.randn(8, 64, device="cuda"))
    one = [t[:, 0].float().repeat_interleave(2, 1).contiguous() for t in (x["q"], x["k"])]
    one += [x["v"][:, 0].float().contiguous(), x["log_alpha"][:, 0].contiguous(), x["beta"][:, 0].contiguous()]
    for bad, err in ((other, ValueError), (torch.zeros(96, 128, device="cuda"), TypeError)):
        with pytest.raises(err):
            st.verify(*args, project=bad)
        with pytest.raises(err):
            st.prefill(*args, project=bad)
        with pytest.raises(err):
            st.step(*one, torch.empty(3, 4, 32, device="cuda"), project=bad)
    with pytest.raises(ValueError):
        st.step(*one, project=w)
    assert torch.equal(st.codes, codes) and st.step_counter == counter


def test_projections_in_forward_mode_leave_the_state():
    """Inside forward-mode differentiation and under a trace linear4 is refused: before the state changes."""
    from torch.autograd import forward_ad as fwd

    from bit_recurrent_state_amd import Config, QState, Weight4
    st = QState(Config(2, 2, 64, 16, mixer=1, fp32_state=True))
    st.load_fp32(torch.randn(2, 2, 16, 64, device="cuda"))
    before, step = st.codes.clone(), st.step_counter
    w = Weight4.quantize(torch.randn(20, 32, device="cuda"), 32)
    q, k, v, o = (torch.randn(2, 2, d, device="cuda") for d in (64, 64, 16, 16))
    a = torch.full_like(q, 0.9)
    kept = o.clone()

    def calls(q, o):
        yield lambda: st.step(q, k, v, a, None, o, project=w)
        yield lambda: st.prefill(q[:, None], k[:, None], v[:, None], a.log()[:, None], project=w)
        yield lambda: st.verify(q[:, None], k[:, None], v[:, None], a.log()[:, None], project=w)

    with fwd.dual_level():
        for go in calls(q, o):
            with pytest.raises(RuntimeError):
                go()
    for i in range(3):
        with pytest.raises(RuntimeError):
            torch.jit.trace(lambda q: list(calls(q, o))[i]() or q, (q,), check_trace=False)
    assert torch.equal(st.codes, before) and st.step_counter == step and torch.equal(o, kept)
    st.step(q, k, v, a, None, o, project=w)
    assert st.step_counter == step + 1



def test_refusals():
    from bit_recurrent_state_amd import Weight4, linear4
    from bit_recurrent_state_amd._lib import QStateError
    codes, scales = weights(16, 128, 64)
    w = Weight4.from_codes(codes, scales)
    x = torch.randn(2, 128, device="cuda")
    bad = codes.clone()
    bad[3, 3] = -8
    for a, b in ((bad, scales), (codes.int(), scales), (codes, scales.half()), (codes, scales[:3]),
                 (codes, scales[:, :0]), (codes[:0], scales[:0])):
        with pytest.raises(ValueError):
            Weight4.from_codes(a, b)
    with pytest.raises(QStateError):
        Weight4.from_codes(codes, scales.repeat_interleave(4, 1))  # groups of 16
    with pytest.raises(QStateError):
        Weight4.quantize(torch.randn(4, 100, device="cuda"), 64)
    with pytest.raises(ValueError):
        Weight4.quantize(torch.randn(4, 128, device="cuda").double())
    for kw in (dict(x=x[:, :64]), dict(x=x.double()), dict(bias=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            linear4(**{"x": x, "weight": w, **kw})
    with pytest.raises(TypeError):
        linear4(x.cpu(), w)
    with pytest.raises(RuntimeError):
        linear4(x.clone().requires_grad_(True), w)
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda t: linear4(t, w), (x,), check_trace=False)


def test_more_rows_than_a_call_takes():
    """Rows of a long prompt: the last ones as by themselves."""
    from bit_recurrent_state_amd import Weight4, linear4
    g = torch.Generator().manual_seed(5)
    w = Weight4.quantize(torch.randn(17, 64, generator=g).cuda(), 32)
    x = torch.randn(1, 64, generator=g).bfloat16().cuda().repeat((1 << 19) + 21, 1)
    x[-30:] = torch.randn(30, 64, generator=g).bfloat16().cuda()
    y = linear4(x, w)
    assert torch.equal(y[-30:], linear4(x[-30:], w))
    assert torch.equal(y[:-30], linear4(x[:1], w).expand(y.shape[0] - 30, -1))
