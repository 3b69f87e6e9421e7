"""Forms of the scan that other tests do not reach, against the recurrence in 64 bits
(GPU): strided rows with gradients, wide column blocks, chunks that decay far in
every type and head size, and single elements instead of whole arrays' norms."""

import pytest
import torch

from scan_reference import GLA, KDA, MIXERS, inputs, rel, scan64, tolerance
from test_gpu_scan import NAMES, TYPES, call, check

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


def _zero_rows(T, H, d, dtype):
    return torch.zeros(T, H, d, dtype=dtype, device="cuda")


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dk", [64, 128, 256])
def test_outputs_small_by_cancellation(mixer, dtype, dk):
    """o as the difference of two numbers a thousand times its size: half a step of its own value,
    as far as FP32 sums go.

    From the state: nothing is written and nothing decays, o = q_a S_a + q_b S_b.  Three matrix
    instructions meet nonzero terms, each rounds the products' sum and the accumulator (6 roundings
    of 2^-24); the split leaves 2^-27 of S and q each: 8 * 2^-24 of the terms.  In 16 bits q's own
    terms (fp16: two) make six instructions: 14.
    Inside a chunk: o = A_0 W_0 + A_1 W_1, where A_0 sums two products, W is beta v rounded once:
    2 for W, 14 for A, 14 for the sum: 30 * 2^-24."""
    m, dt, H, dv, T = MIXERS[mixer], TYPES[dtype], 2, 64, 12
    g = torch.Generator().manual_seed(3)

    def one_to_two(*s):
        return (1 + torch.rand(s, generator=g)).cuda()

    near = 1 - 2.0 ** -9 * torch.rand(H, dv, generator=g).cuda()
    gate = (T, H, dk) if m in (GLA, KDA) else (T, H)
    x = {"q": _zero_rows(T, H, dk, dt), "k": _zero_rows(T, H, dk, dt),
         "v": _zero_rows(T, H, dv, dt), "log_alpha": torch.zeros(gate, device="cuda"),
         "beta": None if m == GLA else torch.full((T, H), 0.5, device="cuda"),
         "initial_state": torch.zeros(1, H, dv, dk, device="cuda"),
         "offsets": torch.tensor([0, T], device="cuda")}

    def outputs(x, terms, K):
        with torch.no_grad():
            o, _ = call(x, m)
        o64 = scan64(x, m, 1)[0]
        bound = torch.finfo(dt).eps / 2 * o64.abs() + K * EPS * terms
        assert ((o.double() - o64).abs() <= bound).all(), float(((o.double() - o64).abs() / bound).max())

    a, b = 5, dk - 3
    S = one_to_two(H, dv)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["initial_state"][0, :, :, a], y["initial_state"][0, :, :, b] = S, -S * near
    q = one_to_two(T, H).to(dt)
    y["q"][:, :, a], y["q"][:, :, b] = q, q
    outputs(y, 2 * (q.double()[:, :, None] * S.double()), 14)

    # tokens 0 and 1 write, into different channels; c adds low bits to A_0
    c = 17
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    q = one_to_two(T, H).to(dt)
    y["k"][0, :, a], y["k"][1, :, b], y["k"][0, :, c] = 1, 1, 2.0 ** -12
    y["q"][2:, :, a], y["q"][2:, :, b] = q[2:], q[2:]
    y["q"][2:, :, c] = one_to_two(T, H).to(dt)[2:]
    v = one_to_two(H, dv).to(dt)
    y["v"][0], y["v"][1] = v, -v
    if m != GLA:
        y["beta"][0] = one_to_two(H)
        y["beta"][1] = y["beta"][0] * (1 - 2.0 ** -10 * torch.rand(H, generator=g).cuda())
    terms = torch.zeros(T, H, dv, dtype=torch.float64, device="cuda")
    terms[2:] = 4 * 2 * q.double()[2:, :, None] * v.double()
    terms[:2] = 1e30  # the writing tokens read nothing of interest
    outputs(y, terms, 30)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dv", [32, 40])
@pytest.mark.parametrize("pad", [8, 4, 3])
def test_gradients_of_strided_rows(mixer, dtype, dv, pad):
    """q, k and v cut from one projection, with its gradient: rows on 16 bytes (8), on 8 or 16 (4),
    and on none (3); key heads shared and not."""
    m, dt, N, lens, H, dk = MIXERS[mixer], TYPES[dtype], 2, [70, 30], 4, 64
    for Hq in (4, 2):
        x = inputs(m, N, lens, H, Hq, dk, dv, dt, "cuda", seed=pad)
        T = sum(lens)
        sizes = [Hq * dk, Hq * dk, H * dv, pad]
        wide = torch.cat([x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1),
                          torch.zeros(T, pad, dtype=dt, device="cuda")], 1).requires_grad_(True)
        q, k, v = (t.unflatten(1, (h, d)) for t, h, d in zip(wide.split(sizes, 1), (Hq, Hq, H), (dk, dk, dv)))
        rest = {n: x[n].clone().requires_grad_(True) for n in ("log_alpha", "beta", "initial_state")
                if x[n] is not None}
        o, S = call({**x, **rest, "q": q, "k": k, "v": v}, m)
        g = torch.Generator().manual_seed(1)
        do, dS = torch.randn(o.shape, generator=g).to(dt).cuda(), torch.randn(S.shape, generator=g).cuda()
        got = torch.autograd.grad((o, S), [wide, *rest.values()], (do, dS))
        o64, S64, leaf = scan64(x, m, N, True)
        names = [n for n in NAMES if x[n] is not None]
        want = dict(zip(names, torch.autograd.grad((o64, S64), [leaf[n] for n in names],
                                                   (do.double(), dS.double()))))
        parts = dict(zip(("q", "k", "v"), (t.unflatten(1, (h, d)) for t, h, d in zip(
            got[0].split(sizes, 1), (Hq, Hq, H), (dk, dk, dv)))))
        parts.update(zip(rest, got[1:]))
        assert rel(o, o64) <= tolerance(dt, False) and rel(S, S64) <= tolerance(torch.float32, False)
        for n, t in parts.items():
            assert rel(t, want[n]) <= tolerance(t.dtype, True), n


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", TYPES)
def test_backward_with_row_strides_of_its_own(mixer, dtype):
    """qstate_scan_backward with another odd stride for each of q, k and v: the bits of packed rows
    in the same form (odd strides split every row), d_o and the gradients packed."""
    from bit_recurrent_state_amd import ScanConfig, qstate_scan_backward
    m, dt, H, Hq, dk, dv, lens = MIXERS[mixer], TYPES[dtype], 3, 1, 128, 33, [66, 9]
    T = sum(lens)
    x = inputs(m, 2, lens, H, Hq, dk, dv, dt, "cuda")
    g = torch.Generator().manual_seed(4)
    do, dS = torch.randn(T, H, dv, generator=g).to(dt).cuda(), torch.randn(2, H, dv, dk, generator=g).cuda()
    rows, strides = {}, {}
    for n, more in (("q", 3), ("k", 13), ("v", 1)):
        h, d = x[n].shape[1:]
        w = torch.zeros(T, h * d + more, dtype=dt, device="cuda")
        w[:, :h * d] = x[n].flatten(1)
        rows[n], strides[n] = w[:, :h * d].view(T, h, d), h * d + more
    c = ScanConfig(2, H, dk, dv, T, Hq, m, dt, strides["q"], strides["k"], strides["v"], H * dv + 5)
    out = {n: None if x[n] is None else torch.empty_like(x[n]) for n in NAMES}
    qstate_scan_backward(c, rows["q"], rows["k"], rows["v"], x["log_alpha"], x["beta"], x["offsets"],
                         x["initial_state"], do, dS, *(out[n] for n in NAMES))
    o64, S64, leaf = scan64(x, m, 2, True)
    names = [n for n in NAMES if x[n] is not None]
    want = torch.autograd.grad((o64, S64), [leaf[n] for n in names], (do.double(), dS.double()))
    for n, w in zip(names, want):
        assert rel(out[n], w) <= tolerance(out[n].dtype, True), n


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,N,dv", [(64, 2, 90), (128, 2, 90), (256, 2, 90), (64, 4, 121), (128, 4, 121),
                                     (256, 4, 121)])
def test_wide_column_blocks(mixer, dtype, dk, N, dv):
    """As many heads and columns as make the chains take 32 columns a workgroup (32 heads, N = 2:
    192 blocks of 32) and, forward up to dk = 128, 64 (N = 4: 512)."""
    m = MIXERS[mixer]
    lens = [70, 9, 0, 66][:N]
    check(inputs(m, N, lens, 32, 16, dk, dv, TYPES[dtype], "cuda"), m, N)


@pytest.mark.parametrize("mixer", ["gla", "kda"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,H,Hq", [(64, 64, 2, 2), (128, 40, 4, 2), (256, 64, 2, 1)])
def test_chunks_that_decay_far(mixer, dtype, dk, dv, H, Hq):
    """Gates per channel: every chunk far; one head's middle chunk far between ordinary ones; one
    channel of it; a state dropped inside a chunk."""
    m = MIXERS[mixer]
    lens = [150, 20]
    for which in range(4):
        x = inputs(m, 2, lens, H, Hq, dk, dv, TYPES[dtype], "cuda", seed=which)
        if which == 0:
            x["log_alpha"] *= 30.0
        elif which == 1:
            x["log_alpha"][64:128, 1] *= 30.0
        elif which == 2:
            x["log_alpha"][70:110, 0, dk - 1] = -2.0
        else:
            x["log_alpha"][100, 1] = -100.0
        check(x, m, 2)


@pytest.mark.parametrize("mixer", ["gla", "kda"])
@pytest.mark.parametrize("dk", [64, 128, 256])
@pytest.mark.parametrize("shape", ["even", "random", "early", "late"])
def test_elements_just_below_a_far_decay(mixer, dk, shape):
    """A chunk of 64 whose channels decay by e^-23.9, every factor e^(c_i - c_j) by itself: q and k
    hold one channel, v writes token j's value into column j, so that o[i, j] = q_i k_j e^(c_i - c_j)
    and the state's column is v_j k_j e^(c_end - c_j) (KDA: nearly so, with beta = 2^-20, against the
    64-bit recurrence).  Relative to each element, in units of 2^-24: sums of log decays held to 2^-25
    each (2), two exponentials to an ulp or two (2 * 4), the reciprocal (1), the splits of the operands
    and the products left out (3), six sums (6): 20; what KDA's state takes off is 64 * 2^-20 of that
    at most, so that its errors do not count, and rounds the sum: 24."""
    m, H, dv, T = MIXERS[mixer], 2, 64, 64
    g = torch.Generator().manual_seed(7)
    w = {"even": torch.ones(T), "random": torch.rand(T, generator=g),
         "early": (torch.arange(T) < 5).double() + 0.01, "late": (torch.arange(T) >= 59).double() + 0.01}[shape]
    w = w.double()[:, None, None] * (0.5 + torch.rand(T, H, dk, generator=g).double())
    la = (-23.9 * w / w.sum(0)).float().cuda()
    ch = 11
    q, k = (torch.zeros(T, H, dk, device="cuda") for _ in range(2))
    q[:, :, ch], k[:, :, ch] = 1 + torch.rand(T, H, generator=g).cuda(), 1.0
    x = {"q": q, "k": k, "v": torch.eye(T, device="cuda")[:, None].repeat(1, H, 1).contiguous(),
         "log_alpha": la, "beta": None if m == GLA else torch.full((T, H), 2.0 ** -20, device="cuda"),
         "initial_state": None, "offsets": torch.tensor([0, T], device="cuda")}
    with torch.no_grad():
        o, S = call(x, m)
    o64, S64, _ = scan64(x, m, 1)
    K = 20 if m == GLA else 24
    for a, b in ((o, o64), (S, S64)):
        err = ((a.double() - b).abs() / b.abs().clamp_min(1e-300))[b != 0]
        assert err.numel() and float(err.max()) <= K * EPS, float(err.max()) / EPS
        assert not a[b == 0].any()
