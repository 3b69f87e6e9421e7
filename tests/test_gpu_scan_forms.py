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
