"""The recurrences over whole sequences and the block norm in 64 bits, token by
token and without any of the library's code, for the tests."""

import torch

GDN, GLA, SCALAR, KDA = 0, 1, 2, 3
MIXERS = {"gdn": GDN, "gla": GLA, "scalar": SCALAR, "kda": KDA}

# Errors are relative to the 2-norm of the reference.
# An FP32 result of the scan goes through at most three chained products forward
# (K S, T R, the state or the output) and five with the backward pass (U, X, dW,
# Y, dq); a product accumulates at most 24 matrix instructions (dk = 128: 4 of 32
# columns times 6 pairs of terms; dk = 256 twice that), each rounding to 2^-24.
FORWARD = 3 * 48 * 2.0 ** -24
BACKWARD = 5 * 48 * 2.0 ** -24


def tolerance(dtype, backward):
    """A 16-bit output is rounded once, by at most half a step of its value, so its norm is too;
    its two-term operands add 2^-16."""
    base = BACKWARD if backward else FORWARD
    return base if dtype == torch.float32 else torch.finfo(dtype).eps / 2 + 2.0 ** -16 + base


def inputs(mixer, N, lens, H, Hq, dk, dv, dtype, device, seed=0, gate=1.0, state=True, gap=0):
    """Packed sequences; `gap` rows of no sequence in front and behind."""
    g = torch.Generator().manual_seed(seed)
    total = sum(lens) + 2 * gap

    def normal(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    q, k = normal(total, Hq, dk), normal(total, Hq, dk)
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    v = normal(total, H, dv)
    beta = torch.sigmoid(normal(total, H))
    la = -torch.nn.functional.softplus(normal(*((total, H, dk) if mixer in (GLA, KDA)
                                                else (total, H))) - 3.0) * gate
    ends = torch.tensor([gap] + lens).cumsum(0)
    x = {"q": q.to(dtype), "k": k.to(dtype), "v": v.to(dtype), "log_alpha": la.float(),
         "beta": None if mixer == GLA else beta.float(),
         "initial_state": (0.3 * normal(N, H, dv, dk)).float() if state else None,
         "offsets": ends.to(torch.int64)}
    return {n: None if t is None else t.to(device) for n, t in x.items()}


def scan64(x, mixer, N, grad=False):
    """(o, final state, the leaves in 64 bits); leaves take gradients if `grad`."""
    names = ("q", "k", "v", "log_alpha", "beta", "initial_state")
    leaf = {n: None if x[n] is None else x[n].detach().double().requires_grad_(grad) for n in names}
    H, dv = leaf["v"].shape[1:]
    Hq, dk = leaf["q"].shape[1:]
    q, k = (leaf[n].repeat_interleave(H // Hq, 1) for n in ("q", "k"))
    a = leaf["log_alpha"].exp()
    a = a if a.dim() == 3 else a.unsqueeze(-1)
    ends = x["offsets"].tolist()
    o = [None] * leaf["v"].shape[0]
    finals = []
    for n in range(N):
        S = (leaf["v"].new_zeros(H, dv, dk) if leaf["initial_state"] is None
             else leaf["initial_state"][n])
        for t in range(ends[n], ends[n + 1]):
            S = S * a[t].unsqueeze(1)
            w = leaf["v"][t]
            if mixer in (GDN, KDA):
                w = w - (S * k[t].unsqueeze(1)).sum(-1)
            if leaf["beta"] is not None:
                w = w * leaf["beta"][t].unsqueeze(-1)
            S = S + w.unsqueeze(-1) * k[t].unsqueeze(1)
            o[t] = (S * q[t].unsqueeze(1)).sum(-1)
        finals.append(S + 0.0 * leaf["v"].sum())  # of the graph even where no token is
    zero = leaf["v"].new_zeros(H, dv)
    o = torch.stack([zero if r is None else r for r in o]) if o else leaf["v"]
    return o, torch.stack(finals), leaf


def norm64(x, weight, gate, residual, scale, next_weight, eps, act):
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        n = n * weight
    if gate is not None:
        s = torch.sigmoid(gate)
        n = n * (gate * s if act == 0 else s)
    if scale is not None:
        n = n * scale
    r = n if residual is None else residual + n
    if next_weight is None:
        return (r,)
    return r, r * torch.rsqrt(r.square().mean(-1, keepdim=True) + eps) * next_weight


def rel(a, b):
    """Distance of a from b, relative to b."""
    a, b = a.detach().double().cpu(), b.detach().double().cpu()
    n = float(b.norm())
    d = float((a - b).norm())
    return d / n if n > 0 else d
