"""Drafted tokens over a stored state in 64 bits, node by node and without any of
the library's code, for the tests."""

import torch

GDN, GLA, SCALAR, KDA = 0, 1, 2, 3
MIXERS = {"gdn": GDN, "gla": GLA, "scalar": SCALAR, "kda": KDA}

# Errors are relative to the 2-norm of the reference.
# An FP32 readout goes through three chained products (K S, the nodes' triangular system, A W); a
# product accumulates at most 48 matrix instructions (dk = 256: 8 of 32 columns times 6 pairs of
# terms), each rounding to 2^-24.  Decays along a path of up to 64 nodes are multiplied up, one
# rounding and an exponential's two ulps each, in q and in k.
VERIFY = (3 * 48 + 2 * 3 * 64) * 2.0 ** -24
# The state's way takes up to 64 decays the same way and adds up to 64 writes.
ACCEPT = (3 * 64 + 64 + 8) * 2.0 ** -24


def tolerance(dtype):
    """A 16-bit output is rounded once, by at most half a step of its value, so its norm is too."""
    return VERIFY if dtype == torch.float32 else torch.finfo(dtype).eps / 2 + VERIFY


def parents_of(shape, N, T, g):
    """int32 [N][T]: "chain", "tree" (several children of the stored state among them), "ragged"
    (rows behind each sequence's own number of nodes are none), "none" (no nodes at all)."""
    t = torch.arange(T)
    if shape == "chain":
        return (t - 1).expand(N, T).to(torch.int32).contiguous()
    if shape == "none":
        return torch.full((N, T), -2, dtype=torch.int32)
    p = (torch.rand((N, T), generator=g) * (t + 1)).long().clamp(max=t) - 1
    if shape == "ragged":
        p = torch.where(t < torch.randint(0, T + 1, (N, 1), generator=g), p, -2)
    return p.to(torch.int32)


def inputs(mixer, N, T, shape, H, Hq, dk, dv, dtype, device, seed=0, gate=1.0):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    q, k = normal(N, T, Hq, dk), normal(N, T, Hq, dk)
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    la = -torch.nn.functional.softplus(normal(*((N, T, H, dk) if mixer in (GLA, KDA)
                                                else (N, T, H))) - 3.0) * gate
    x = {"q": q.to(dtype), "k": k.to(dtype), "v": normal(N, T, H, dv).to(dtype),
         "log_alpha": la.float(),
         "beta": None if mixer == GLA else torch.sigmoid(normal(N, T, H)).float(),
         "parents": parents_of(shape, N, T, g)}
    S = (0.3 * normal(N, H, dv, dk)).float()
    return {n: None if t is None else t.to(device) for n, t in x.items()}, S.to(device)


def node_mask(parents):
    """bool [N][T]: rows that are nodes, and whose whole path is."""
    ok = torch.zeros(parents.shape, dtype=torch.bool)
    for n, row in enumerate(parents.tolist()):
        for t, p in enumerate(row):
            ok[n, t] = -1 <= p < t and (p < 0 or bool(ok[n, p]))
    return ok


def verify64(x, S, mixer):
    """(o, writes, the state behind every node [T][N][H][dv][dk])."""
    N, T, H, dv = x["v"].shape
    rep = H // x["q"].shape[2]
    ok = node_mask(x["parents"]).to(S.device)
    par = x["parents"].long().clamp(min=-1)
    par = torch.where(ok, par, torch.full_like(par, -1))
    rows = torch.arange(N, device=S.device)
    kept, o, writes = [S.double()], [], []
    for t in range(T):
        live = ok[:, t, None, None]
        before = torch.stack(kept)[par[:, t] + 1, rows]
        q, k = (x[n][:, t].double().repeat_interleave(rep, 1) for n in ("q", "k"))
        a = x["log_alpha"][:, t].double().clamp(min=-87.0).exp()
        a = a if a.dim() == 3 else a.unsqueeze(-1)
        d = before * a.unsqueeze(2)
        w = x["v"][:, t].double()
        if mixer in (GDN, KDA):
            w = w - (d * k.unsqueeze(2)).sum(-1)
        if x["beta"] is not None:
            w = w * x["beta"][:, t].double().unsqueeze(-1)
        d = d + w.unsqueeze(-1) * k.unsqueeze(2)
        kept.append(d)
        zero = torch.zeros_like(w)
        o.append(torch.where(live, (d * q.unsqueeze(2)).sum(-1), zero))
        writes.append(torch.where(live, w, zero))
    return torch.stack(o, 1), torch.stack(writes, 1), torch.stack(kept[1:])


def accept64(x, S, states, last):
    """The state behind each sequence's last node."""
    ok = node_mask(x["parents"])
    out = S.double().clone()
    T = x["parents"].shape[1]
    for n, t in enumerate(last.tolist()):
        if 0 <= t < T and ok[n, t]:
            out[n] = states[t, n]
    return out
