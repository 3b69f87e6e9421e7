"""What the sequence operators are measured on: the scan of a gated recurrence
over whole sequences, its gradients, and the norms around the mixer block with
theirs.

A scan case is N sequences packed behind each other ([tokens][heads][d] with
offsets [N + 1]); "lens" says how the lengths are drawn: "equal" (T each) or
"ragged" (0..T, the first of them T).  A norm case is [rows][groups][width].
Sizes are those of the decode workloads (heads 4 to 32, dk = 64 / 128, dv = 64
/ 128, Mamba2's shared B and C) at lengths from one token to a long prompt.
"""

import math

import torch

own = False

GDN, GLA, SCALAR, KDA = 0, 1, 2, 3
_MIXER = {"gdn": GDN, "gla": GLA, "scalar": SCALAR, "kda": KDA}
_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _scan(name, op, mixer, dtype, N, T, lens, H, Hq, dk, dv, state):
    c = {"op": op, "mixer": mixer, "dtype": dtype, "N": N, "T": T, "lens": lens, "H": H, "Hq": Hq,
         "dk": dk, "dv": dv, "state": state}
    return dict(c, name=name) if name else c


def _norm(name, op, dtype, rows, groups, width, gate, residual, scale, after, before):
    c = {"op": op, "dtype": dtype, "rows": rows, "groups": groups, "width": width, "gate": gate,
         "residual": residual, "scale": scale, "after": after, "before": before}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token for each of 64 running sequences: serving's smallest step
        _scan("gdn_tokens", "scan", "gdn", "bf16", 64, 1, "equal", 16, 16, 128, 128, True),
        # short chunks of new tokens of running sequences, some with none (a serving batch)
        _scan("gla_chunks", "scan", "gla", "f32", 96, 33, "ragged", 16, 16, 128, 128, True),
        # prompts of unequal length before decoding, key heads shared by two value heads
        _scan("gdn_prompts", "scan", "gdn", "bf16", 6, 2900, "ragged", 32, 16, 128, 128, False),
        # one long prompt, a decay for each key channel
        _scan("kda_long", "scan", "kda", "bf16", 1, 8190, "equal", 16, 16, 128, 128, False),
        # a small training step in FP32 at the smallest head size, odd lengths, odd dv
        _scan("gla_small_grad", "scan_grad", "gla", "f32", 3, 131, "ragged", 4, 4, 64, 40, True),
        # a training step of one Gated DeltaNet layer
        _scan("gdn_grad", "scan_grad", "gdn", "bf16", 2, 2048, "equal", 16, 16, 128, 128, False),
        # a training step of one Mamba2 layer: B and C shared by all heads, head size 64
        _scan("mamba2_grad", "scan_grad", "scalar", "bf16", 4, 1024, "equal", 32, 1, 128, 64, False),
        # a training step of one KDA layer on packed documents
        _scan("kda_grad", "scan_grad", "kda", "bf16", 5, 777, "ragged", 16, 16, 128, 128, True),
        # the readout's norm and gate, one decoded token of 64 sequences
        _norm("readout_norm", "norm", "bf16", 64, 32, 128, True, False, False, "shared", "none"),
        # the block's end over a prompt: norm, gate, residual, scale, the next block's norm
        _norm("block_norm", "norm", "bf16", 8191, 1, 4096, True, True, True, "shared", "shared"),
        # the readout's norm in training, a weight for each head
        _norm("readout_norm_grad", "norm_grad", "f32", 2047, 16, 128, True, False, False, "each", "none"),
        # the block's end in training
        _norm("block_norm_grad", "norm_grad", "bf16", 8192, 1, 4096, True, True, True, "shared", "shared"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["scan", "scan_grad", "norm", "norm_grad"])
    if op in ("scan", "scan_grad"):
        mixer = rng.choice(["gdn", "gla", "scalar", "kda"])
        T = _log_int(rng, 1, 8190 if op == "scan" else 2048)
        H = rng.choice([4, 16, 32])
        Hq = rng.choice([H, H, H // 2, 1])
        tokens = (16384 if op == "scan" else 4096) * 16 // H
        N = max(1, min(_log_int(rng, 1, 128), tokens // T))
        return _scan(None, op, mixer, rng.choice(["bf16", "bf16", "f16", "f32"]), N, T,
                     rng.choice(["equal", "ragged"]), H, Hq, rng.choice([64, 128]),
                     rng.choice([40, 64, 128]), rng.choice([True, False]))
    groups = rng.choice([1, 1, 16, 32])
    width = rng.choice([64, 128]) if groups > 1 else _log_int(rng, 64, 4096)
    rows = _log_int(rng, 1, max(1, min(65536, 8192 * 4096 // (groups * width))))
    residual = rng.choice([True, False])
    return _norm(None, op, rng.choice(["bf16", "f16", "f32"]), rows, groups, width,
                 rng.choice([True, False]), residual, residual and rng.choice([True, False]),
                 rng.choice(["shared", "each"]), rng.choice(["none", "shared"]))


# ---- inputs -----------------------------------------------------------------------------------


def _lengths(case):
    if case["lens"] == "equal":
        return [case["T"]] * case["N"]
    g = torch.Generator().manual_seed(case["N"] * 8191 + case["T"])
    rest = torch.randint(0, case["T"] + 1, (case["N"] - 1,), generator=g).tolist()
    return [case["T"]] + rest


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPE[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if "mixer" not in case:
        shape = (case["rows"], case["groups"], case["width"])
        each = case["after"] == "each"
        s = {"x": normal(*shape).to(dt), "gate": normal(*shape).to(dt) if case["gate"] else None,
             "residual": (2.0 * normal(*shape)).to(dt) if case["residual"] else None,
             "weight": 1.0 + 0.1 * normal(*(shape[1:] if each else shape[2:])),
             "scale": 0.5 + 0.1 * normal(shape[2]) if case["scale"] else None,
             "next_weight": 1.0 + 0.1 * normal(shape[2]) if case["before"] == "shared" else None}
        if case["op"] == "norm_grad":
            s["dy"] = normal(*shape).to(dt)
            s["dh"] = normal(*shape).to(dt) if case["before"] == "shared" else None
        return s
    N, H, Hq, dk, dv = (case[n] for n in ("N", "H", "Hq", "dk", "dv"))
    lens = _lengths(case)
    total, longest = sum(lens), max(lens)
    soft = torch.nn.functional.softplus
    q, k, v = normal(total, Hq, dk), normal(total, Hq, dk), normal(total, H, dv)
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    beta = torch.sigmoid(normal(total, H))
    if case["mixer"] in ("gla", "kda"):  # alpha = sigmoid(N(3, 1))^(1/16) for each channel
        log_alpha = -soft(-(3.0 + normal(total, H, dk))) / 16.0
    elif case["mixer"] == "scalar":  # alpha = exp(-softplus(a_h) dt), the write weight is dt
        beta = 0.001 + 0.099 * torch.rand((total, H), generator=g, device="cuda")
        log_alpha = -soft(normal(H) - 3.0) * beta
    else:
        log_alpha = -soft(normal(total, H) - 4.0)
    s = {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "log_alpha": log_alpha,
         "beta": None if case["mixer"] == "gla" else beta,
         "S0": 0.3 * normal(N, H, dv, dk) if case["state"] else None}
    if case["op"] == "scan_grad":
        s["do"] = normal(total, H, dv).to(dt)
        s["dS"] = 0.1 * normal(N, H, dv, dk)
    ends = torch.tensor([0] + lens).cumsum(0)
    s["offsets"] = ends.cuda()
    # token i of the packed rows is row `place[i]` of a padded [N][longest]
    at = torch.repeat_interleave(torch.arange(N), torch.tensor(lens))
    s["place"] = (at * longest + torch.arange(total) - ends[at]).cuda()
    s["longest"] = longest
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    for n in ("q", "k", "v", "log_alpha", "beta", "S0", "x", "gate", "residual", "weight", "scale", "next_weight"):
        if case["op"].endswith("_grad") and s.get(n) is not None:
            s[n].requires_grad_(True)
    return s


# ---- the plain form ---------------------------------------------------------------------------


def _padded(x, s, N, length):
    """[tokens][...] -> [N][length][...], zeros behind each sequence's end."""
    y = x.new_zeros((N * s["longest"],) + x.shape[1:]).index_copy(0, s["place"], x)
    y = y.view((N, s["longest"]) + x.shape[1:])
    return torch.cat([y, y.new_zeros((N, length - s["longest"]) + x.shape[1:])], 1)


def _inverse(L, C):
    """(I + L)^-1 for strictly lower triangular L: the inverses of the diagonal blocks, each twice
    as large as before, [[P, 0], [-Q L21 P, Q]] from the halves' P and Q."""
    X = torch.eye(C, device=L.device).expand(L.shape)
    i = torch.arange(C, device=L.device)
    for bit in range((C - 1).bit_length()):
        row, col = (i >> bit)[:, None], (i >> bit)[None, :]
        X = X - X @ (L * ((row % 2 == 1) & (col == row - 1))) @ X
    return X


def _plain_scan(s):
    """Chunks of C tokens: products inside every chunk at once, then one loop over the chunks that
    carries the state (the recurrence leaves no other order).  All in 32 bits, the sums of log
    decays in 64."""
    case = s["case"]
    mixer, N, H, dk, dv = case["mixer"], case["N"], case["H"], case["dk"], case["dv"]
    vector, delta = mixer in ("gla", "kda"), mixer in ("gdn", "kda")
    # a power of two, no longer than the sequences need
    C = min(16 if vector else 64, 1 << (s["longest"] - 1).bit_length())
    n = max(1, -(-s["longest"] // C))

    def chunks(x):  # [tokens][H][...] -> [N][H][n][C][...]
        x = _padded(x, s, N, n * C)
        return x.view((N, n, C) + x.shape[2:]).movedim(3, 1)

    q, k = (s[x].float().repeat_interleave(H // case["Hq"], 1) for x in ("q", "k"))
    q, k, v = chunks(q), chunks(k), chunks(s["v"].float())
    c = chunks(s["log_alpha"].double()).cumsum(3)
    b = torch.ones_like(v[..., 0]) if mixer == "gla" else chunks(s["beta"])
    i = torch.arange(C, device=q.device)
    below = i[:, None] >= i[None, :]
    if vector:
        G = (c.unsqueeze(4) - c.unsqueeze(3)).float().masked_fill(~below[:, :, None], -math.inf).exp()
        A = (q.unsqueeze(4) * k.unsqueeze(3) * G).sum(-1)
        L = (k.unsqueeze(4) * k.unsqueeze(3) * G).sum(-1) if delta else None
    else:
        G = (c.unsqueeze(4) - c.unsqueeze(3)).float().masked_fill(~below, -math.inf).exp()
        A = (q @ k.mT.contiguous()) * G
        L = (k @ k.mT.contiguous()) * G if delta else None
        c = c.unsqueeze(-1)
    e = c.float().exp()
    out = (c[..., -1:, :] - c).float().exp()
    last = e[..., -1:, :]  # [N][H][n][1][dk or 1]
    qe, ke, ko = q * e, k * e, k * out
    if delta:
        X = _inverse(torch.tril(L, -1) * b.unsqueeze(-2), C)
        v, ke = X @ v, X @ ke
    S = q.new_zeros((N, H, dv, dk)) if s["S0"] is None else s["S0"]
    o = []
    for vc, kc, qc, Ac, bc, oc, lc in zip(*(x.unbind(2) for x in (v, ke, qe, A, b, ko, last))):
        St = S.mT.contiguous()
        u = vc - kc @ St if delta else vc
        w = u * bc.unsqueeze(-1)
        o.append(qc @ St + Ac @ w)
        S = S * lc + w.mT.contiguous() @ oc
    o = torch.stack(o, 2).movedim(1, 3).reshape(N, n * C, H, dv)[:, :s["longest"]]
    return o.reshape(N * s["longest"], H, dv)[s["place"]].to(s["v"].dtype), S


_EPS = 1e-6


def _plain_norm(s):
    y = s["x"].float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * s["weight"]
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z / (1.0 + torch.exp(-z)))
    if s["scale"] is not None:
        y = y * s["scale"]
    if s["residual"] is not None:
        y = s["residual"].float() + y
    dt = s["x"].dtype
    if s["next_weight"] is None:
        return (y.to(dt),)
    h = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + _EPS) * s["next_weight"]
    return y.to(dt), h.to(dt)


# ---- one pass ---------------------------------------------------------------------------------

_SCAN_LEAVES = ("q", "k", "v", "log_alpha", "beta", "S0")
_NORM_LEAVES = ("x", "gate", "residual", "weight", "scale", "next_weight")


def _forward(s):
    case = s["case"]
    if "mixer" in case:
        if own:
            from bit_recurrent_state_amd import scan
            return scan(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"], mixer=_MIXER[case["mixer"]],
                        initial_state=s["S0"], offsets=s["offsets"])
        return _plain_scan(s)
    if own:
        from bit_recurrent_state_amd import block_norm
        y = block_norm(s["x"], weight=s["weight"], gate=s["gate"], residual=s["residual"],
                       scale=s["scale"], next_weight=s["next_weight"], eps=_EPS)
        return y if isinstance(y, tuple) else (y,)
    return _plain_norm(s)


def run(s):
    op = s["case"]["op"]
    if not op.endswith("_grad"):
        with torch.no_grad():
            return list(_forward(s))
    out = _forward(s)
    leaves = [s[n] for n in (_SCAN_LEAVES if op == "scan_grad" else _NORM_LEAVES) if s[n] is not None]
    seeds = (s["do"], s["dS"]) if op == "scan_grad" else tuple(x for x in (s["dy"], s["dh"]) if x is not None)
    return [x.detach() for x in out] + list(torch.autograd.grad(out, leaves, seeds))


# ---- the definition in 64 bits ----------------------------------------------------------------


def _exact_scan(case, s):
    """Token by token: S = S diag(alpha), w, S += w k^T, o = S q, over sequences sorted by length."""
    N, H, dk, dv = case["N"], case["H"], case["dk"], case["dv"]
    ends = s["offsets"].tolist()
    grad = case["op"] == "scan_grad"
    x = {n: None if s[n] is None else s[n].detach().double().requires_grad_(grad) for n in _SCAN_LEAVES}
    alpha = x["log_alpha"].exp()
    alpha = alpha if alpha.dim() == 3 else alpha.unsqueeze(-1)
    q, k = (x[n].repeat_interleave(H // case["Hq"], 1) for n in ("q", "k"))
    order = sorted(range(N), key=lambda j: ends[j] - ends[j + 1])
    S = torch.zeros((N, H, dv, dk), dtype=torch.float64, device="cuda") if x["S0"] is None else x["S0"]
    S = S[order]
    done, rows, o = [], [], []
    for t in range(s["longest"]):
        live = [j for j in order if ends[j + 1] - ends[j] > t]
        if len(live) < S.shape[0]:
            done.append(S[len(live):])
            S = S[:len(live)]
        at = torch.tensor([ends[j] + t for j in live], device="cuda")
        kt, w = k[at], x["v"][at]
        S = S * alpha[at].unsqueeze(2)
        if case["mixer"] in ("gdn", "kda"):
            w = w - (S * kt.unsqueeze(2)).sum(-1)
        if x["beta"] is not None:
            w = w * x["beta"][at].unsqueeze(-1)
        S = S + w.unsqueeze(-1) * kt.unsqueeze(2)
        o.append((S * q[at].unsqueeze(2)).sum(-1))
        rows.append(at)
    S = torch.cat([S] + done[::-1])
    back = torch.empty(N, dtype=torch.int64)
    back[order] = torch.arange(N)
    S = S[back.cuda()]
    o = torch.zeros_like(x["v"]).index_copy(0, torch.cat(rows), torch.cat(o))
    if not grad:
        return [o, S]
    leaves = [x[n] for n in _SCAN_LEAVES if x[n] is not None]
    grads = torch.autograd.grad((o, S), leaves, (s["do"].double(), s["dS"].double()))
    return [o.detach(), S.detach()] + list(grads)


def _exact_norm(case, s):
    """The forward and its gradients written out by hand."""
    D = case["width"]
    x, w = s["x"].detach().double(), s["weight"].detach().double()
    r1 = 1.0 / torch.sqrt((x * x).sum(-1, keepdim=True) / D + _EPS)
    z = None if s["gate"] is None else s["gate"].detach().double()
    a = 1.0 if z is None else z * torch.sigmoid(z)
    c = 1.0 if s["scale"] is None else s["scale"].detach().double()
    y = x * r1 * w * a * c
    if s["residual"] is not None:
        y = y + s["residual"].detach().double()
    out, w2 = [y], s["next_weight"]
    if w2 is not None:
        w2 = w2.detach().double()
        r2 = 1.0 / torch.sqrt((y * y).sum(-1, keepdim=True) / D + _EPS)
        out.append(y * r2 * w2)
    if case["op"] == "norm":
        return out
    dy, dw2 = s["dy"].double(), None
    if w2 is not None:
        dh = s["dh"].double()
        dw2 = (dh * y * r2).sum((0, 1))
        m = dh * w2
        dy = dy + r2 * (m - y * r2 * r2 * (m * y).sum(-1, keepdim=True) / D)
    n = x * r1
    dn = dy * c * a * w
    grads = [r1 * (dn - n * (dn * n).sum(-1, keepdim=True) / D)]
    if z is not None:
        sg = torch.sigmoid(z)
        grads.append(dy * c * n * w * (sg + z * sg * (1.0 - sg)))
    if s["residual"] is not None:
        grads.append(dy)
    grads.append((dy * c * a * n).sum(0 if w.dim() == 2 else (0, 1)))
    if s["scale"] is not None:
        grads.append((dy * n * w * a).sum((0, 1)))
    if dw2 is not None:
        grads.append(dw2)
    return out + grads


def exact(case, seed):
    s = _inputs(case, seed)
    if "mixer" not in case:
        return _exact_norm(case, s)
    if case["op"] == "scan_grad":
        # the states of every token are kept for the backward sweep
        if sum(_lengths(case)) * case["H"] * case["dk"] * case["dv"] * 8 * 4 > 120e9:
            return None
        return _exact_scan(case, s)
    with torch.no_grad():
        return _exact_scan(case, s)


# ---- the work ---------------------------------------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if "mixer" not in case:
        e = case["rows"] * case["groups"] * case["width"]
        streams = 2 + case["gate"] + case["residual"] + (case["before"] == "shared")
        flops = e * (6 + 4 * case["gate"] + 2 * case["residual"] + 4 * (case["before"] == "shared"))
        if case["op"] == "norm_grad":
            # the outputs' gradients are read, those of x, gate and residual written
            streams += 2 + case["gate"] + case["residual"] + (case["before"] == "shared")
            flops *= 3
        return {"bytes": e * size * streams, "flops": flops}
    H, Hq, dk, dv = case["H"], case["Hq"], case["dk"], case["dv"]
    mean = case["T"] if case["lens"] == "equal" else (case["T"] + (case["N"] - 1) * case["T"] / 2) / case["N"]
    tokens = int(case["N"] * mean)
    vector, delta = case["mixer"] in ("gla", "kda"), case["mixer"] in ("gdn", "kda")
    state = case["N"] * H * dk * dv * 4
    gates = 4 * H * ((dk if vector else 1) + (case["mixer"] != "gla"))
    per_token = (2 * Hq * dk + 2 * H * dv) * size + gates
    # decay, (S k,) write and S q for each element of the state
    flops = tokens * H * dk * dv * (5 + 2 * delta)
    bytes_ = tokens * per_token + state * (1 + case["state"])
    if case["op"] == "scan_grad":
        # do read, dq, dk, dv and the gates' gradients written; the final state's gradient read
        bytes_ += tokens * (per_token + H * dv * size) + state * (1 + case["state"])
        flops *= 3
    return {"bytes": bytes_, "flops": flops}
