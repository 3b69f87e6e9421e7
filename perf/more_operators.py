"""What decoding drafted tokens is measured on: a tree of drafted tokens over the stored recurrent
state (verify), the state's way along the accepted path (accept), the group norm of the readout with
its gradients, and the projections around them with 4-bit weights.

A verify or accept case is N sequences of T drafted nodes each; "shape" says how they hang together:
"chain" (every node on the one before), "tree" (parents drawn), "ragged" (a tree, and each sequence
has its own number of nodes, the rest of its T rows hold none).  "store" is what the state is held in:
"f32", "int8", "int4", or "mix" (the first quarter of the heads INT8, the others INT4), with scales
per value row and `group` key columns.  A norm case is [rows][groups][width], a linear case [rows][inputs]
times [outputs][inputs].  Sizes are those of the decode workloads (heads 4 to 32, dk = 64 / 128,
dv = 64 / 128, 1 to 256 sequences) and of a model width of 4096 around them.
"""

import math

import torch

own = False

GDN, GLA, SCALAR, KDA = 0, 1, 2, 3
_MIXER = {"gdn": GDN, "gla": GLA, "scalar": SCALAR, "kda": KDA}
_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _draft(name, op, mixer, dtype, N, T, shape, H, Hq, dk, dv, store, group):
    c = {"op": op, "mixer": mixer, "dtype": dtype, "N": N, "T": T, "shape": shape, "H": H, "Hq": Hq,
         "dk": dk, "dv": dv, "store": store, "group": group}
    return dict(c, name=name) if name else c


def _norm(name, op, dtype, rows, groups, width, mode, center):
    c = {"op": op, "dtype": dtype, "rows": rows, "groups": groups, "width": width, "mode": mode,
         "center": center}
    return dict(c, name=name) if name else c


def _linear(name, dtype, rows, inputs, outputs, group, bias):
    c = {"op": "linear", "dtype": dtype, "rows": rows, "inputs": inputs, "outputs": outputs,
         "group": group, "bias": bias}
    return dict(c, name=name) if name else c


def listed():
    return [
        # five drafted tokens of one sequence, one after the other: the smallest call
        _draft("verify_one", "verify", "gdn", "f32", 1, 5, "chain", 4, 4, 64, 40, "f32", 64),
        # the largest: a serving batch, 16 nodes each, over INT4 states (a quarter of the heads INT8)
        _draft("verify_tree", "verify", "gdn", "bf16", 256, 16, "tree", 32, 32, 128, 128, "mix", 32),
        # a decay for each key channel, an odd number of nodes, sequences with fewer of them
        _draft("verify_kda", "verify", "kda", "f16", 64, 33, "ragged", 16, 16, 128, 128, "int8", 64),
        # wide trees over a Mamba2-style layer, B and C shared by all heads
        _draft("verify_mamba2", "verify", "scalar", "bf16", 32, 64, "tree", 32, 1, 128, 64, "int4", 64),
        # the accepted path of a few sequences enters FP32 states
        _draft("accept_f32", "accept", "kda", "f16", 16, 8, "ragged", 16, 16, 128, 128, "f32", 64),
        # the accepted path of a serving batch enters INT8 states
        _draft("accept_int8", "accept", "gdn", "bf16", 128, 16, "tree", 16, 16, 128, 128, "int8", 32),
        # the readout's group norm and gate (RetNet), one decoded token of 64 sequences
        _norm("group_norm_readout", "norm", "bf16", 64, 32, 128, "gate", True),
        # the gated RMS norm of a Mamba2 block over a prompt, the gate before the norm
        _norm("group_norm_prompt", "norm", "bf16", 8191, 8, 512, "gate_first", False),
        # a training step of the group norm with its activation
        _norm("group_norm_grad", "norm_grad", "bf16", 8192, 32, 128, "activate", True),
        # the output projection of one decoded token
        _linear("linear_one", "bf16", 1, 4096, 4096, 64, False),
        # the input projections (q, k, v of 32 heads of 128 together) of 16 decoded tokens
        _linear("linear_batch", "bf16", 16, 4096, 12288, 128, False),
        # drafted tokens of a few sequences, odd sizes, a bias
        _linear("linear_draft", "f16", 61, 2080, 4100, 32, True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["verify", "verify", "accept", "norm", "norm_grad", "linear"])
    if op in ("verify", "accept"):
        mixer = rng.choice(["gdn", "gla", "scalar", "kda"])
        H, dk, T = rng.choice([4, 16, 32]), rng.choice([64, 128]), _log_int(rng, 1, 64)
        most = 131072 // (H * T) if mixer in ("gdn", "scalar") else 150000000 // (H * T * T * dk)
        if op == "accept":
            most = min(most, 2048 // H)
        return _draft(None, op, mixer, rng.choice(["bf16", "bf16", "f16", "f32"]),
                      max(1, min(_log_int(rng, 1, 256), most)), T,
                      rng.choice(["chain", "tree", "ragged"]), H, rng.choice([H, H, H // 2, 1]), dk,
                      rng.choice([40, 64, 128]),
                      rng.choice(["f32", "int8", "int4", "mix"] if op == "verify" else ["f32", "int8"]),
                      rng.choice([32, 64]))
    if op == "linear":
        group = rng.choice([32, 64, 128])
        return _linear(None, rng.choice(["bf16", "bf16", "f16", "f32"]), _log_int(rng, 1, 64),
                       group * _log_int(rng, 1, 4096 // group), _log_int(rng, 16, 8192), group,
                       rng.choice([True, False]))
    groups = rng.choice([1, 4, 16, 32])
    width = _log_int(rng, 32, 4096 // groups)
    rows = _log_int(rng, 1, max(1, min(65536, 8192 * 4096 // (groups * width))))
    return _norm(None, op, rng.choice(["bf16", "f16", "f32"]), rows, groups, width,
                 rng.choice(["plain", "gate", "gate_first", "activate"]), rng.choice([True, False]))


# ---- inputs -----------------------------------------------------------------------------------


def _heads8(case):
    """How many heads, from the first one, are held in INT8."""
    return {"f32": 0, "int8": case["H"], "int4": 0, "mix": case["H"] // 4}[case["store"]]


def _quantized(S, r, G):
    """Codes and scales of S [.., dk]: absmax over G columns, rounded to nearest."""
    x = S.unflatten(-1, (-1, G))
    m = x.abs().amax(-1, keepdim=True)
    return (x * (r / m)).round().to(torch.int8).flatten(-2), (m / r).squeeze(-1)


def _nibbles(c):
    """Two codes a byte, the even column in the low four bits."""
    c = c.view(torch.uint8)
    return (c[..., 0::2] & 15) | (c[..., 1::2] << 4)


def _parents(case, g):
    """[N][T] parents; -1 is the stored state, -2 marks a row of no node."""
    N, T = case["N"], case["T"]
    t = torch.arange(T, device="cuda")
    if case["shape"] == "chain":
        return (t - 1).expand(N, T).to(torch.int32).contiguous()
    # node 0 continues the sequence, later ones hang on one of the six nodes before them
    back = torch.randint(1, 7, (N, T), generator=g, device="cuda")
    p = torch.where(t == 0, -1, (t - back).clamp(min=0))
    if case["shape"] == "ragged":
        nodes = torch.randint(0, T + 1, (N, 1), generator=g, device="cuda")
        nodes[0] = T
        p = torch.where(t < nodes, p, -2)
    return p.to(torch.int32)


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DTYPE[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if case["op"] in ("norm", "norm_grad"):
        rows, groups, width = case["rows"], case["groups"], case["width"]
        C = groups * width
        s = {"x": (normal(rows, C) + 0.5).to(dt),
             "gate": normal(rows, C).to(dt) if case["mode"] in ("gate", "gate_first") else None,
             "weight": 1.0 + 0.1 * normal(C), "bias": 0.1 * normal(C)}
        if case["op"] == "norm_grad":
            s["dy"] = normal(rows, C).to(dt)
        return s
    if case["op"] == "linear":
        M, K, O, G = case["rows"], case["inputs"], case["outputs"], case["group"]
        codes, scales = _quantized(normal(O, K) / math.sqrt(K), 7.0, G)
        return {"x": normal(M, K).to(dt), "codes": codes, "scales": scales,
                "bias": normal(O) if case["bias"] else None}
    N, T, H, Hq, dk, dv = (case[n] for n in ("N", "T", "H", "Hq", "dk", "dv"))
    soft = torch.nn.functional.softplus
    q, k, v = normal(N, T, Hq, dk), normal(N, T, Hq, dk), normal(N, T, H, dv)
    q, k = (x / x.square().sum(-1, keepdim=True).sqrt() for x in (q, k))
    beta = torch.sigmoid(normal(N, T, H))
    if case["mixer"] in ("gla", "kda"):  # alpha = sigmoid(N(3, 1))^(1/16) for each channel
        log_alpha = -soft(-(3.0 + normal(N, T, H, dk))) / 16.0
    elif case["mixer"] == "scalar":  # alpha = exp(-softplus(a_h) dt), the write weight is dt
        beta = 0.001 + 0.099 * torch.rand((N, T, H), generator=g, device="cuda")
        log_alpha = -soft(normal(H) - 3.0) * beta
    else:
        log_alpha = -soft(normal(N, T, H) - 4.0)
    s = {"q": q.to(dt), "k": k.to(dt), "v": v.to(dt), "log_alpha": log_alpha,
         "beta": None if case["mixer"] == "gla" else beta, "parents": _parents(case, g)}
    S = 0.3 * normal(N, H, dv, dk)
    if case["store"] == "f32":
        s["state"] = S
    else:
        n = _heads8(case)
        c8, s8 = _quantized(S[:, :n], 127.0, case["group"])
        c4, s4 = _quantized(S[:, n:], 7.0, case["group"])
        s["codes"] = torch.cat([c8.view(torch.uint8).flatten(1), _nibbles(c4).flatten(1)], 1)
        s["scales"] = torch.cat([s8, s4], 1)
    if case["op"] == "accept":
        # what verify left for the nodes, and the last node that was accepted (-1: none)
        s["writes"] = 0.3 * normal(N, T, H, dv)
        nodes = (s["parents"] != -2).sum(1)
        u = torch.rand(N, generator=g, device="cuda")
        s["last"] = ((u * (nodes + 1)).long().clamp(max=T) - 1).minimum(nodes - 1).to(torch.int32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] == "norm_grad":
        for n in ("x", "gate", "weight", "bias"):
            if s[n] is not None:
                s[n].requires_grad_(True)
    if case["op"] == "linear":
        s["nibbles"] = _nibbles(s.pop("codes"))
    if own:
        from bit_recurrent_state_amd import Config, Draft, QState, Weight4
        if case["op"] == "linear":
            s["weight"] = Weight4.from_nibbles(s["nibbles"], s["scales"])
        elif case["op"] in ("verify", "accept"):
            n, H = _heads8(case), case["H"]
            st = QState(Config(batch=case["N"], heads=H, dk=case["dk"], dv=case["dv"], group=case["group"],
                               mixer=_MIXER[case["mixer"]], fp32_state=case["store"] == "f32",
                               head_bits=None if case["store"] == "f32" else [8] * n + [4] * (H - n)))
            if case["store"] == "f32":
                st.codes.copy_(s["state"].flatten())
            else:
                st.codes.copy_(s["codes"].flatten())
                st.scales.copy_(s["scales"].flatten())
            s["handle"] = st
            if case["op"] == "accept":
                s["draft"] = Draft(s["k"], s["log_alpha"], s["parents"], s["writes"])
    return s


# ---- the plain form ---------------------------------------------------------------------------


def _signed(b):
    """The two codes of each byte, as numbers."""
    b = torch.stack([b & 15, b >> 4], -1).flatten(-2).to(torch.int8)
    return torch.where(b > 7, b - 16, b)


def _values(s):
    """The stored state [N][H][dv][dk] in FP32."""
    case = s["case"]
    if case["store"] == "f32":
        return s["state"]
    N, H, dv, dk, n = case["N"], case["H"], case["dv"], case["dk"], _heads8(case)
    cut = n * dv * dk
    c8 = s["codes"][:, :cut].view(torch.int8).view(N, n, dv, dk)
    c4 = _signed(s["codes"][:, cut:]).view(N, H - n, dv, dk)
    c = torch.cat([c8, c4], 1).float().unflatten(-1, (-1, case["group"]))
    return (c * s["scales"].unsqueeze(-1)).flatten(-2)


def _ancestors(parents):
    """[N][T][T]: whether column j is row i's node itself or lies on its way to the stored state;
    rows of no node are empty."""
    T = parents.shape[1]
    i = torch.arange(T, device=parents.device)
    M = ((parents.unsqueeze(2) == i) | (i[:, None] == i)).float()
    for _ in range((T - 1).bit_length()):
        M = ((M @ M) > 0).float()
    return M * (parents >= -1).unsqueeze(2)


def _inverse(L, T):
    """(I + L)^-1 for strictly lower triangular L: the inverses of the diagonal blocks, each twice
    as large as before, [[P, 0], [-Q L21 P, Q]] from the halves' P and Q."""
    X = torch.eye(T, device=L.device).expand(L.shape)
    i = torch.arange(T, device=L.device)
    for bit in range((T - 1).bit_length()):
        row, col = (i >> bit)[:, None], (i >> bit)[None, :]
        X = X - X @ (L * ((row % 2 == 1) & (col == row - 1))) @ X
    return X


def _paths(s):
    """What both draft operators need: ancestors [N][1][T][T], k [N][H][T][dk] in FP32, and the sums of
    log decays along each node's path [N][H][T][dk or 1] in 64 bits."""
    case = s["case"]
    M = _ancestors(s["parents"])
    k = s["k"].float().repeat_interleave(case["H"] // case["Hq"], 2).movedim(2, 1)
    g = s["log_alpha"].double().movedim(2, 1)
    g = g if g.dim() == 4 else g.unsqueeze(-1)
    return M.unsqueeze(1), k, M.double().unsqueeze(1) @ g


def _plain_verify(s):
    """All nodes at once: the products between nodes and their ancestors, the delta rule's triangular
    system, and the products with the stored state."""
    case = s["case"]
    H, T = case["H"], case["T"]
    vector, delta = case["mixer"] in ("gla", "kda"), case["mixer"] in ("gdn", "kda")
    M, k, c = _paths(s)
    q = s["q"].float().repeat_interleave(H // case["Hq"], 2).movedim(2, 1)
    v = s["v"].float().movedim(2, 1)
    S = _values(s).mT.contiguous()
    b = s["beta"].movedim(2, 1) if s["beta"] is not None else torch.ones_like(v[..., 0])
    if vector:
        G = (c.unsqueeze(3) - c.unsqueeze(2)).float().masked_fill(M.unsqueeze(-1) == 0, -math.inf).exp()
        A = (q.unsqueeze(3) * k.unsqueeze(2) * G).sum(-1)
        L = (k.unsqueeze(3) * k.unsqueeze(2) * G).sum(-1) if delta else None
    else:
        G = (c - c.mT).float().masked_fill(M == 0, -math.inf).exp()
        A = (q @ k.mT.contiguous()) * G
        L = (k @ k.mT.contiguous()) * G if delta else None
    e = c.float().exp()
    u = v
    if delta:
        u = _inverse(torch.tril(L, -1) * b.unsqueeze(-2), T) @ (v - (k * e) @ S)
    node = (s["parents"] >= -1)[:, None, :, None]
    w = (u * b.unsqueeze(-1)).masked_fill(~node, 0.0)
    o = ((q * e) @ S + A @ w).masked_fill(~node, 0.0)
    return [o.movedim(1, 2).to(s["v"].dtype), w.movedim(1, 2).contiguous()]


def _plain_accept(s):
    """The state behind the last accepted node, stored again."""
    case = s["case"]
    M, k, c = _paths(s)
    last = s["last"].long()
    at = last.clamp(min=0)
    N = torch.arange(case["N"], device=at.device)
    path = M[N, 0, at] * (last >= 0).unsqueeze(1)  # [N][T]
    end = c[N, :, at].unsqueeze(2)  # [N][H][1][dk or 1]
    f = (end - c).float().masked_fill(path[:, None, :, None] == 0, -math.inf).exp()
    w = s["writes"].movedim(2, 1)
    S = _values(s)
    new = S * end.float().exp() + w.mT.contiguous() @ (k * f)
    none = (last < 0)[:, None, None, None]
    if case["store"] == "f32":
        s["state"].copy_(torch.where(none, S, new))
        return [s["state"]]
    codes, scales = _quantized(new, 127.0, case["group"])
    codes = codes.view(torch.uint8).flatten(1)
    s["codes"].copy_(torch.where(none.flatten(1), s["codes"], codes))
    s["scales"].copy_(torch.where(none, s["scales"], scales))
    return [_int8_values(s["codes"], s["scales"], case)]


def _int8_values(codes, scales, case):
    """The values that INT8 codes stand for, as a model's own type holds them."""
    c = codes.view(torch.int8).view(scales.shape + (case["group"],))
    return c * scales.unsqueeze(-1).to(torch.bfloat16)


_EPS = 1e-5


def _plain_norm(s):
    case = s["case"]
    u = s["x"].float()
    if s["gate"] is not None:
        z = s["gate"].float()
        a = z / (1.0 + torch.exp(-z))
    if case["mode"] == "gate_first":
        u = u * a
    u = u.unflatten(-1, (case["groups"], case["width"]))
    if case["center"]:
        u = u - u.mean(-1, keepdim=True)
    h = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + _EPS)
    n = h.flatten(-2) * s["weight"] + s["bias"]
    if case["mode"] == "gate":
        n = n * a
    if case["mode"] == "activate":
        n = n / (1.0 + torch.exp(-n))
    return n.to(s["x"].dtype)


def _plain_linear(s):
    w = _signed(s["nibbles"]).float().unflatten(-1, (-1, s["case"]["group"])) * s["scales"].unsqueeze(-1)
    y = s["x"].float() @ w.flatten(-2).t()
    return (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype)


# ---- one pass ---------------------------------------------------------------------------------


def _norm_forward(s):
    if own:
        from bit_recurrent_state_amd import group_norm
        case = s["case"]
        return group_norm(s["x"], case["groups"], weight=s["weight"], bias=s["bias"], gate=s["gate"],
                          gate_first=case["mode"] == "gate_first", activate=case["mode"] == "activate",
                          center=case["center"], eps=_EPS)
    return _plain_norm(s)


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "norm_grad":
        y = _norm_forward(s)
        leaves = [s[n] for n in ("x", "gate", "weight", "bias") if s[n] is not None]
        return [y.detach()] + list(torch.autograd.grad(y, leaves, s["dy"]))
    with torch.no_grad():
        if op == "norm":
            return [_norm_forward(s)]
        if op == "linear":
            if own:
                from bit_recurrent_state_amd import linear4
                return [linear4(s["x"], s["weight"], s["bias"])]
            return [_plain_linear(s)]
        if op == "verify":
            if own:
                o, draft = s["handle"].verify(s["q"], s["k"], s["v"], s["log_alpha"], s["beta"],
                                              parents=s["parents"])
                return [o, draft.writes]
            return _plain_verify(s)
        if own:
            st = s["handle"]
            st.accept(s["draft"], s["last"])
            N, H, dv, dk, G = (case[n] for n in ("N", "H", "dv", "dk", "group"))
            if case["store"] == "f32":
                return [st.codes.view(N, H, dv, dk)]
            return [_int8_values(st.codes, st.scales.view(N, H, dv, dk // G), case)]
        return _plain_accept(s)


# ---- the definition in 64 bits ----------------------------------------------------------------


def _exact_state(case, s):
    if case["store"] == "f32":
        return s["state"].double()
    N, H, dv, dk, G = (case[n] for n in ("N", "H", "dv", "dk", "group"))
    n = _heads8(case)
    raw = s["codes"].to(torch.int16)
    eight, four = raw[:, :n * dv * dk], raw[:, n * dv * dk:]
    eight = eight - 256 * (eight > 127)
    low, high = four % 16, four // 16
    four = torch.stack([low - 16 * (low > 7), high - 16 * (high > 7)], 2).reshape(N, -1)
    c = torch.cat([eight, four], 1).double().view(N, H, dv, dk // G, G)
    return (c * s["scales"].double()[..., None]).view(N, H, dv, dk)


def _exact_verify(case, s):
    """Node by node: each from the state of its parent, which is kept."""
    N, T, H, dk, dv = (case[n] for n in ("N", "T", "H", "dk", "dv"))
    rep = H // case["Hq"]
    alpha = s["log_alpha"].double().exp()
    alpha = alpha if alpha.dim() == 4 else alpha[..., None]
    kept = torch.empty((T + 1, N, H, dv, dk), dtype=torch.float64, device="cuda")
    kept[0] = _exact_state(case, s)
    rows = torch.arange(N, device="cuda")
    o, writes = [], []
    for t in range(T):
        p = s["parents"][:, t].long()
        live = (p >= -1).double()[:, None, None]
        k = s["k"][:, t].double().repeat_interleave(rep, 1)
        q = s["q"][:, t].double().repeat_interleave(rep, 1)
        S = kept[(p + 1).clamp(min=0), rows] * alpha[:, t, :, None, :]
        w = s["v"][:, t].double()
        if case["mixer"] in ("gdn", "kda"):
            w = w - (S * k[:, :, None]).sum(-1)
        if s["beta"] is not None:
            w = w * s["beta"][:, t].double()[..., None]
        S = S + w[..., None] * k[:, :, None]
        kept[t + 1] = S
        o.append((S * q[:, :, None]).sum(-1) * live)
        writes.append(w * live)
    return [torch.stack(o, 1), torch.stack(writes, 1)]


def _exact_accept(case, s):
    """The path is walked from its start, token by token."""
    N, T, H, dk = (case[n] for n in ("N", "T", "H", "dk"))
    old = _exact_state(case, s)
    S = old.clone()
    alpha = s["log_alpha"].double().exp()
    alpha = alpha if alpha.dim() == 4 else alpha[..., None]
    parents, last = s["parents"].tolist(), s["last"].tolist()
    on = torch.zeros((N, T), dtype=torch.bool)
    for n in range(N):
        t = last[n]
        while t >= 0:
            on[n, t] = True
            t = parents[n][t]
    on = on.cuda()
    for t in range(T):
        k = s["k"][:, t].double().repeat_interleave(H // case["Hq"], 1)
        step = S * alpha[:, t, :, None, :] + s["writes"][:, t].double()[..., None] * k[:, :, None]
        S = torch.where(on[:, t, None, None, None], step, S)
    if case["store"] == "f32":
        return [S]
    G = case["group"]
    x = S.view(S.shape[:3] + (dk // G, G))
    m = x.abs().amax(-1, keepdim=True)
    x = torch.round(x * 127.0 / m) * (m / 127.0)
    x = torch.where(on.any(1)[:, None, None, None, None], x, old.view(x.shape))
    return [x]


def _exact_norm(case, s):
    """The forward and its gradients written out by hand."""
    shape = (case["rows"], case["groups"], case["width"])
    x = s["x"].detach().double().view(shape)
    w, b = (s[n].detach().double().view(shape[1:]) for n in ("weight", "bias"))
    mode, D = case["mode"], case["width"]
    z = s["gate"].detach().double().view(shape) if s["gate"] is not None else None
    if z is not None:
        sg = torch.sigmoid(z)
        a, da = z * sg, sg + z * sg * (1.0 - sg)
    u = x * a if mode == "gate_first" else x
    if case["center"]:
        u = u - u.sum(-1, keepdim=True) / D
    r = 1.0 / torch.sqrt((u * u).sum(-1, keepdim=True) / D + _EPS)
    h = u * r
    n = h * w + b
    sn = torch.sigmoid(n)
    y = n * a if mode == "gate" else n * sn if mode == "activate" else n
    flat = (case["rows"], case["groups"] * case["width"])
    if case["op"] == "norm":
        return [y.view(flat)]
    dy = s["dy"].double().view(shape)
    dn = dy * a if mode == "gate" else dy * (sn + n * sn * (1.0 - sn)) if mode == "activate" else dy
    dh = dn * w
    du = dh - h * (dh * h).sum(-1, keepdim=True) / D
    if case["center"]:
        du = du - dh.sum(-1, keepdim=True) / D
    du = du * r
    grads = [du * a if mode == "gate_first" else du]
    if mode == "gate":
        grads.append(dy * n * da)
    if mode == "gate_first":
        grads.append(du * x * da)
    return [y.view(flat)] + [d.reshape(flat) for d in grads] + [(dn * h).sum(0).flatten(), dn.sum(0).flatten()]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(case, s)
    if case["op"] == "linear":
        c = s["codes"].double().view(case["outputs"], -1, case["group"])
        y = torch.matmul(s["x"].double(), (c * s["scales"].double()[..., None]).flatten(1).T)
        return [y if s["bias"] is None else y + s["bias"].double()]
    return (_exact_verify if case["op"] == "verify" else _exact_accept)(case, s)


# ---- the work ---------------------------------------------------------------------------------


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "linear":
        M, K, O, G = (case[n] for n in ("rows", "inputs", "outputs", "group"))
        return {"bytes": O * K // 2 + O * K // G * 4 + M * (K + O) * size + 4 * O * case["bias"],
                "flops": 2 * M * K * O}
    if case["op"] in ("norm", "norm_grad"):
        e = case["rows"] * case["groups"] * case["width"]
        gate = case["mode"] in ("gate", "gate_first")
        streams, flops = 2 + gate, e * (8 + 4 * (case["mode"] != "plain"))
        if case["op"] == "norm_grad":  # dy is read, the gradients of x and the gate written
            streams, flops = streams + 2 + gate, 3 * flops
        return {"bytes": e * size * streams, "flops": flops}
    N, T, H, Hq, dk, dv = (case[n] for n in ("N", "T", "H", "Hq", "dk", "dv"))
    vector, delta = case["mixer"] in ("gla", "kda"), case["mixer"] in ("gdn", "kda")
    values, n = dv * dk, _heads8(case)
    state = 4 * H * values
    if case["store"] != "f32":
        state = n * values + (H - n) * values // 2 + 4 * H * values // case["group"]
    gates = 4 * H * ((dk if vector else 1) + (case["mixer"] != "gla"))
    if case["op"] == "verify":
        # q, k, v and o, the writes; the state is read
        token = (2 * Hq * dk + 2 * H * dv) * size + gates + 4 * H * dv
        nodes = N * T if case["shape"] != "ragged" else T + (N - 1) * T // 2
        flops = nodes * H * (2 * values * (1 + delta) + 4 * (dk + dv) * (1 + delta))
        return {"bytes": N * state + nodes * token, "flops": flops}
    # about a quarter of a tree's nodes lie on a path, half of a chain's: k, the gates and the writes of these
    nodes = N * max(1, T // (2 if case["shape"] == "chain" else 4))
    return {"bytes": 2 * N * state + nodes * (Hq * dk * size + gates + 4 * H * dv),
            "flops": nodes * H * 2 * values + N * H * values}
