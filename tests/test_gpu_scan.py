"""The scan and its gradients against the recurrence in 64 bits (GPU)."""

import pytest
import torch

from scan_reference import GDN, GLA, KDA, MIXERS, SCALAR, inputs, rel, scan64, tolerance

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = ("q", "k", "v", "log_alpha", "beta", "initial_state")


def call(x, mixer, **kw):
    from bit_recurrent_state_amd import scan
    return scan(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], mixer=mixer,
                initial_state=x["initial_state"], offsets=kw.pop("offsets", x.get("offsets")))


def gradients(x, mixer, do, dS):
    leaves = {n: x[n].detach().clone().requires_grad_(True) for n in NAMES if x[n] is not None}
    o, S = call({**x, **leaves}, mixer)
    return o, S, dict(zip(leaves, torch.autograd.grad((o, S), list(leaves.values()), (do, dS))))


def check(x, mixer, N, grad=True):
    o64, S64, leaf = scan64(x, mixer, N, grad)
    dt = x["v"].dtype
    if not grad:
        with torch.no_grad():
            o, S = call(x, mixer)
    else:
        g = torch.Generator().manual_seed(5)
        do = torch.randn(x["v"].shape, generator=g).to(dt).cuda()
        dS = (0.1 * torch.randn(S64.shape, generator=g)).cuda()
        o, S, got = gradients(x, mixer, do, dS)
        want = torch.autograd.grad((o64, S64), [leaf[n] for n in got], (do.double(), dS.double()),
                                   allow_unused=True)
        want = [torch.zeros_like(leaf[n]) if w is None else w for n, w in zip(got, want)]
        for (n, a), b in zip(got.items(), want):
            assert a.shape == x[n].shape and a.dtype == x[n].dtype
            assert rel(a, b) <= tolerance(a.dtype, True), n
    assert o.shape == x["v"].shape and o.dtype == dt and S.dtype == torch.float32
    assert rel(o, o64) <= tolerance(dt, False)
    assert rel(S, S64) <= tolerance(torch.float32, False)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,H,Hq", [(64, 64, 2, 2), (128, 128, 2, 1), (256, 40, 1, 1),
                                        (128, 1, 3, 1), (64, 200, 2, 2)])
def test_shapes_and_types(mixer, dtype, dk, dv, H, Hq):
    """Lengths 0, 1, around the token-by-token limit and around a chunk."""
    m = MIXERS[mixer]
    lens = [65, 0, 1, 8, 9, 64]
    check(inputs(m, len(lens), lens, H, Hq, dk, dv, TYPES[dtype], "cuda"), m, len(lens))


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("lens", [[300], [128, 127], [0, 0], [1] * 70, [3, 190, 2]])
def test_lengths(mixer, lens):
    m = MIXERS[mixer]
    check(inputs(m, len(lens), lens, 2, 2, 64, 48, torch.bfloat16, "cuda", state=len(lens) != 2),
          m, len(lens))


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("gate", [0.0, 20.0, 300.0])
def test_gates(mixer, gate):
    """No decay at all, and decays that leave almost nothing of a chunk (the sums of their
    logarithms pass 8, 88 and 1000 within one)."""
    m = MIXERS[mixer]
    check(inputs(m, 2, [150, 20], 2, 2, 128, 64, torch.float32, "cuda", gate=gate), m, 2)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("lens", [[100], [5]])
def test_dropped_state(mixer, lens):
    """A decay of minus infinity starts anew: what was before does not matter any more."""
    m = MIXERS[mixer]
    x = inputs(m, 1, lens, 2, 2, 64, 16, torch.float32, "cuda")
    cut = lens[0] * 3 // 5
    x["log_alpha"][cut] = -float("inf")
    with torch.no_grad():
        o, S = call(x, m)
        y = dict(x, initial_state=torch.zeros_like(x["initial_state"]))
        for n in ("q", "k", "v", "log_alpha", "beta"):
            y[n] = None if x[n] is None else x[n][cut:].contiguous()
        y["offsets"] = torch.tensor([0, lens[0] - cut], device="cuda")
        o2, S2 = call(y, m)
    assert rel(o[cut:], o2) <= 2 * tolerance(torch.float32, False)
    assert rel(S, S2) <= 2 * tolerance(torch.float32, False)


@pytest.mark.parametrize("mixer", ["gdn", "scalar"])
def test_no_write_weight(mixer):
    """beta = 0 (nothing is written) in some tokens and in all of a sequence."""
    m = MIXERS[mixer]
    x = inputs(m, 2, [70, 30], 2, 2, 64, 32, torch.float32, "cuda")
    x["beta"][::3] = 0.0
    x["beta"][70:] = 0.0
    check(x, m, 2)


@pytest.mark.parametrize("mixer", MIXERS)
def test_rows_of_no_sequence(mixer):
    """Rows before the first and behind the last sequence: poison there changes nothing, outputs
    and gradients there stay zero (scan) or as they were (qstate_scan)."""
    from bit_recurrent_state_amd import ScanConfig, qstate_scan
    m = MIXERS[mixer]
    x = inputs(m, 2, [70, 6], 2, 2, 64, 32, torch.bfloat16, "cuda", gap=3)
    for n in ("q", "k", "v", "log_alpha", "beta"):
        if x[n] is not None:
            x[n][:3] = float("nan")
            x[n][-3:] = float("nan")
    do = torch.randn(x["v"].shape, device="cuda").bfloat16()
    dS = torch.randn(2, 2, 32, 64, device="cuda")
    o, S, g = gradients(x, m, do, dS)
    inner = {n: t if t is None or n in ("offsets", "initial_state") else t[3:-3].contiguous()
             for n, t in x.items()}
    inner["offsets"] = x["offsets"] - 3
    o2, S2, g2 = gradients(inner, m, do[3:-3], dS)
    assert torch.equal(o[3:-3], o2) and torch.equal(S, S2)
    assert not o[:3].any() and not o[-3:].any()
    for n in g:
        if n == "initial_state":
            assert torch.equal(g[n], g2[n])
        else:
            assert torch.equal(g[n][3:-3], g2[n]), n
            assert not g[n][:3].any() and not g[n][-3:].any(), n
    c = ScanConfig(2, 2, 64, 32, 82, mixer=m, dtype=torch.bfloat16)
    o3 = torch.full_like(x["v"], 7.0)
    qstate_scan(c, x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["offsets"],
                x["initial_state"], o3)
    assert torch.equal(o3[3:-3], o2) and (o3[:3] == 7).all() and (o3[-3:] == 7).all()


@pytest.mark.parametrize("mixer", MIXERS)
def test_nan_stays_in_its_head(mixer):
    """A NaN spoils its sequence and head, and nothing else; nothing before its chunk."""
    m = MIXERS[mixer]
    x = inputs(m, 3, [80, 140, 40], 2, 2, 64, 32, torch.float32, "cuda")
    with torch.no_grad():
        o, S = call(x, m)
        for n in ("q", "k", "v", "log_alpha"):
            y = dict(x, **{n: x[n].clone()})
            y[n][80 + 100, 1] = float("nan")  # second sequence, second head, second chunk
            o2, S2 = call(y, m)
            same = torch.ones_like(o, dtype=torch.bool)
            same[80 + 64:80 + 140, 1] = False
            assert torch.equal(o2[same], o[same]), n
            assert o2[80 + 100, 1].isnan().any(), n
            keep = torch.ones(3, 2, dtype=torch.bool)
            keep[1, 1] = False
            assert torch.equal(S2[keep.cuda()], S[keep.cuda()]), n


def test_views_strides_and_dense_batches():
    """q, k, v as parts of one projection; dense [N, T]; transposed heads; odd row strides."""
    m, N, T, H, Hq, dk, dv = GDN, 2, 75, 4, 2, 64, 32
    for dtype in (torch.bfloat16, torch.float32):
        x = inputs(m, N, [T] * N, H, Hq, dk, dv, dtype, "cuda")
        with torch.no_grad():
            o, S = call(x, m)
            for pad in (0, 8, 3):  # 3: rows off any 16-byte boundary
                parts = [x["q"].flatten(1), x["k"].flatten(1), x["v"].flatten(1)]
                wide = torch.cat(parts + [parts[0][:, :pad]], 1)
                q, k, v = (t.view(N * T, h, d) for t, h, d in zip(
                    wide.split([Hq * dk, Hq * dk, H * dv] + ([pad] if pad else []), 1),
                    (Hq, Hq, H), (dk, dk, dv)))
                o2, S2 = call(dict(x, q=q, k=k, v=v), m)
                assert rel(o2, o) <= tolerance(dtype, False) and rel(S2, S) <= tolerance(torch.float32, False)
            d = {n: x[n].view((N, T) + x[n].shape[1:]) for n in ("q", "k", "v", "log_alpha", "beta")}
            o3, S3 = call(dict(x, **d), m, offsets=None)
            assert torch.equal(o3.flatten(0, 1), o) and torch.equal(S3, S)
            t = {n: d[n].transpose(1, 2).contiguous().transpose(1, 2) for n in ("q", "k", "v")}
            o4, S4 = call(dict(x, **{**d, **t}), m, offsets=None)
            assert torch.equal(o4, o3) and torch.equal(S4, S)


@pytest.mark.parametrize("mixer", MIXERS)
def test_pieces_join(mixer):
    """A sequence in pieces of any length, each from the state the last one left."""
    m = MIXERS[mixer]
    x = inputs(m, 1, [200], 2, 2, 64, 32, torch.float32, "cuda")
    with torch.no_grad():
        o, S = call(x, m)
        s, outs, at = x["initial_state"], [], 0
        for n in (1, 7, 64, 0, 9, 119):
            part = {k: None if x[k] is None else x[k][at:at + n].contiguous()
                    for k in ("q", "k", "v", "log_alpha", "beta")}
            off = torch.tensor([0, n], device="cuda")
            y, s = call(dict(part, initial_state=s, offsets=off), m)
            outs.append(y)
            at += n
    assert rel(torch.cat(outs), o) <= 2 * tolerance(torch.float32, False)
    assert rel(s, S) <= 2 * tolerance(torch.float32, False)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("T", [1, 100])
def test_state_in_place_and_optional_outputs(mixer, T):
    from bit_recurrent_state_amd import ScanConfig, qstate_scan
    m = MIXERS[mixer]
    x = inputs(m, 3, [T] * 3, 2, 1, 128, 40, torch.bfloat16, "cuda")
    c = ScanConfig(3, 2, 128, 40, 3 * T, 1, m, torch.bfloat16)
    args = (x["q"], x["k"], x["v"], x["log_alpha"], x["beta"])
    for off in (x["offsets"], None):
        o, S = torch.empty_like(x["v"]), torch.empty_like(x["initial_state"])
        qstate_scan(c, *args, off, x["initial_state"], o, S)
        S2, S3, o2 = x["initial_state"].clone(), torch.empty_like(S), torch.empty_like(o)
        qstate_scan(c, *args, off, S2, None, S2)
        qstate_scan(c, *args, off, x["initial_state"], o2, None)
        qstate_scan(c, *args, off, x["initial_state"], None, S3)
        assert torch.equal(S2, S) and torch.equal(S3, S) and torch.equal(o2, o)


def test_bad_offsets_stay_inside():
    """Offsets that break the rule give some result, and nothing outside the arrays is touched."""
    m = GDN
    x = inputs(m, 3, [70, 70, 4], 2, 2, 64, 32, torch.bfloat16, "cuda")
    guard = torch.full((3 * 144, 2, 32), 5.0, device="cuda", dtype=torch.bfloat16)
    from bit_recurrent_state_amd import ScanConfig, qstate_scan
    c = ScanConfig(3, 2, 64, 32, 144, mixer=m, dtype=torch.bfloat16)
    for bad in ([0, 200, 100, 50], [-5, 10, 1 << 40, 3], [144, 0, 144, 0], [7, 7, 7, 900]):
        off = torch.tensor(bad, device="cuda")
        qstate_scan(c, x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], off, None, guard[144:288])
        assert (guard[:144] == 5).all() and (guard[288:] == 5).all()


@pytest.mark.parametrize("mixer", MIXERS)
def test_same_call_same_bits(mixer):
    m = MIXERS[mixer]
    x = inputs(m, 4, [130, 64, 7, 333], 4, 2, 128, 64, torch.bfloat16, "cuda")
    do, dS = torch.randn_like(x["v"]), torch.randn(4, 4, 64, 128, device="cuda")
    first = gradients(x, m, do, dS)
    for _ in range(3):
        torch.empty(1 << 26, device="cuda").fill_(float("nan"))  # what workspaces may hold
        again = gradients(x, m, do, dS)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert all(torch.equal(first[2][n], again[2][n]) for n in first[2])


def test_two_streams_and_graphs():
    """Calls on two streams at once; forward and backward captured into a graph, replayed with
    eager work between, on new inputs."""
    from bit_recurrent_state_amd import ScanConfig, qstate_scan, qstate_scan_backward, qstate_scan_workspace
    m, lens = KDA, [100, 3, 65]
    xs = [inputs(m, 3, lens, 2, 2, 64, 32, torch.bfloat16, "cuda", seed=s) for s in range(3)]
    with torch.no_grad():
        want = [call(x, m) for x in xs]
        side = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(5):
            got = []
            for s, x in zip(side, xs):
                with torch.cuda.stream(s):
                    got.append(call(x, m))
            torch.cuda.synchronize()
            for (o, S), (o2, S2) in zip(want, got):
                assert torch.equal(o, o2) and torch.equal(S, S2)
    T = sum(lens)
    c = ScanConfig(3, 2, 64, 32, T, mixer=m, dtype=torch.bfloat16)
    x = {n: t.clone() for n, t in xs[0].items()}
    do, dS = torch.randn(T, 2, 32, device="cuda").bfloat16(), torch.randn(3, 2, 32, 64, device="cuda")
    o, S = torch.empty_like(x["v"]), torch.empty_like(dS)
    out = [torch.empty_like(x[n]) for n in NAMES]
    ws = [torch.empty(qstate_scan_workspace(c, b), dtype=torch.uint8, device="cuda") for b in (False, True)]
    args = [x[n] for n in ("q", "k", "v", "log_alpha", "beta", "offsets", "initial_state")]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        qstate_scan(c, *args, o, S, ws[0])
        qstate_scan_backward(c, *args, do, dS, *out, workspace=ws[1])
    for i in (1, 2, 0, 2):
        for n in NAMES:
            x[n].copy_(xs[i][n])
        graph.replay()
        torch.cuda.synchronize()
        o2, S2, g = gradients(xs[i], m, do, dS)
        assert torch.equal(o, o2) and torch.equal(S, S2)
        assert all(torch.equal(a, g[n]) for a, n in zip(out, NAMES))


def test_partial_gradients():
    """Losses of one output only, and leaves that want none."""
    m = GDN
    x = inputs(m, 2, [70, 20], 2, 2, 64, 32, torch.float32, "cuda")
    do, dS = torch.randn_like(x["v"]), torch.randn(2, 2, 32, 64, device="cuda")
    for a, b in ((do, torch.zeros_like(dS)), (torch.zeros_like(do), dS)):
        _, _, want = gradients(x, m, a, b)
        leaves = {n: x[n].detach().clone().requires_grad_(n in ("v", "log_alpha")) for n in NAMES}
        o, S = call({**x, **leaves}, m)
        (o * a).sum().backward() if a is do else (S * b).sum().backward()
        for n in NAMES:
            if n in ("v", "log_alpha"):
                assert torch.equal(leaves[n].grad, want[n])
            else:
                assert leaves[n].grad is None


def test_refusals():
    from bit_recurrent_state_amd import scan
    x = inputs(GDN, 1, [4], 4, 2, 64, 8, torch.float32, "cuda")
    ok = dict(q=x["q"], k=x["k"], v=x["v"], log_alpha=x["log_alpha"], beta=x["beta"], mixer=GDN,
              offsets=x["offsets"], initial_state=x["initial_state"])
    scan(**ok)
    for change in (dict(mixer=5), dict(mixer=GLA), dict(q=x["q"].bfloat16()), dict(q=x["q"][:3]),
                   dict(k=x["k"][:, :1]), dict(beta=x["beta"].double()), dict(beta=x["beta"][:, :2]),
                   dict(log_alpha=x["log_alpha"].bfloat16()), dict(offsets=x["offsets"].int()),
                   dict(offsets=x["offsets"][:1]), dict(initial_state=x["initial_state"][:, :2]),
                   dict(offsets=None), dict(v=x["v"].double()),
                   dict(q=x["q"][:, [0, 1, 1]], k=x["k"][:, [0, 1, 1]])):
        with pytest.raises((ValueError, TypeError)):
            scan(**{**ok, **change})
    with pytest.raises(TypeError):
        scan(**{**ok, "beta": None})
    from bit_recurrent_state_amd._lib import QStateError
    y = inputs(GDN, 1, [4], 2, 2, 96, 8, torch.float32, "cuda")
    with pytest.raises(QStateError):
        call(y, GDN)


@pytest.mark.parametrize("fp32", [True, False])
@pytest.mark.parametrize("mixer", MIXERS)
def test_prefill_then_decode(mixer, fp32):
    """A prompt, then steps token by token, with the readout's norm: against the whole sequence's
    scan; with an INT8 state, against the same steps from the prompt's state."""
    from bit_recurrent_state_amd import Config, QState, ReadoutNorm, block_norm
    m, B, H, dk, dv, T, n = MIXERS[mixer], 2, 3, 64, 32, 40, 6
    x = inputs(m, B, [T + n] * B, H, H, dk, dv, torch.float32, "cuda", state=False)
    x = {k: None if t is None else t.view((B, T + n) + t.shape[1:]) if k != "offsets" else t
         for k, t in x.items()}
    gate = torch.randn(B, T + n, H, dv, device="cuda")
    weight = torch.randn(H, dv, device="cuda")
    names = ("q", "k", "v", "log_alpha", "beta")
    head = {k: None if x[k] is None else x[k][:, :T].contiguous() for k in names}
    st = QState(Config(B, H, dk, dv, 32, m, fp32_state=fp32))
    o = st.prefill(*(head[k] for k in names), norm=ReadoutNorm(weight, gate[:, :T].contiguous()))
    with torch.no_grad():
        full, end = call(dict(x, initial_state=None), m, offsets=None)
        want = block_norm(full, weight=weight, gate=gate)
        assert rel(o, want[:, :T]) <= 4 * tolerance(torch.float32, False)
        if not fp32:  # the stored state stands for the scan's, to half a step of each group
            _, S = call(dict(head, initial_state=None), m, offsets=None)
            back = torch.empty_like(S)
            st.store_fp32(back)
            step = S.view(B, H, dv, dk // 32, 32).abs().amax(-1, keepdim=True) / 127
            assert ((back - S).view_as(S.view(B, H, dv, dk // 32, 32)).abs() <= step * 0.5001).all()
            assert st.step_counter == 1
    for t in range(T, T + n):
        one = {k: None if x[k] is None else x[k][:, t].contiguous() for k in names}
        y = torch.empty(B, H, dv, device="cuda")
        st.step(one["q"], one["k"], one["v"], one["log_alpha"].exp(), one["beta"], y,
                norm=ReadoutNorm(weight, gate[:, t].contiguous()))
        if fp32:
            assert rel(y, want[:, t]) <= 8 * tolerance(torch.float32, False)
    if fp32:
        S = torch.empty(B, H, dv, dk, device="cuda")
        st.store_fp32(S)
        assert rel(S, end) <= 4 * tolerance(torch.float32, False)
    st.close()


def test_training_chain():
    """Scan, norm, gate, residual and the next norm in one graph: gradients against 64 bits."""
    from bit_recurrent_state_amd import block_norm
    from scan_reference import norm64
    m, N, lens, H, dv = GDN, 2, [70, 33], 2, 64
    x = inputs(m, N, lens, H, H, 64, dv, torch.float32, "cuda")
    T = sum(lens)
    g = torch.Generator().manual_seed(3)
    gate, res = (torch.randn(T, H * dv, generator=g).cuda() for _ in range(2))
    w, sc, nw = ((1 + 0.1 * torch.randn(d, generator=g)).cuda() for d in (dv, H * dv, H * dv))
    leaves = {n: x[n].clone().requires_grad_(True) for n in NAMES}
    extra = [t.clone().requires_grad_(True) for t in (gate, res, w, sc, nw)]
    o, S = call({**x, **leaves}, m)
    y = block_norm(o, weight=extra[2])
    r, h = block_norm(y.reshape(T, H * dv), gate=extra[0], residual=extra[1], scale=extra[3],
                      next_weight=extra[4])
    got = torch.autograd.grad((r.sin().sum() + (h * r).sum() + S.sum()), list(leaves.values()) + extra)
    o64, S64, leaf = scan64(x, m, N, True)
    e64 = [t.double().requires_grad_(True) for t in (gate, res, w, sc, nw)]
    (y64,) = norm64(o64, e64[2], None, None, None, None, 1e-6, 0)
    r64, h64 = norm64(y64.reshape(T, H * dv), None, e64[0], e64[1], e64[3], e64[4], 1e-6, 0)
    want = torch.autograd.grad((r64.sin().sum() + (h64 * r64).sum() + S64.sum()),
                               [leaf[n] for n in NAMES] + e64)
    for i, (a, b) in enumerate(zip(got, want)):
        assert rel(a, b) <= 4 * tolerance(torch.float32, True), i


@pytest.mark.parametrize("handle", [False, True])
def test_own_workspace_belongs_to_the_stream(handle):
    """A call on a stream that is not the current one takes its workspace from that stream's
    memory, so that later work of the current stream cannot be given it while the call runs."""
    from bit_recurrent_state_amd import NormConfig, ScanConfig, qstate_norm_backward, qstate_scan
    from bit_recurrent_state_amd import norm, sequence
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    x = inputs(GDN, 2, [40, 9], 2, 2, 64, 32, torch.float32, "cuda")
    o, want = torch.empty_like(x["v"]), call(x, GDN)[0]
    g = torch.randn(30, 1, 64, device="cuda")
    dw, r = torch.empty(64, device="cuda"), 1 / (g.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()
    torch.cuda.synchronize()
    made = []

    def watch(module, name):
        real = getattr(module, name)

        def f(*args, **kw):
            made.append(real(*args, **kw))
            return made[-1]
        return real, f

    for module in (sequence, norm):
        real, f = watch(module, "_own_workspace")
        module._own_workspace = f
        try:
            if module is sequence:
                c = ScanConfig(2, 2, 64, 32, 49)
                qstate_scan(c, x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["offsets"],
                            x["initial_state"], o, stream=stream)
            else:
                qstate_norm_backward(NormConfig(30, 1, 64), g, dr=g, dweight=dw, stream=stream)
        finally:
            module._own_workspace = real
    side.synchronize()
    for _, (at, n) in made:
        segments = [s for s in torch.cuda.memory_snapshot()
                    if s["address"] <= at < s["address"] + s["total_size"]]
        assert [s["stream"] for s in segments] == [side.cuda_stream]
    assert len(made) == 2 and torch.equal(o, want)
    assert rel(dw, (g.double() ** 2 * r).sum((0, 1))) <= 30 * 2 ** -22


def test_rows_far_apart():
    """Rows of q, k and v that lie farther apart than the kernels take are copied."""
    x = inputs(GDN, 1, [3], 1, 1, 64, 16, torch.bfloat16, "cuda")
    want = call(x, GDN)
    far = (1 << 22) + 8
    wide = torch.zeros(2 * far + 256, dtype=torch.bfloat16, device="cuda")
    parts = {}
    for i, n in enumerate(("q", "k", "v")):
        w = x[n].shape[2]
        parts[n] = wide.as_strided((3, 1, w), (far, w, 1), 80 * i)
        parts[n].copy_(x[n])
    got = call({**x, **parts}, GDN)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_readout_norm_refused_before_the_step():
    """A readout norm that does not fit is refused before the state changes."""
    from bit_recurrent_state_amd import Config, QState, ReadoutNorm
    cfg = Config(batch=2, heads=2, dk=64, dv=32, group=32, mixer=GDN)
    st = QState(cfg)
    g = torch.Generator().manual_seed(3)
    f32 = lambda *s: torch.randn(*s, generator=g).cuda()
    st.load_fp32(f32(2, 2, 32, 64))
    before = torch.empty(2, 2, 32, 64, device="cuda")
    st.store_fp32(before)
    q, k, v, o = f32(2, 2, 64), f32(2, 2, 64), f32(2, 2, 32), f32(2, 2, 32)
    alpha, beta = torch.full((2, 2), 0.9, device="cuda"), torch.full((2, 2), 0.5, device="cuda")
    bad = [ReadoutNorm(weight=f32(31)), ReadoutNorm(gate=f32(2, 2, 31)), ReadoutNorm(eps=0.0),
           ReadoutNorm(act=7), ReadoutNorm(weight=f32(3, 32)), ReadoutNorm(gate=v.bfloat16())]
    from bit_recurrent_state_amd._lib import QStateError
    for norm in bad:
        with pytest.raises((ValueError, TypeError, QStateError)):
            st.step(q, k, v, alpha, beta, o, norm=norm)
        with pytest.raises((ValueError, TypeError, QStateError)):
            st.prefill(q[:, None], k[:, None], v[:, None], alpha[:, None].log(), beta[:, None], norm=norm)
    with pytest.raises(ValueError):
        st.step(q, k, v, alpha, beta, None, norm=ReadoutNorm())
    after = torch.empty_like(before)
    st.store_fp32(after)
    assert torch.equal(before, after)


@pytest.mark.parametrize("decay", [-0.05, -50.0])
@pytest.mark.parametrize("mixer", MIXERS)
def test_single_tokens_without_a_state(mixer, decay):
    """No gate lies between a token and itself: without a state its gradient is exactly zero."""
    m, lens = MIXERS[mixer], [1, 1, 0, 1]
    x = inputs(m, 4, lens, 2, 1, 128, 40, torch.bfloat16, "cuda", state=False)
    x["log_alpha"].fill_(decay)
    g = torch.Generator().manual_seed(9)
    do = torch.randn(x["v"].shape, generator=g).bfloat16().cuda()
    dS = torch.randn(4, 2, 40, 128, generator=g).cuda()
    _, _, got = gradients(x, m, do, dS)
    assert not got["log_alpha"].any()
    assert all(got[n].any() for n in ("q", "k", "v"))
    check(x, m, 4)


@pytest.mark.parametrize("mixer", MIXERS)
def test_rows_beyond_32_bits(mixer):
    """A sequence behind 2^31 elements of v: the same bits as alone (about 60 GB)."""
    from bit_recurrent_state_amd import ScanConfig, qstate_scan, qstate_scan_backward
    m, H, dk, dv, n = MIXERS[mixer], 16, 64, 2048, 100
    before = -(-(1 << 31) // (H * dv)) // 64 * 64 + 64  # on a chunk's boundary, as alone
    x = inputs(m, 1, [n], H, H, dk, dv, torch.bfloat16, "cuda")
    g = torch.Generator().manual_seed(2)
    do = torch.randn(x["v"].shape, generator=g).bfloat16().cuda()
    dS = torch.randn(1, H, dv, dk, generator=g).cuda()
    o, S, want = gradients(x, m, do, dS)
    big = {}
    for name in ("q", "k", "v", "log_alpha", "beta"):
        if x[name] is not None:
            big[name] = torch.empty((before + n,) + x[name].shape[1:], dtype=x[name].dtype, device="cuda")
            big[name][before:] = x[name]
    args = [big.get(k) for k in ("q", "k", "v", "log_alpha", "beta")]
    args += [x["offsets"] + before, x["initial_state"]]
    c = ScanConfig(1, H, dk, dv, before + n, mixer=m, dtype=torch.bfloat16)
    o2, S2 = torch.empty_like(big["v"]), torch.empty_like(S)
    qstate_scan(c, *args, o2, S2)
    assert torch.equal(o2[before:], o) and torch.equal(S2, S)
    o2[before:] = do
    out = {k: torch.empty_like(v) for k, v in big.items()}
    out["initial_state"] = torch.empty_like(S)
    qstate_scan_backward(c, *args, o2, dS, *(out.get(k) for k in NAMES))
    for k, t in out.items():
        assert torch.equal(t if k == "initial_state" else t[before:], want[k]), k
    del args, big, out, o2
    torch.cuda.empty_cache()


def test_training_step_in_a_graph():
    """scan, block_norm and their gradients captured through autograd, over leaves that no eager
    pass has used; replayed on new inputs with eager work between."""
    from bit_recurrent_state_amd import block_norm
    m, lens = KDA, [70, 0, 30]
    xs = [inputs(m, 3, lens, 2, 1, 64, 32, torch.bfloat16, "cuda", seed=s) for s in range(3)]
    weight, gate = torch.rand(2, 32, device="cuda"), torch.randn_like(xs[0]["v"])
    dr, dS = torch.randn_like(xs[0]["v"]), torch.randn(3, 2, 32, 64, device="cuda")

    def step(x, leaves):
        o, S = call({**x, **leaves}, m)
        r = block_norm(o, weight=leaves["weight"], gate=gate)
        return [r, S, *torch.autograd.grad((r, S), list(leaves.values()), (dr, dS))]

    def leaves_of(x):
        leaves = {n: x[n].detach().clone().requires_grad_(True) for n in NAMES}
        return {**leaves, "weight": weight.clone().requires_grad_(True)}

    want = [[t.detach() for t in step(x, leaves_of(x))] for x in xs]
    leaves = leaves_of(xs[0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = [t.detach() for t in step(xs[0], leaves)]
    for i in (1, 0, 2, 1):
        with torch.no_grad():
            for n in NAMES:
                leaves[n].copy_(xs[i][n])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
        again = step(xs[i], leaves_of(xs[i]))
        assert all(torch.equal(a, b) for a, b in zip(again, want[i]))


def test_captured_backward_beside_an_eager_graph_is_refused(monkeypatch):
    """The same check in the operators, without a capture: it stands before any launch."""
    from bit_recurrent_state_amd import block_norm
    x = inputs(GDN, 1, [20], 1, 1, 64, 32, torch.float32, "cuda")
    leaves = {n: x[n].detach().clone().requires_grad_(True) for n in NAMES}
    w = torch.ones(32, device="cuda", requires_grad=True)
    o, _ = call({**x, **leaves}, GDN)
    eager = block_norm(o, weight=w)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        o2, _ = call({**x, **leaves}, GDN)
        y = block_norm(o2.detach(), weight=w)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
        for out, leaf in ((o2, leaves["q"]), (y, w)):
            with pytest.raises(RuntimeError, match="drop the results"):
                torch.autograd.grad(out.sum(), leaf, retain_graph=True)
        del eager, o
        torch.autograd.grad(o2.sum(), leaves["q"])
        torch.autograd.grad(y.sum(), w)
    torch.cuda.synchronize()


def _prefill_case():
    from bit_recurrent_state_amd import Config, QState
    B, H, dk, dv, T = 3, 4, 64, 32, 5
    st = QState(Config(B, H, dk, dv, 32, GDN, fp32_state=True))
    x = inputs(GDN, B, [T] * B, H, H, dk, dv, torch.float32, "cuda", state=False)
    p = [x[n].view((B, T) + x[n].shape[1:]) for n in ("q", "k", "v", "log_alpha", "beta")]
    S = torch.randn(B, H, dv, dk, device="cuda")
    st.load_fp32(S)
    return st, p, S, torch.rand(H, dv, device="cuda"), torch.randn(B, T, H, dv, device="cuda")


def test_readout_norm_shapes():
    """A weight or a gate of the right size and another shape is refused before the state changes; a
    gate may have o's shape or hold its values in a row."""
    from bit_recurrent_state_amd import ReadoutNorm
    st, p, S, w, G = _prefill_case()
    one = [t[:, 0].contiguous() for t in p]
    one[3] = one[3].exp()
    o = torch.empty_like(one[2])
    g = G[:, 0].contiguous()
    for norm in (ReadoutNorm(w.t().contiguous()), ReadoutNorm(gate=g.transpose(0, 1).contiguous()),
                 ReadoutNorm(gate=g.transpose(1, 2).contiguous())):
        with pytest.raises(ValueError):
            st.step(*one, o, norm=norm)
    for norm in (ReadoutNorm(w.t().contiguous()), ReadoutNorm(gate=G.transpose(0, 1).contiguous()),
                 ReadoutNorm(gate=G.transpose(1, 2).contiguous())):
        with pytest.raises(ValueError):
            st.prefill(*p, norm=norm)
    back = torch.empty_like(S)
    st.store_fp32(back)
    assert torch.equal(back, S)
    want = st.prefill(*p, norm=ReadoutNorm(w, G))
    st.load_fp32(S)
    assert torch.equal(st.prefill(*p, norm=ReadoutNorm(w, G.flatten(0, 1))), want)
    st.load_fp32(S)
    st.step(*one, o, norm=ReadoutNorm(w, g))
    st.load_fp32(S)
    o2 = torch.empty_like(o).view(-1)
    st.step(*one, o2, norm=ReadoutNorm(w, g.view(-1)))
    assert torch.equal(o2.view_as(o), o)
    st.close()


@pytest.mark.parametrize("handle", [False, True])
def test_prefill_on_another_stream(handle):
    from bit_recurrent_state_amd import ReadoutNorm
    st, p, S, w, G = _prefill_case()
    want = st.prefill(*p, norm=ReadoutNorm(w, G))
    end = torch.empty_like(S)
    st.store_fp32(end)
    st.load_fp32(S)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = []
    real = st.store_fp32
    st.store_fp32 = lambda *a, **kw: (seen.append(torch.cuda.current_stream()), real(*a, **kw))
    got = st.prefill(*p, norm=ReadoutNorm(w, G), stream=side.cuda_stream if handle else side)
    side.synchronize()
    back = torch.empty_like(S)
    real(back)
    assert torch.equal(got, want) and torch.equal(back, end)
    assert [s.cuda_stream for s in seen] == [side.cuda_stream]
    at = got.data_ptr()  # o lies in that stream's memory
    assert [s["stream"] for s in torch.cuda.memory_snapshot()
            if s["address"] <= at < s["address"] + s["total_size"]] == [side.cuda_stream]
    st.close()
