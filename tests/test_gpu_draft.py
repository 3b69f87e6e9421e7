"""Drafted tokens over the stored state against the recurrence in 64 bits (GPU)."""

import pytest
import torch

from draft_reference import (ACCEPT, GDN, GLA, KDA, MIXERS, SCALAR, VERIFY, accept64, inputs, node_mask,
                             tolerance, verify64)
from scan_reference import rel

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def handle(mixer, S, store="f32", group=32, rounding=0, **kw):
    """A handle that holds S, and the values it holds."""
    from bit_recurrent_state_amd import Config, QState
    N, H, dv, dk = S.shape
    bits = {"f32": None, "int8": [8] * H, "int4": [4] * H, "mix": [8 if h % 3 == 0 else 4 for h in range(H)]}
    if store == "channels":
        per = max(1, group // 16)
        kw["channel_bits"] = [[8 if (q // per + h) % 2 == 0 else 4 for q in range(dk // 16)]
                              for h in range(H)]
    else:
        kw["head_bits"] = bits[store]
    st = QState(Config(N, H, dk, dv, group, mixer, rounding, store == "f32", **kw))
    st.load_fp32(S)
    held = torch.empty_like(S)
    st.store_fp32(held)
    return st, held


def verify(st, x, **kw):
    return st.verify(x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], parents=x["parents"], **kw)


def lasts(x, seed=0):
    """A node of each sequence, -1 for some."""
    g = torch.Generator().manual_seed(seed)
    ok = node_mask(x["parents"])
    out = []
    for n in range(ok.shape[0]):
        at = ok[n].nonzero().flatten().tolist()
        pick = int(torch.randint(-1, len(at), (1,), generator=g)) if n else len(at) - 1
        out.append(at[pick] if pick >= 0 else -1)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def check(mixer, N, T, shape, H, Hq, dk, dv, dtype, store="f32", group=32, **kw):
    x, S = inputs(mixer, N, T, shape, H, Hq, dk, dv, dtype, "cuda", **kw)
    st, held = handle(mixer, S, store, group)
    before = st.codes.clone()
    o, draft = verify(st, x)
    assert torch.equal(st.codes, before)
    want, writes, states = verify64(x, held, mixer)
    assert o.dtype == dtype and o.shape == x["v"].shape
    none = ~node_mask(x["parents"]).to("cuda")
    assert not o[none].any() and not draft.writes[none].any()
    assert rel(o, want) <= tolerance(dtype)
    assert rel(draft.writes, writes) <= VERIFY
    last = lasts(x)
    step = st.step_counter
    st.accept(draft, last)
    assert st.step_counter == step + 1
    got = torch.empty_like(S)
    st.store_fp32(got)
    goal = accept64(x, held, states, last)
    kept = last < 0
    assert torch.equal(got[kept], held[kept])
    if store == "f32":
        assert rel(got, goal) <= ACCEPT + VERIFY
    else:  # half a code of its group's scale, and what the values themselves are off by
        r = {"int8": 127.0, "int4": 7.0, "mix": 7.0, "channels": 7.0}[store]
        big = goal.unflatten(-1, (-1, group)).abs().amax(-1, keepdim=True).expand(-1, -1, -1, -1, group)
        off = (got.double() - goal).abs()[~kept]
        slack = 0.5 / r * (1.0 + 2.0 ** -10) + (ACCEPT + VERIFY) * 16
        assert bool((off <= slack * big.flatten(-2)[~kept]).all())
    return st, x


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dk,dv,H,Hq", [(64, 64, 2, 2), (128, 128, 2, 1), (256, 40, 1, 1),
                                        (128, 1, 3, 1), (64, 201, 2, 2)])
def test_shapes_and_types(mixer, dtype, dk, dv, H, Hq):
    check(MIXERS[mixer], 3, 11, "tree", H, Hq, dk, dv, TYPES[dtype])


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("T,shape", [(1, "chain"), (2, "tree"), (16, "chain"), (17, "ragged"), (32, "tree"),
                                     (33, "chain"), (64, "tree"), (64, "chain"), (64, "ragged"),
                                     (5, "none")])
def test_trees(mixer, T, shape):
    check(MIXERS[mixer], 5, T, shape, 2, 2, 64, 48, torch.float32)
    check(MIXERS[mixer], 5, min(T, 32), shape, 1, 1, 256, 16, torch.bfloat16)


@pytest.mark.parametrize("mixer", ["gdn", "gla"])
@pytest.mark.parametrize("store", ["int8", "int4", "mix", "channels"])
@pytest.mark.parametrize("dk,group", [(64, 16), (64, 64), (128, 16), (128, 32), (128, 64), (128, 128),
                                      (256, 32), (256, 128)])
def test_stored_forms(mixer, store, dk, group):
    check(MIXERS[mixer], 2, 6, "tree", 4, 2, dk, 72, torch.float32, store, group)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("store", ["int8", "int4", "mix", "channels"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_stored_forms_of_16_bit_rows(mixer, store, dtype):
    """16-bit rows over quantized states, one to four tiles of nodes, one and two tiles of value columns."""
    for N, T, shape, Hq, dk, dv, group in ((3, 16, "tree", 1, 128, 128, 32), (2, 17, "ragged", 2, 64, 128, 16),
                                           (2, 33, "tree", 1, 128, 72, 64), (2, 64, "tree", 4, 64, 128, 32),
                                           (2, 64, "chain", 2, 128, 64, 128), (3, 48, "ragged", 1, 128, 40, 16),
                                           (2, 32, "tree", 2, 256, 72, 64), (2, 9, "tree", 1, 256, 128, 16)):
        check(MIXERS[mixer], N, T, shape, 4, Hq, dk, dv, TYPES[dtype], store, group)


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("gate", [0.0, 20.0, 300.0, 5000.0])
def test_gates(mixer, gate):
    """No decay at all, and decays that leave nothing of what was before."""
    check(MIXERS[mixer], 2, 40, "tree", 2, 2, 128, 32, torch.float32, gate=gate)
    check(MIXERS[mixer], 2, 9, "chain", 2, 2, 64, 32, torch.float32, "int8", gate=gate)


@pytest.mark.parametrize("mixer", MIXERS)
def test_dropped_state(mixer):
    """A log decay of minus infinity: nothing of the path before counts."""
    m = MIXERS[mixer]
    x, S = inputs(m, 2, 7, "chain", 2, 2, 64, 16, torch.float32, "cuda")
    x["log_alpha"][:, 4] = -float("inf")
    st, _ = handle(m, S)
    o, _ = verify(st, x)
    st2, _ = handle(m, torch.zeros_like(S))
    y = {n: None if t is None else t[:, 4:].contiguous() for n, t in x.items()}
    y["parents"] = None
    o2, _ = verify(st2, y)
    assert rel(o[:, 4:], o2) <= 2 * VERIFY


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("store", ["f32", "int4"])
def test_poison_in_rows_of_no_node(mixer, store):
    """NaN and infinities in padding, and rows that hang on it, change nothing."""
    m = MIXERS[mixer]
    x, S = inputs(m, 3, 21, "ragged", 2, 1, 64, 32, torch.bfloat16, "cuda", seed=3)
    x["parents"][1, 2] = -7
    x["parents"][1, 5] = 2  # hangs on padding
    x["parents"][0, 4] = 4  # on itself
    x["parents"][0, 6] = 30  # on no row
    st, _ = handle(m, S, store)
    o, draft = verify(st, x)
    none = ~node_mask(x["parents"]).to("cuda")
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "log_alpha", "beta"):
        if y[n] is not None:
            y[n][none] = float("nan") if n != "v" else float("inf")
    o2, draft2 = verify(st, y)
    assert torch.equal(o, o2) and torch.equal(draft.writes, draft2.writes)
    assert not o[none].any()
    st2, _ = handle(m, S, store)
    last = lasts(x)
    st.accept(draft, last)
    st2.accept(draft2, last)
    assert torch.equal(st.codes, st2.codes)


@pytest.mark.parametrize("mixer", MIXERS)
def test_nan_stays_in_its_head(mixer):
    m = MIXERS[mixer]
    x, S = inputs(m, 3, 20, "tree", 2, 2, 64, 32, torch.float32, "cuda")
    st, _ = handle(m, S, "int8")
    o, d = verify(st, x)
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["v"][1, 5, 1, 3] = float("nan")
    o2, d2 = verify(st, y)
    assert torch.isnan(o2[1, 5, 1, 3])
    o2[1, :, 1] = o[1, :, 1]
    assert torch.equal(o2, o)
    last = torch.full((3,), 5, dtype=torch.int32, device="cuda")
    keep = st.codes.clone()
    st.accept(d, last)
    good = st.codes.view(3, 2, 32, 64).clone()
    st.codes.copy_(keep)
    st2, _ = handle(m, S, "int8")
    st2.accept(d2, last)
    bad = st2.codes.view(3, 2, 32, 64)
    assert torch.equal(bad[0], good[0]) and torch.equal(bad[2], good[2]) and torch.equal(bad[1, 0], good[1, 0])


def below(parents, n, t):
    """bool [N][T]: node t of sequence n and what hangs on it."""
    hit = torch.zeros(parents.shape, dtype=torch.bool)
    hit[n, t] = True
    for i, p in enumerate(parents[n].tolist()):
        if 0 <= p < i and hit[n, p]:
            hit[n, i] = True
    return hit


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "beta"])
@pytest.mark.parametrize("dtype,T,dk,dv,store", [("bf16", 14, 128, 128, "int4"), ("bf16", 64, 128, 72, "mix"),
                                                 ("f32", 40, 64, 48, "f32"), ("f16", 31, 256, 128, "int8")])
def test_broken_branch(mixer, name, dtype, T, dk, dv, store):
    """NaN and infinities in a node change no bit of the nodes that do not hang on it."""
    m = MIXERS[mixer]
    x, S = inputs(m, 2, T, "tree", 2, 2, dk, dv, TYPES[dtype], "cuda", seed=T)
    if x[name] is None:
        return
    st, _ = handle(m, S, store)
    o, d = verify(st, x)
    for value in (float("nan"), float("inf")):
        for t in (0, T // 3, T - 2):
            y = {n: None if a is None else a.clone() for n, a in x.items()}
            y[name][1, t, 1].view(-1)[-1] = value
            o2, d2 = verify(st, y)
            hit = below(x["parents"].cpu(), 1, t).cuda()
            for a, b in ((o, o2), (d.writes, d2.writes)):
                assert torch.equal(a[~hit], b[~hit]) and torch.equal(a[:, :, 0], b[:, :, 0])
            assert not o2[1, t, 1].isfinite().all()
            if name == "v":  # its column alone
                assert torch.equal(o2[..., :-1], o[..., :-1])
                assert not o2[hit][:, 1, -1].isfinite().any()
            # a path beside it enters the state as if it were not there
            ways = [i for i in range(T) if not hit[1, i]]
            last = torch.tensor([T - 1, ways[-1] if ways else -1], dtype=torch.int32, device="cuda")
            a, _ = handle(m, S, store)
            b, _ = handle(m, S, store)
            a.accept(d, last)
            b.accept(d2, last)
            assert torch.equal(a.codes, b.codes) and (store == "f32" or torch.equal(a.scales, b.scales))


def overflowing(m, T, branch, dtype, dk, dv, store):
    """A tree with a path of nodes `branch` whose keys are finite but so long that products of two of
    them, 1e24, have squares beyond FP32: with and without, and the nodes that hang on the path."""
    x, S = inputs(m, 2, T, "chain", 2, 2, dk, dv, TYPES[dtype], "cuda", seed=T)
    parents, other = [], -1
    for t in range(T):
        if t in branch:
            parents.append(([-1] + branch)[branch.index(t)])
            continue
        on = branch[-1] if t % 5 == 4 and branch[-1] < t else other if t % 3 else -1
        parents.append(on)
        other = t if on != branch[-1] else other
    x["parents"][:] = torch.tensor(parents, dtype=torch.int32, device="cuda")
    y = {n: None if t is None else t.clone() for n, t in x.items()}
    y["k"][1, branch] = (1e12 * x["k"][1, branch[0]].float()).to(TYPES[dtype])
    return x, y, S, below(x["parents"].cpu(), 1, branch[0])


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,branch,dk,dv,store", [(6, [0, 1, 2], 128, 128, "int4"), (20, [4, 13, 15], 64, 72, "f32"),
                                                  (40, [1, 17, 20], 128, 48, "mix"), (31, [16, 17, 18, 19], 256, 32, "int8")])
def test_products_beyond_the_range(mixer, dtype, T, branch, dk, dv, store):
    """Keys whose products overflow change no bit of the nodes that do not hang on them."""
    m = MIXERS[mixer]
    x, y, S, hit = overflowing(m, T, branch, dtype, dk, dv, store)
    st, _ = handle(m, S, store)
    o, d = verify(st, x)
    o2, d2 = verify(st, y)
    assert bool(o[~hit.cuda()].isfinite().all()) and bool(o2[1, branch[0]].isfinite().all())
    for a, b in ((o, o2), (d.writes, d2.writes)):
        assert torch.equal(a[~hit.cuda()], b[~hit.cuda()])
    last = torch.tensor([T - 1, [i for i in range(T) if not hit[1, i]][-1]], dtype=torch.int32, device="cuda")
    a, _ = handle(m, S, store)
    b, _ = handle(m, S, store)
    a.accept(d, last)
    b.accept(d2, last)
    assert torch.equal(a.codes, b.codes) and (store == "f32" or torch.equal(a.scales, b.scales))


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("dtype,dk,dv,store", [("f32", 64, 40, "f32"), ("bf16", 128, 128, "int8")])
def test_products_beyond_the_range_behind_a_common_node(mixer, dtype, dk, dv, store):
    """Node 0 has a long key, which its children 1 and 3 live with; what overflows behind 1 changes no bit
    of 3 and the nodes behind it."""
    m = MIXERS[mixer]
    x, S = inputs(m, 2, 20, "chain", 2, 1, dk, dv, TYPES[dtype], "cuda", seed=2)
    x["parents"][:] = torch.tensor([-1, 0, 1, 0, 3, 2] + list(range(4, 18)), dtype=torch.int32, device="cuda")
    x["k"][:, 0] = (1e12 * x["k"][:, 0].float()).to(TYPES[dtype])
    y = dict(x, k=x["k"].clone())
    y["k"][:, 1:3] = x["k"][:, :1]
    hit = (below(x["parents"].cpu(), 0, 1) | below(x["parents"].cpu(), 1, 1)).cuda()
    st, _ = handle(m, S, store)
    (o, d), (o2, d2) = verify(st, x), verify(st, y)
    assert not hit.all() and not hit[:, [0, 3, 4]].any()
    for a, b in ((o, o2), (d.writes, d2.writes)):
        assert torch.equal(a[~hit], b[~hit]) and bool(a[~hit].isfinite().all())


@pytest.mark.parametrize("last", [-1, -5, 9, 1 << 30, 3])
def test_last_that_is_no_node(last):
    x, S = inputs(GDN, 2, 9, "tree", 2, 2, 64, 32, torch.float32, "cuda")
    x["parents"][:, 3] = -2
    for store in ("f32", "int8"):
        st, _ = handle(GDN, S, store)
        _, draft = verify(st, x)
        before = st.codes.clone()
        scales = None if st.scales is None else st.scales.clone()
        st.accept(draft, torch.full((2,), last, dtype=torch.int32, device="cuda"))
        assert torch.equal(st.codes, before) and (scales is None or torch.equal(st.scales, scales))


@pytest.mark.parametrize("mixer", MIXERS)
@pytest.mark.parametrize("store", ["f32", "int8"])
def test_against_single_steps(mixer, store):
    """A drafted chain reads out what `step` does token by token on FP32 states, and decoding goes on
    from the accepted state."""
    m = MIXERS[mixer]
    x, S = inputs(m, 2, 6, "chain", 2, 2, 128, 64, torch.float32, "cuda")
    st, held = handle(m, S, store)
    plain, _ = handle(m, held)
    x["parents"] = None
    o, draft = verify(st, x)
    st.accept(draft, torch.full((2,), 3, dtype=torch.int32, device="cuda"))
    one = torch.empty(2, 2, 64, device="cuda")
    for t in range(4):
        a = x["log_alpha"][:, t].exp().contiguous()
        b = None if x["beta"] is None else x["beta"][:, t].contiguous()
        plain.step(x["q"][:, t].contiguous(), x["k"][:, t].contiguous(), x["v"][:, t].contiguous(), a, b, one)
        assert rel(o[:, t], one) <= 2 * VERIFY
    got, want = torch.empty_like(S), torch.empty_like(S)
    st.store_fp32(got)
    plain.store_fp32(want)
    if store == "f32":
        assert rel(got, want) <= 2 * (ACCEPT + VERIFY)
    else:
        assert rel(got, want) <= 0.5 / 127 * 6.0  # half a code, an absmax being below 6 deviations


@pytest.mark.parametrize("mixer", ["kda", "gdn"])
@pytest.mark.parametrize("rounding", [0, 1])
@pytest.mark.parametrize("store,dk,group", [("int8", 64, 32), ("mix", 128, 16), ("channels", 128, 32),
                                            ("int4", 256, 128)])
def test_quantized_as_an_import(mixer, rounding, store, dk, group):
    """The quantizer is the import's: the state behind the path, computed on an FP32 handle and
    imported with the same counter, seed and layer, has the same codes.  With a gate per channel the
    arithmetic before is the same too; one gate a token enters through the scale, and codes whose value
    lies at a border may differ by one."""
    m = MIXERS[mixer]
    x, S = inputs(m, 3, 8, "tree", 4, 4, dk, 40, torch.float32, "cuda")
    st, held = handle(m, S, store, group, rounding, seed=12345, layer=3)
    st.step_counter = 77
    plain, _ = handle(m, held)
    _, draft = verify(st, x)
    last = torch.tensor([7, 2, 0], dtype=torch.int32, device="cuda")
    st.accept(draft, last)
    plain.accept(draft, last)
    S2 = torch.empty_like(S)
    plain.store_fp32(S2)
    other, _ = handle(m, S, store, group, rounding, seed=12345, layer=3)
    other.step_counter = 77
    other.load_fp32(S2)
    assert st.step_counter == other.step_counter == 78
    if m == KDA:
        assert torch.equal(st.codes, other.codes) and torch.equal(st.scales, other.scales)
    else:
        a, b = torch.empty_like(S), torch.empty_like(S)
        st.store_fp32(a)
        other.store_fp32(b)
        assert rel(st.scales, other.scales) <= 2.0 ** -20
        far = (a - b).abs() > 2.0 ** -16 * b.abs().amax()
        assert float(far.float().mean()) < 1e-3
        step = other.scales.view(3, 4, 40, -1).repeat_interleave(group, -1)
        assert bool(((a - b).abs() <= 1.01 * step + 1e-6).all())


@pytest.mark.parametrize("store,group", [("int8", 32), ("int4", 16), ("channels", 16)])
def test_bounded_directional_rounding(store, group):
    """Within one code of the value, and never on the other side of the stored value from it."""
    x, S = inputs(GLA, 3, 8, "tree", 4, 4, 128, 40, torch.float32, "cuda")
    st, held = handle(GLA, S, store, group, 2)
    _, draft = verify(st, x)
    want, _, states = verify64(x, held, GLA)
    last = torch.tensor([7, 3, 0], dtype=torch.int32, device="cuda")
    st.accept(draft, last)
    got = torch.empty_like(S)
    st.store_fp32(got)
    goal = accept64(x, held, states, last)
    step = st.scales.view(3, 4, 40, -1).repeat_interleave(group, -1).double()
    eps = 1e-5 * goal.abs().amax()
    assert bool(((got - goal).abs() <= step + eps).all())
    up = goal - held
    wrong = ((got - held) * up < 0) & ((got - held).abs() > eps) & (up.abs() > eps)
    # a clamp to the code range may undo a step; nothing else may
    edge = (got.abs() / step.clamp(min=1e-30)) > {"int8": 126.5, "int4": 6.5, "channels": 6.5}[store]
    assert not bool((wrong & ~edge).any())


def test_strides_and_copies():
    """q, k and v as parts of wider rows, at any alignment, and as transposed views."""
    x, S = inputs(GDN, 3, 7, "tree", 2, 2, 64, 32, torch.bfloat16, "cuda")
    st, _ = handle(GDN, S, "int8")
    want, draft = verify(st, x)
    for pad in (0, 1, 8):
        wide = torch.cat([x["q"].flatten(2), x["k"].flatten(2), x["v"].flatten(2),
                          x["v"].flatten(2)[..., :pad]], 2)
        y = dict(x, q=wide[..., :128].view(3, 7, 2, 64), k=wide[..., 128:256].view(3, 7, 2, 64),
                 v=wide[..., 256:320].view(3, 7, 2, 32))
        o, d = verify(st, y)
        assert torch.equal(o, want) and torch.equal(d.writes, draft.writes)
        if pad == 8:
            assert d.k.data_ptr() == y["k"].data_ptr()
        a, _ = handle(GDN, S, "int8")
        b, _ = handle(GDN, S, "int8")
        last = torch.tensor([6, 1, 3], dtype=torch.int32, device="cuda")
        a.accept(draft, last)
        b.accept(d, last)
        assert torch.equal(a.codes, b.codes)
    y = {n: None if t is None else t.transpose(0, 1).contiguous().transpose(0, 1) for n, t in x.items()}
    assert torch.equal(verify(st, y)[0], want)


def test_one_output_only():
    from bit_recurrent_state_amd import DraftConfig, qstate_verify
    x, S = inputs(KDA, 2, 5, "tree", 2, 1, 64, 33, torch.float16, "cuda")
    st, _ = handle(KDA, S, "int4")
    o, draft = verify(st, x)
    c = DraftConfig(5, 1, torch.float16)
    a, b = torch.empty_like(o), torch.empty_like(draft.writes)
    rest = (x["q"], x["k"], x["v"], x["log_alpha"], x["beta"], x["parents"])
    qstate_verify(st.cfg, c, st.codes, st.scales, *rest, a)
    qstate_verify(st.cfg, c, st.codes, st.scales, *rest, None, b)
    assert torch.equal(a, o) and torch.equal(b, draft.writes)


def test_streams_and_graphs():
    """On another stream than the current one; captured once and replayed, the rounds in between eager."""
    x, S = inputs(GDN, 4, 12, "tree", 4, 2, 128, 64, torch.bfloat16, "cuda")
    last = lasts(x)
    st, _ = handle(GDN, S, "int8")
    want, draft = verify(st, x)
    st.accept(draft, last)
    after = st.codes.clone()
    st2, _ = handle(GDN, S, "int8")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, d = verify(st2, x, stream=s)
    st2.accept(d, last, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, want) and torch.equal(st2.codes, after)
    st3, _ = handle(GDN, S, "int8")
    start, scales = st3.codes.clone(), st3.scales.clone()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        o, d = verify(st3, x)
        st3.accept(d, last)
    for _ in range(3):
        st3.codes.copy_(start)
        st3.scales.copy_(scales)
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(st3.codes, after)


def test_a_round_of_decoding():
    """Drafts, the readout's norm and gate, acceptance, and the next draft, several times over, against
    the recurrence in 64 bits on FP32 states."""
    from bit_recurrent_state_amd import ReadoutNorm
    S = None
    for r in range(4):
        x, S0 = inputs(GDN, 3, 10, "ragged", 2, 2, 64, 32, torch.float32, "cuda", seed=r)
        if S is None:
            st, held = handle(GDN, S0)
            S = held.double()
        w = 1.0 + 0.1 * torch.randn(32, device="cuda")
        z = torch.randn(x["v"].shape, device="cuda")
        o, draft = verify(st, x, norm=ReadoutNorm(w, z))
        want, _, states = verify64(x, S, GDN)
        y = want * torch.rsqrt(want.square().mean(-1, keepdim=True) + 1e-6) * w.double()
        y = y * z.double() * torch.sigmoid(z.double())
        none = ~node_mask(x["parents"]).to("cuda")
        assert rel(o[~none], y[~none]) <= 64 * VERIFY
        last = lasts(x, r)
        st.accept(draft, last)
        S = accept64(x, S, states, last)
        got = torch.empty_like(S0)
        st.store_fp32(got)
        assert rel(got, S) <= (r + 1) * (ACCEPT + VERIFY)


@pytest.mark.parametrize("mixer", ["gdn", "kda"])
@pytest.mark.parametrize("gate_first", [False, True])
def test_norm_of_rows_of_no_node(mixer, gate_first):
    """The norm and the projection take padding as rows of zeros: what is in it reaches no node, and it
    comes out as the projection of bias (and gate)."""
    from bit_recurrent_state_amd import ReadoutNorm, Weight4
    m = MIXERS[mixer]
    x, S = inputs(m, 3, 13, "ragged", 2, 2, 64, 32, torch.bfloat16, "cuda", seed=5)
    x["parents"][0, 4] = -2
    none = ~node_mask(x["parents"]).to("cuda")
    assert none.any() and not none.all()
    st, _ = handle(m, S, "int4")
    g = torch.Generator(device="cuda").manual_seed(3)
    w, b = (torch.randn(2, 32, device="cuda", generator=g) for _ in range(2))
    z = torch.randn(x["v"].shape, device="cuda", generator=g).bfloat16()
    z2 = torch.where(none[..., None, None], torch.full_like(z, float("nan")), z)
    project = Weight4.quantize(torch.randn(48, 64, device="cuda", generator=g), 32)
    for p in (None, project):
        o, _ = verify(st, x, norm=ReadoutNorm(w, z, bias=b, gate_first=gate_first), project=p)
        o2, _ = verify(st, x, norm=ReadoutNorm(w, z2, bias=b, gate_first=gate_first), project=p)
        assert torch.equal(o[~none], o2[~none]) and o2[none].isnan().all()
        if p is None:
            want = b.expand_as(z)[none]
            if not gate_first:
                want = want.double() * torch.nn.functional.silu(z[none].double())
            # a rounding of the product, of its activation (as exp, sum, quotient, product) and to bfloat16
            assert bool(((o[none] - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all())


@pytest.mark.parametrize("name", ["q", "k", "v", "log_alpha", "beta", "weight", "gate", "bias"])
def test_gradients_are_refused(name):
    """Not differentiable: where a gradient or a tangent is wanted, nothing is launched."""
    from torch.autograd import forward_ad as fwd

    from bit_recurrent_state_amd import Draft, ReadoutNorm
    x, S = inputs(GDN, 2, 5, "tree", 2, 2, 64, 32, torch.float32, "cuda")
    st, _ = handle(GDN, S)
    extra = {"weight": torch.ones(32, device="cuda"), "bias": torch.zeros(32, device="cuda"),
             "gate": torch.randn(x["v"].shape, device="cuda")}
    _, draft = verify(st, x)
    last = torch.zeros(2, dtype=torch.int32, device="cuda")
    before, step = st.codes.clone(), st.step_counter

    def go(change):
        y = {n: change(t) if n == name else t for n, t in {**x, **extra}.items()}
        return verify(st, y, norm=ReadoutNorm(y["weight"], y["gate"], bias=y["bias"]))

    def leaf(t):
        return t.clone().requires_grad_(True)

    with pytest.raises(RuntimeError):
        go(leaf)
    with fwd.dual_level(), pytest.raises(RuntimeError):
        go(lambda t: fwd.make_dual(t, torch.ones_like(t)))
    with torch.no_grad():
        got = go(leaf)[0]
    assert torch.equal(got, go(lambda t: t)[0])
    if name in ("k", "log_alpha"):
        d = Draft(leaf(draft.k) if name == "k" else draft.k,
                  leaf(draft.log_alpha) if name == "log_alpha" else draft.log_alpha,
                  draft.parents, draft.writes)
        with pytest.raises(RuntimeError):
            st.accept(d, last)
        with fwd.dual_level(), pytest.raises(RuntimeError):
            st.accept(draft, last)
        assert torch.equal(st.codes, before) and st.step_counter == step
        with torch.no_grad():
            st.accept(d, last)
        assert st.step_counter == step + 1


def test_behind_2_to_the_31_elements():
    """Sequences whose FP32 state lies behind 2^31 elements give what they give alone."""
    from bit_recurrent_state_amd import Config, QState
    N, H, dk, dv = 2049, 64, 128, 128
    x, S = inputs(GDN, 3, 5, "tree", H, 1, dk, dv, torch.bfloat16, "cuda")
    st = QState(Config(N, H, dk, dv, mixer=GDN, fp32_state=True))
    st.codes.view(N, H, dv, dk)[-3:] = S
    few, _ = handle(GDN, S)
    want, draft = verify(few, x)
    wide = {n: torch.zeros((N,) + t.shape[1:], dtype=t.dtype, device="cuda") for n, t in x.items()}
    for n, t in x.items():
        wide[n][-3:] = t
    wide["parents"][:-3] = -2
    o, d = verify(st, wide)
    assert torch.equal(o[-3:], want) and not o[:-3].any()
    last = torch.full((N,), -1, dtype=torch.int32, device="cuda")
    last[-3:] = torch.tensor([4, 2, 0])
    st.accept(d, last)
    few.accept(draft, last[-3:].contiguous())
    assert torch.equal(st.codes.view(N, H, dv, dk)[-3:], few.codes.view(3, H, dv, dk))
    assert not st.codes.view(N, H, dv, dk)[:-3].any()


def test_refusals():
    from bit_recurrent_state_amd import Draft
    from bit_recurrent_state_amd._lib import QStateError
    x, S = inputs(GDN, 2, 5, "tree", 2, 2, 64, 32, torch.float32, "cuda")
    st, _ = handle(GDN, S)
    for bad in (dict(q=x["q"][:, :4]), dict(v=x["v"][:1]), dict(k=x["k"].bfloat16()),
                dict(log_alpha=x["log_alpha"].double()), dict(log_alpha=x["log_alpha"][..., None]),
                dict(beta=x["beta"][:, :2]), dict(parents=x["parents"].long()),
                dict(parents=x["parents"][:1]), dict(v=x["v"].flatten(2))):
        with pytest.raises(ValueError):
            verify(st, dict(x, **bad))
    for bad in (dict(q=x["q"].cpu()), dict(parents=x["parents"].cpu()), dict(beta=None)):
        with pytest.raises((TypeError, ValueError)):
            verify(st, dict(x, **bad))
    y, _ = inputs(GDN, 2, 65, "tree", 2, 2, 64, 32, torch.float32, "cuda")
    none = {n: None if t is None else t[:, :0] for n, t in x.items()}
    for T in (y, none):  # one to 64 rows
        with pytest.raises(QStateError):
            verify(st, T)
    _, draft = verify(st, x)
    last = torch.zeros(2, dtype=torch.int32, device="cuda")
    step = st.step_counter
    for bad in (last.long(), last[:1]):
        with pytest.raises(ValueError):
            st.accept(draft, bad)
    with pytest.raises(ValueError):
        st.accept(Draft(draft.k, draft.log_alpha, draft.parents, draft.writes[:, :3]), last)
    with pytest.raises(TypeError):
        st.accept(draft, last.cpu())
    assert st.step_counter == step
    for kw in (dict(window=4), dict(group_axis=1)):
        odd, _ = handle(GDN, S, "int8", **kw)
        with pytest.raises(QStateError):
            verify(odd, x)
        with pytest.raises(QStateError):
            odd.accept(draft, last)
    with pytest.raises(RuntimeError):
        torch.jit.trace(lambda q: verify(st, dict(x, q=q))[0], (x["q"],), check_trace=False)
