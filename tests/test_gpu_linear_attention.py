"""Linear attention against its definition in 64 bits (GPU), and the definition's gradients against differences (CPU).

Bounds.  An output adds products q_t . (gamma^n k_s) v_s.  With |.| for the same sum of magnitudes (A below), rounding
the products of a tile, or the state as it is read, to the inputs' type moves it by at most half a step of that type
times A, fp32 sums and powers by a few hundred steps of 2^-23 (their depth is below d + 64 + two a tile), and the
output's own rounding by half a step.  States are only moved by the fp32 part.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

gpu = pytest.mark.gpu
DT = {"f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tbe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import table_embedding_bags_gb300 as m

    m.load_library()
    return m


def definition(q, k, v, decay, offsets, s0, scale):
    """o [N, H, d], s_last [S, H, d, d], token by token in 64 bits."""
    N, H, d = q.shape
    S = len(offsets) - 1
    gamma = torch.exp(-decay)[:, None, None]
    o = torch.zeros_like(q)
    last = torch.zeros(S, H, d, d, dtype=q.dtype) if s0 is None else s0.clone()
    for s in range(S):
        state = last[s]
        for t in range(offsets[s], offsets[s + 1]):
            state = gamma * state + k[t][:, :, None] * v[t][:, None, :]
            o[t] = scale * torch.einsum("hi,hij->hj", q[t], state)
        last[s] = state
    return o, last


def gradients(do, q, k, v, decay, offsets, s0, ds_last, scale):
    N, H, d = q.shape
    S = len(offsets) - 1
    gamma = torch.exp(-decay)[:, None, None]
    dq, dk, dv = (torch.zeros_like(q) for _ in range(3))
    ds0 = torch.zeros(S, H, d, d, dtype=q.dtype) if ds_last is None else ds_last.clone()
    for s in range(S):
        state = torch.zeros(H, d, d, dtype=q.dtype) if s0 is None else s0[s]
        for t in range(offsets[s], offsets[s + 1]):
            state = gamma * state + k[t][:, :, None] * v[t][:, None, :]
            dq[t] = scale * torch.einsum("hij,hj->hi", state, do[t])
        g = ds0[s]
        for t in reversed(range(offsets[s], offsets[s + 1])):
            g = g + scale * q[t][:, :, None] * do[t][:, None, :]
            dk[t] = torch.einsum("hij,hj->hi", g, v[t])
            dv[t] = torch.einsum("hij,hi->hj", g, k[t])
            g = gamma * g
        ds0[s] = g
    return dq, dk, dv, ds0


def make(lengths, H, d, kind, seed, state=False, decays=(0.7, 0.01, 0.1, 0.0, 3.0), layout="slices"):
    gen = torch.Generator().manual_seed(seed)
    N, S = sum(lengths), len(lengths)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    if layout == "slices":  # of one projection, heads of 3 d
        p = normal(N, H, 3, d).to(DT[kind]).cuda()
        q, k, v = p[:, :, 0], p[:, :, 1], p[:, :, 2]
    elif layout == "heads first":
        q, k, v = (normal(H, N, d).to(DT[kind]).cuda().transpose(0, 1) for _ in range(3))
    elif layout == "off":  # rows that start on odd elements
        q, k, v = (normal(N, H, d + 3).to(DT[kind]).cuda()[:, :, 1:1 + d] for _ in range(3))
    else:
        q, k, v = (normal(N, H, d).to(DT[kind]).cuda() for _ in range(3))
    r = {"q": q, "k": k, "v": v, "do": normal(N, H, d).to(DT[kind]).cuda(),
         "decay": torch.tensor([decays[h % len(decays)] for h in range(H)], device="cuda"),
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64), device="cuda"),
         "s0": normal(S, H, d, d).cuda() if state else None, "ds_last": normal(S, H, d, d).cuda() if state else None}
    return r


def wide(t):
    return None if t is None else t.detach().double().cpu()


def close(got, want, size, half, fp32, what):
    """|got - want| <= (half + fp32) size + half |want|, with the smallest numbers of the type."""
    got = wide(got)
    tol = (half + fp32) * size + half * want.abs() + (2.0**-24 if half == 2.0**-11 else 1e-37) + 2.0**-30 * size.max()
    assert got.shape == want.shape
    off = (got - want).abs()
    assert (off <= tol).all(), f"{what}: worst {(off / tol).max().item():.3g} of the bound"


def run_and_check(tbe, c, kind, scale=0.3, grads=True):
    half = torch.finfo(DT[kind]).eps / 2
    q, k, v, do, s0, dl = (wide(c[n]) for n in ("q", "k", "v", "do", "s0", "ds_last"))
    decay, offsets = wide(c["decay"]), c["offsets"].tolist()
    fp32 = (q.shape[2] + 128 + max(np.diff(offsets), default=0) / 16) * 2.0**-22
    ab = lambda t: None if t is None else t.abs()  # noqa: E731
    o, last = definition(q, k, v, decay, offsets, s0, scale)
    size, size_last = definition(q.abs(), k.abs(), v.abs(), decay, offsets, ab(s0), abs(scale))
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=scale, want_last=True,
                                 dev_status=st)
    close(f.o, o, size, half, fp32, "o")
    if len(offsets) > 1:
        close(f.s_last, last, size_last, 0.0, fp32, "s_last")
    plain = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=scale)
    assert plain.s_last is None
    close(plain.o, o, size, half, fp32 + 2.0**-15, "o without last states")  # (states in two terms of bf16)
    if grads:
        args = (do, q, k, v)
        want = gradients(*args, decay, offsets, s0, dl, scale)
        sizes = gradients(*(t.abs() for t in args), decay, offsets, ab(s0), ab(dl), abs(scale))
        b = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"],
                                              ds_last=c["ds_last"], scale=scale, dev_status=st)
        for name, w, z in zip(("dq", "dk", "dv"), want, sizes):
            close(getattr(b, name), w, z, half, fp32, name)
        if c["s0"] is None:
            assert b.ds0 is None
        elif len(offsets) > 1:
            close(b.ds0, want[3], sizes[3], 0.0, fp32, "ds0")
    assert st.item() == 0
    return f


LENGTHS = {
    "one": [1],
    "tile": [64],
    "over": [65],
    "short": [1, 0, 3, 20, 0, 0, 17, 31, 2, 63, 64, 1, 40, 0],
    "ends on tiles": [64, 128, 0, 64],
    "long": [700],
    "mixed": [0, 5, 300, 1, 1, 1, 200, 90, 0],
    "singles": [1] * 150,
    "empties": [2] + [0] * 200 + [70] + [0] * 140 + [3],
}


@gpu
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("state", [False, True])
def test_against_definition(tbe, name, d, kind, state):
    if state and name in ("empties", "singles") and d == 128:
        pytest.skip("64-bit states of so many sequences take long")
    run_and_check(tbe, make(LENGTHS[name], 2, d, kind, d + len(name), state), kind)


@gpu
@pytest.mark.parametrize("layout", ["slices", "heads first", "off", "plain"])
@pytest.mark.parametrize("d", [1, 7, 8, 33, 63, 64, 65, 72, 100, 120, 127, 128])
def test_layouts_and_odd_widths(tbe, d, layout):
    run_and_check(tbe, make([30, 0, 99], 3, d, "bf16", d, True, layout=layout), "bf16")


@gpu
@pytest.mark.parametrize("d", [64, 128])
def test_many_runs(tbe, d):
    """Several runs of tiles to a sequence, sequences that cross, begin and end in them; int32 offsets."""
    c = make([1500, 3, 0, 700, 2900, 64], 1, d, "f16", 5, True, decays=(0.002,))
    c["offsets"] = c["offsets"].int()
    f = run_and_check(tbe, c, "f16")
    again = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=0.3, want_last=True)
    assert torch.equal(again.o, f.o) and torch.equal(again.s_last, f.s_last)


@gpu
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_step_goes_on_where_the_prefill_ended(tbe, kind):
    c = make([40, 1, 130], 3, 100, kind, 3, True)
    f = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], want_last=True)
    n = make([1, 1, 1], 3, 100, kind, 4)
    state = f.s_last.clone()
    o = tbe.tbe_linear_attention_step(n["q"], n["k"], n["v"], n["decay"], state, scale=0.5)
    want_o, want = definition(wide(n["q"]), wide(n["k"]), wide(n["v"]), wide(n["decay"]), [0, 1, 2, 3], wide(f.s_last), 0.5)
    size_o, size = definition(*(wide(n[x]).abs() for x in "qkv"), wide(n["decay"]), [0, 1, 2, 3], wide(f.s_last).abs(), 0.5)
    half = torch.finfo(DT[kind]).eps / 2
    close(o, want_o, size_o, half, 2.0**-14, "o")
    close(state, want, size, 0.0, 2.0**-21, "state")


def test_gradients_of_the_definition_against_differences():
    gen = torch.Generator().manual_seed(1)
    N, H, d, offsets = 9, 2, 4, [0, 4, 4, 9]
    normal = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k, v, do, s0, dl = normal(N, H, d), normal(N, H, d), normal(N, H, d), normal(N, H, d), normal(3, H, d, d), normal(3, H, d, d)
    decay = torch.tensor([0.3, 1.1], dtype=torch.float64)
    got = gradients(do, q, k, v, decay, offsets, s0, dl, 0.7)

    def value(*x):
        o, last = definition(x[0], x[1], x[2], decay, offsets, x[3], 0.7)
        return (o * do).sum() + (last * dl).sum()

    inputs = [q, k, v, s0]
    for i, g in enumerate(got):
        way = normal(*inputs[i].shape)
        h = 1e-5
        up, down = list(inputs), list(inputs)
        up[i], down[i] = inputs[i] + h * way, inputs[i] - h * way
        slope = (value(*up) - value(*down)) / (2 * h)
        assert abs(slope - (g * way).sum()) <= 1e-8 * (1 + abs(slope))


# ---------------------------------------------------------------------------
# values and sizes at the edges
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 100])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("what,value", [("v", float("nan")), ("v", float("inf")), ("k", float("nan")), ("q", float("nan")),
                                        ("do", float("-inf")), ("v", "row before a tile's end")])
def test_what_is_no_number_stays_in_its_sequence(tbe, what, value, kind, d, state):
    lengths = [20, 31, 0, 90, 5, 300, 17]
    c = make(lengths, 2, d, kind, 8, state)
    clean = {n: (t.clone() if isinstance(t, torch.Tensor) else t) for n, t in c.items()}
    bad, token = (1, 24) if isinstance(value, float) else (3, 125)
    c[what] = c[what].clone()
    c[what][token, 1] = value if isinstance(value, float) else float("nan")
    f, b = both(tbe, c)
    g, h = both(tbe, clean)
    ends = np.cumsum(lengths)
    inside = torch.zeros(sum(lengths), dtype=torch.bool, device="cuda")
    inside[ends[bad] - lengths[bad]:ends[bad]] = True
    half = torch.finfo(DT[kind]).eps / 2
    outs = [(f.o, g.o)] * (what != "do") + [(x, y) for x, y in zip(b[:3], h[:3])]
    assert any(not x[inside].isfinite().all() for x, _ in outs)
    for x, y in outs:  # other sequences, and the same one's other head: as before but for their rounding
        assert x[~inside].isfinite().all() and x[:, 0].isfinite().all()
        size = y.double().abs().max()
        assert ((x - y)[~inside].double().abs() <= 4 * half * size).all()
    if state:
        others = [s for s in range(len(lengths)) if s != bad]
        assert f.s_last[others].isfinite().all() and b.ds0[others].isfinite().all()


def both(tbe, c, scale=0.3):
    f = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=scale,
                                 want_last=c["s0"] is not None)
    b = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"],
                                          ds_last=c["ds_last"], scale=scale)
    return f, b


@gpu
def test_a_state_that_is_no_number_stays_in_its_sequence(tbe):
    c = make([20, 30, 0, 70], 2, 64, "bf16", 9, True)
    c["s0"][1, 0, 3, 5] = float("inf")
    f, _ = both(tbe, c)
    assert not f.o[20:50, 0].isfinite().all()
    assert f.o[:20].isfinite().all() and f.o[50:].isfinite().all() and f.o[:, 1].isfinite().all()


@gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q,k,v,scale", [(300.0, 300.0, 1e-2, 1e-4), (1e-3, 1e-3, 1.0, 1e3), (1.0, 200.0, 200.0, 1e-4),
                                         (1e-4, 1e-4, 1e-3, 1e8), (8e3, 5e-4, 1.0, 0.1)])
def test_products_and_states_beyond_half_precision(tbe, q, k, v, scale, d):
    """fp16 inputs whose products, or states, lie outside fp16's range, with outputs inside it."""
    c = make([10, 200, 3], 2, d, "f16", 10, True)
    for n, f in (("q", q), ("k", k), ("v", v)):
        c[n] = (c[n].float() * f).half()
    c["s0"] *= k * v
    c["do"] = (c["do"].float() * 1e-2).half()
    c["ds_last"] *= 1e-2
    run_and_check(tbe, c, "f16", scale, grads=False)


@gpu
def test_rows_of_very_different_size(tbe):
    c = make([60, 200], 1, 64, "f16", 11)
    c["q"] = c["q"].clone()
    c["q"][::3] *= 2.0**-12
    c["k"] = c["k"].clone()
    c["k"][::5] *= 2.0**-10
    run_and_check(tbe, c, "f16", 1.0)


@gpu
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_decays_at_the_ends(tbe, kind):
    c = make([100, 1, 300], 5, 48, kind, 12, True, decays=(0.0, 1e-6, 40.0, 200.0, 1e9))
    run_and_check(tbe, c, kind)
    c["decay"][4] = float("inf")  # only the token itself is remembered
    f, b = both(tbe, c)
    own = 0.3 * (wide(c["q"]) * wide(c["k"])).sum(-1, keepdim=True) * wide(c["v"])
    assert torch.allclose(wide(f.o)[:, 4], own[:, 4], rtol=0.02, atol=1e-2) and all(x.isfinite().all() for x in b[:3])


@gpu
@pytest.mark.parametrize("lengths", [[], [0], [0, 0, 0]])
def test_nothing_to_do(tbe, lengths):
    c = make(lengths, 2, 32, "bf16", 13, True)
    f, b = both(tbe, c)
    assert f.o.shape == (0, 2, 32) and torch.equal(f.s_last, c["s0"]) and torch.equal(b.ds0, c["ds_last"])
    c["s0"] = None
    f = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], want_last=True)
    assert not f.s_last.any()


@gpu
def test_only_some_states(tbe):
    """Gradients where states come in but no gradient of the last ones does, and the other way round."""
    c = make([30, 100, 0], 2, 40, "bf16", 14, True)
    run_and_check(tbe, {**c, "ds_last": torch.zeros_like(c["ds_last"])}, "bf16")
    q, k, v, do, s0 = (wide(c[n]) for n in ("q", "k", "v", "do", "s0"))
    b = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=0.3)
    want = gradients(do, q, k, v, wide(c["decay"]), c["offsets"].tolist(), s0, None, 0.3)
    for x, w in zip(b, want):
        assert float((wide(x) - w).norm()) <= 0.01 * float(w.norm())


@gpu
@pytest.mark.parametrize("offsets", [[0, 50, 40, 100], [5, 50, 100, 100], [0, 50, 100, 90], [0, -7, 100, 100],
                                     [0, 10**12, 100, 100], [100, 100, 100, 100], [0, 0, 0, 0]])
def test_broken_offsets_are_reported(tbe, offsets):
    c = make([30, 30, 40], 2, 64, "bf16", 15, True)
    c["offsets"] = torch.tensor(offsets, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], want_last=True, dev_status=st)
    assert st.item() == tbe.TBE_DEV_BAD_OFFSETS
    st.zero_()
    tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"],
                                      ds_last=c["ds_last"], dev_status=st)
    assert st.item() == tbe.TBE_DEV_BAD_OFFSETS


@gpu
@pytest.mark.parametrize("d", [64, 66])
def test_given_outputs_and_what_lies_between(tbe, d):
    c = make([70, 200], 3, d, "f16", 16)
    want = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"]).o
    room = torch.full((270, 3, d + 10), 7.0, dtype=torch.float16, device="cuda")
    got = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], out=room[:, :, 2:2 + d]).o
    assert got.data_ptr() == room[:, :, 2:].data_ptr() and torch.equal(got, want)
    assert (room[:, :, :2] == 7).all() and (room[:, :, 2 + d:] == 7).all()
    grads = torch.full((3, 3, 270, d + 1), 7.0, dtype=torch.float16, device="cuda")
    b = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"],
                                          out=tuple(g[:, :, :d].transpose(0, 1) for g in grads))
    alone = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"])
    assert all(torch.equal(x, y) for x, y in zip(b[:3], alone[:3])) and (grads[..., d] == 7).all()


@gpu
def test_streams_and_graphs(tbe):
    """Side by side on two streams, and captured and replayed with other contents, as on the current stream."""
    c, e = make([1500, 700, 3], 2, 64, "bf16", 17, True), make([900, 40, 1263], 2, 64, "bf16", 18, True)
    want = [both(tbe, x) for x in (c, e)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = both(tbe, e)
    here = both(tbe, c)
    torch.cuda.current_stream().wait_stream(side)
    same(here, want[0])
    same(other, want[1])
    given = tbe.tbe_linear_attention(e["q"], e["k"], e["v"], e["decay"], e["offsets"], s0=e["s0"], scale=0.3, want_last=True,
                                     stream=side)
    side.synchronize()
    assert torch.equal(given.o, want[1][0].o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = both(tbe, c)
    for n in ("q", "k", "v", "do", "offsets", "s0", "ds_last"):
        c[n].copy_(e[n])
    graph.replay()
    same(captured, want[1])


def same(a, b):
    for x, y in zip([*a[0], *a[1]], [*b[0], *b[1]]):
        assert torch.equal(x, y)


@gpu
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("B,H,d,layout", [(1, 1, 1, "plain"), (3, 2, 63, "off"), (200, 3, 64, "slices"), (5, 4, 128, "heads first"),
                                          (7, 1, 127, "plain"), (33, 5, 100, "slices")])
def test_single_tokens(tbe, B, H, d, layout, kind):
    n = make([1] * B, H, d, kind, 19, True, layout=layout)
    state = n["s0"].clone()
    o = tbe.tbe_linear_attention_step(n["q"], n["k"], n["v"], n["decay"], state, scale=0.2)
    args = [wide(n[x]) for x in "qkv"]
    offsets = list(range(B + 1))
    want_o, want = definition(*args, wide(n["decay"]), offsets, wide(n["s0"]), 0.2)
    size_o, size = definition(*(x.abs() for x in args), wide(n["decay"]), offsets, wide(n["s0"]).abs(), 0.2)
    close(o, want_o, size_o, torch.finfo(DT[kind]).eps / 2, (d + 4) * 2.0**-23, "o")
    close(state, want, size, 0.0, 2.0**-21, "state")


@gpu
def test_refusals(tbe):
    c = make([20, 30], 2, 64, "bf16", 20, True)
    args = dict(q=c["q"], k=c["k"], v=c["v"], decay=c["decay"], offsets=c["offsets"], s0=c["s0"])

    def refused(**other):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_linear_attention(**{**args, **other})
        if not {"out", "want_last"} & set(other):
            with pytest.raises(tbe.TBEError):
                tbe.tbe_linear_attention_backward(c["do"], **{**args, **other})

    for name in "qkv":
        refused(**{name: args[name].cpu()})
        refused(**{name: args[name].float()})
        refused(**{name: args[name][:-1]})
        refused(**{name: args[name].transpose(1, 2)})
        refused(**{name: args[name][:, :1].expand(50, 2, 64)})
    refused(q=c["q"].float(), k=c["k"].float(), v=c["v"].float())
    big = torch.zeros(50, 2, 129, dtype=torch.bfloat16, device="cuda")
    refused(q=big, k=big, v=big, s0=None)
    refused(decay=None)
    refused(decay=c["decay"].double())
    refused(decay=c["decay"][:1])
    refused(offsets=c["offsets"].float())
    refused(offsets=c["offsets"][:0])
    refused(offsets=c["offsets"][:1])
    refused(s0=c["s0"][:1])
    refused(s0=c["s0"].half())
    refused(scale=float("inf"))
    refused(out=torch.empty(50, 2, 64, device="cuda"))
    refused(out=c["q"][:, :, :32])
    with pytest.raises(tbe.TBEError):
        tbe.tbe_linear_attention_backward(c["do"][:3], **args)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_linear_attention_backward(c["do"], **args, ds_last=c["ds_last"][:1])
    with pytest.raises(tbe.TBEError):
        tbe.tbe_linear_attention_backward(c["do"], **args, out=(None, None))
    n = make([1, 1], 2, 64, "bf16", 21, True)
    for state in (None, n["s0"][:1], n["s0"].half(), n["s0"].transpose(2, 3)):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_linear_attention_step(n["q"], n["k"], n["v"], n["decay"], state)


@gpu
@pytest.mark.parametrize("N,H,d,row", [(200, 1, 100, 104), (1, 3, 64, 64), (1, 1, 7, 7), (130, 1, 60, 64)])
def test_one_head_or_one_token(tbe, N, H, d, row):
    """A stride that nothing is reached by says nothing."""
    c = make([N], H, d, "bf16", 22, True)
    for n in ("q", "k", "v", "do"):
        room = torch.zeros(N, H, row, dtype=torch.bfloat16, device="cuda")
        room[:, :, :d] = c[n]
        c[n] = room[:, :, :d]
    run_and_check(tbe, c, "bf16")
