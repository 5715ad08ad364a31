"""Gated recurrence over jagged sequences against its definition in 64 bits (GPU).

The reference runs token by token in numpy float64.  Tolerances are running
bounds, computed with it: each step's error is what the recurrence makes of
the error before it, plus the rounding of the step's own fp32 operations
(REL: about eight operations of two units in the last place each; ABS: a
decay near 1 is rounded to 2^-24), plus half a unit of the output's type.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

REL, ABS = 2.0 ** -19, 2.0 ** -23
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


@pytest.fixture(scope="module")
def tbe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import table_embedding_bags_gb300 as m

    m.load_library()
    return m


def dtype(name):
    return {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}[name]


def sigmoid(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def softplus(x):
    return np.logaddexp(0, x)


def rate(decay):
    """softplus, 0 below the smallest normal fp32 number (by the operator's definition)."""
    sp = softplus(decay)
    return np.where(sp < 2.0 ** -126, 0, sp)


def gates(x, r, g, decay, c):
    u = c * rate(decay) * sigmoid(r)
    a = np.exp(-u)
    beta = np.sqrt(-np.expm1(-2 * u))
    return u, a, beta, beta * sigmoid(g) * x


def reference(x, r, g, decay, offsets, h0, c, dh=None, dh_last=None):
    """Outputs and their error bounds; all arrays float64."""
    N, C = x.shape
    S = len(offsets) - 1
    u, a, beta, b = gates(x, r, g, decay, c)
    h, before, E, Ebefore = (np.zeros((N, C)) for _ in range(4))
    h_last, E_last = np.zeros((S, C)), np.zeros((S, C))
    for s in range(S):
        cur, e = (h0[s] if h0 is not None else np.zeros(C)), np.zeros(C)
        for t in range(offsets[s], offsets[s + 1]):
            before[t], Ebefore[t] = cur, e
            e = a[t] * e + np.abs(cur) * (ABS + REL * u[t]) + REL * np.abs(b[t]) + ABS * (np.abs(a[t] * cur) + np.abs(b[t]))
            cur = a[t] * cur + b[t]
            h[t], E[t] = cur, e
        h_last[s], E_last[s] = cur, e
    out = {"h": (h, E), "h_last": (h_last, E_last)}
    if dh is None:
        return out
    G, EG = np.zeros((N, C)), np.zeros((N, C))
    dh0, Edh0 = np.zeros((S, C)), np.zeros((S, C))
    for s in range(S):
        cur, e = (dh_last[s] if dh_last is not None else np.zeros(C)), np.zeros(C)
        for t in range(offsets[s + 1] - 1, offsets[s] - 1, -1):
            G[t] = dh[t] + cur
            EG[t] = e + ABS * (np.abs(dh[t]) + np.abs(cur))
            e = a[t] * EG[t] + np.abs(G[t]) * (ABS + REL * u[t]) + ABS * np.abs(a[t] * G[t])
            cur = a[t] * G[t]
        dh0[s], Edh0[s] = cur, e
    sr, sg = sigmoid(r), sigmoid(g)
    slope = np.divide(u * a * a, beta, out=np.zeros_like(u), where=beta > 0)
    c1, c2 = slope * sg * x, u * a * before
    w = G * (c1 - c2)
    Ew = EG * np.abs(c1 - c2) + np.abs(G) * (2 * REL * (np.abs(c1) + np.abs(c2)) + u * a * Ebefore)
    out["dx"] = G * beta * sg, EG * beta * sg + 2 * REL * np.abs(G * beta * sg)
    dg = G * beta * sg * x
    out["dgate"] = dg * (1 - sg), (EG * np.abs(beta * sg * x) + 2 * REL * np.abs(dg)) * (1 - sg) + ABS * np.abs(dg)
    out["drecur"] = w * (1 - sr), Ew * (1 - sr) + ABS * np.abs(w)
    ratio = sigmoid(decay) / softplus(decay)
    out["ddecay"] = ratio * w.sum(0), ratio * (Ew.sum(0) + (REL + 64 * ABS) * np.abs(w).sum(0))
    out["dh0"] = dh0, Edh0
    return out


def check(got, ref, kind, what):
    value, err = ref
    got = got.detach().double().cpu().numpy()
    tol = 2 * err + (HALF_ULP[kind] * (np.abs(value) + err) * 1.01 + SUBNORMAL[kind]) + 1e-37
    off = np.abs(got - value)
    assert np.all(off <= tol), f"{what}: worst {np.max(off / tol):.3g} of the bound at {np.argmax(off / tol)}"


def make(N, S, C, kind, seed, h0=True, lengths=None, i32=False):
    """Inputs on the device as slices of one projection, and the same in float64."""
    rng = np.random.default_rng(seed)
    if lengths is None:
        lengths = rng.multinomial(N, rng.dirichlet(np.full(S, 0.7)))
    offsets = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)
    proj = torch.from_numpy(rng.standard_normal((N, 3 * C)).astype(np.float32)).to("cuda", dtype(kind))
    decay = rng.uniform(-7, 0, C).astype(np.float32)
    d = {"x": proj[:, :C], "recur": proj[:, C:2 * C], "gate": proj[:, 2 * C:], "decay": torch.from_numpy(decay).cuda(),
         "offsets": torch.from_numpy(offsets).to("cuda", torch.int32 if i32 else torch.int64),
         "h0": torch.from_numpy(rng.standard_normal((S, C)).astype(np.float32)).cuda() if h0 else None}
    d["dh"] = torch.from_numpy(rng.standard_normal((N, C)).astype(np.float32)).to("cuda", dtype(kind))
    d["dh_last"] = torch.from_numpy(rng.standard_normal((S, C)).astype(np.float32)).cuda()
    return d


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def ref_of(d, c=8.0, back=True):
    args = [f64(d[k]) for k in ("x", "recur", "gate", "decay")]
    return reference(*args, d["offsets"].cpu().numpy().astype(np.int64), f64(d["h0"]), c,
                     f64(d["dh"]) if back else None, f64(d["dh_last"]) if back else None)


def run(tbe, d, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]
    f = tbe.tbe_gated_scan(*ins, h0=d["h0"], want_states=True, dev_status=st, **kw)
    b = tbe.tbe_gated_scan_backward(d["dh"], *ins, f.states, h0=d["h0"], dh_last=d["dh_last"], dev_status=st, **kw)
    assert int(st) == 0
    return f, b


def check_all(tbe, d, kind, **kw):
    f, b = run(tbe, d, **kw)
    ref = ref_of(d, kw.get("sharpness", 8.0))
    check(f.h, ref["h"], kind, "h")
    check(f.h_last, ref["h_last"], "f32", "h_last")
    for name in ("dx", "drecur", "dgate"):
        check(getattr(b, name), ref[name], kind, name)
    check(b.ddecay, ref["ddecay"], "f32", "ddecay")
    if d["h0"] is not None:
        check(b.dh0, ref["dh0"], "f32", "dh0")
    else:
        assert b.dh0 is None
    return f, b


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,S,C", [(1, 1, 1), (7, 3, 5), (127, 1, 64), (128, 2, 33), (129, 4, 66), (640, 300, 40),
                                   (1000, 9, 130), (2500, 2, 32)])
def test_forward_and_backward(tbe, N, S, C, kind):
    """Tile edges, widths that are no multiple of a vector, empty sequences."""
    check_all(tbe, make(N, S, C, kind, N + C, h0=N % 2 == 0, i32=S % 2 == 0), kind)


@pytest.mark.parametrize("N,S", [(128 * 16, 1), (128 * 16 + 1, 2), (128 * 256 + 77, 1), (128 * 300, 3)])
def test_long_sequences_join_tiles_groups_and_rows(tbe, N, S):
    """Sequences over many tiles: the joins within a group, across groups and across rows of groups."""
    check_all(tbe, make(N, S, 34, "f32", N, lengths=[N - (S - 1) * 5] + [5] * (S - 1)), "f32")


@pytest.mark.parametrize("lengths", [[0, 0, 5, 0], [128, 0, 0, 128, 0], [0] * 700 + [3] + [0] * 700, [1] * 300,
                                     [127, 1, 128, 256, 0, 0, 1, 0]])
def test_empty_sequences_and_tile_edges(tbe, lengths):
    check_all(tbe, make(sum(lengths), len(lengths), 6, "f32", 3, lengths=lengths), "f32")


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [6, 34, 129, 256])
@pytest.mark.parametrize("lengths", [[1] * 700 + [5000] + [2] * 900, [4000] + [0] * 500 + [1] * 900 + [0] * 40,
                                     [0] * 400 + [3, 40] * 90 + [2500], [37] * 300])
def test_many_sequences_of_uneven_length(tbe, lengths, C, kind):
    """Sequences that do not lie where equal lengths would put them, at every width of copy."""
    check_all(tbe, make(sum(lengths), len(lengths), C, kind, C, lengths=lengths, i32=C % 2 == 0), kind)


@pytest.mark.parametrize("kind,C", [("f16", 64), ("bf16", 34), ("bf16", 33)])
def test_long_half_precision_sequences(tbe, kind, C):
    """Many blocks along the tokens: a block's way back to the last start is longer than a warp's."""
    check_all(tbe, make(40000, 2, C, kind, C, lengths=[39000, 1000]), kind)


def test_nothing_but_empty_sequences(tbe):
    d = make(0, 5, 9, "bf16", 1, lengths=[0] * 5)
    f, b = run(tbe, d)
    assert f.h.shape == (0, 9) and torch.equal(f.h_last, d["h0"])
    assert torch.equal(b.dh0, d["dh_last"]) and not b.ddecay.any()


def test_no_sequences(tbe):
    d = make(0, 1, 4, "f32", 1, lengths=[0])
    off = d["offsets"][:1]
    e = torch.empty(0, 4, device="cuda")
    f = tbe.tbe_gated_scan(d["x"], d["recur"], d["gate"], d["decay"], off, want_states=True)
    b = tbe.tbe_gated_scan_backward(e, d["x"], d["recur"], d["gate"], d["decay"], off, f.states)
    assert f.h_last.shape == (0, 4) and not b.ddecay.any()


def test_extreme_gates(tbe):
    """Closed and open gates: -inf carries the state on unchanged, large values forget it; decays from
    never (softplus near 0) to at once."""
    d = make(300, 3, 16, "f32", 5, lengths=[100, 150, 50])
    d["recur"][::7] = -float("inf")
    d["recur"][3::7] = 80.0
    d["gate"][::5] = -float("inf")
    d["gate"][2::5] = 90.0
    d["decay"][0], d["decay"][1], d["decay"][2] = -100.0, 30.0, -17.0
    f, b = check_all(tbe, d, "f32")
    h = f.h.cpu()
    for t in range(7, 100, 7):  # recur = -inf: exactly the state before (a run of 8 tokens starts from joined
        if t % 8:               # maps, whose rounding is not the run before's: there the bound above holds)
            assert torch.equal(h[t], h[t - 1]), t
    assert torch.isfinite(b.drecur).all() and torch.isfinite(b.ddecay).all()


@pytest.mark.parametrize("where", ["x", "recur"])
def test_nan_stays_in_its_sequence(tbe, where):
    d = make(1500, 4, 8, "f32", 6, lengths=[400, 500, 0, 600])
    clean = run(tbe, d)
    d[where][450, 3] = float("nan")
    f, b = run(tbe, d)
    assert torch.isnan(f.h[450:900, 3]).all()  # from there to the end of its sequence
    keep = torch.ones(1500, dtype=torch.bool)
    keep[450:900] = False
    assert torch.equal(f.h[keep.cuda()], clean[0].h[keep.cuda()])
    other = [0, 1, 2, 4, 5, 6, 7]
    assert torch.equal(f.h[:, other], clean[0].h[:, other])
    keep[400:900] = False
    for name in ("dx", "drecur", "dgate"):
        assert torch.equal(getattr(b, name)[keep.cuda()], getattr(clean[1], name)[keep.cuda()])
    assert torch.equal(b.ddecay[other], clean[1].ddecay[other])


def test_results_do_not_depend_on_timing_or_stream(tbe):
    d = make(40_000, 3, 96, "bf16", 7, lengths=[30_000, 0, 10_000])
    f0, b0 = run(tbe, d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        with torch.cuda.stream(side):
            f, b = run(tbe, d)
        torch.cuda.current_stream().wait_stream(side)
        for p, q in zip((*f0, *b0), (*f, *b)):
            assert torch.equal(p, q)


def test_strides_and_given_outputs(tbe):
    """Odd row strides and starts (one channel per lane), outputs into slices; the rest stays untouched."""
    d = make(333, 5, 24, "f16", 8)
    want_f, want_b = run(tbe, d)
    wide = torch.full((333, 101), 3.0, device="cuda", dtype=torch.float16)
    for i, k in enumerate(("x", "recur", "gate")):
        wide[:, 1 + 25 * i:25 + 25 * i] = d[k]
        d[k] = wide[:, 1 + 25 * i:25 + 25 * i]
    ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]
    room = torch.full((333, 101), 7.0, device="cuda", dtype=torch.float16)
    f = tbe.tbe_gated_scan(*ins, h0=d["h0"], want_states=True, out=room[:, 76:100])
    assert f.h.data_ptr() == room[:, 76:].data_ptr()
    assert torch.equal(f.h, want_f.h) and torch.equal(f.states, want_f.states)
    out = tuple(room[:, 1 + 25 * i:25 + 25 * i] for i in range(3))
    b = tbe.tbe_gated_scan_backward(d["dh"], *ins, f.states, h0=d["h0"], dh_last=d["dh_last"], out=out)
    for name in ("dx", "drecur", "dgate", "ddecay", "dh0"):
        assert torch.equal(getattr(b, name), getattr(want_b, name)), name
    assert (room[:, [0, 25, 50, 75, 100]] == 7).all()


def test_sharpness_and_no_last_gradient(tbe):
    d = make(500, 4, 12, "f32", 9, h0=False)
    check_all(tbe, d, "f32", sharpness=2.5)
    f, b = run(tbe, {**d, "dh_last": None})
    ref = reference(*[f64(d[k]) for k in ("x", "recur", "gate", "decay")], d["offsets"].cpu().numpy(), None, 8.0,
                    f64(d["dh"]), None)
    check(b.dx, ref["dx"], "f32", "dx")
    check(b.ddecay, ref["ddecay"], "f32", "ddecay")


@pytest.mark.parametrize("name", ["x", "recur", "gate", "decay", "h0"])
def test_gradients_against_differences(tbe, name):
    """<gradient, v> against the central difference of the 64-bit loss along v (relative truncation error of
    step 1e-5: about 1e-10 times third derivatives; fp32 gradients: 1e-5)."""
    d = make(260, 3, 10, "f32", 11)
    _, b = run(tbe, d)
    grad = {"x": b.dx, "recur": b.drecur, "gate": b.dgate, "decay": b.ddecay, "h0": b.dh0}[name]
    rng = np.random.default_rng(12)
    v = rng.standard_normal(tuple(grad.shape))
    arrays = {k: f64(d[k]) for k in ("x", "recur", "gate", "decay", "h0")}
    off, dh, dl = d["offsets"].cpu().numpy(), f64(d["dh"]), f64(d["dh_last"])

    def loss(step):
        z = {**arrays, name: arrays[name] + step * v}
        o = reference(z["x"], z["recur"], z["gate"], z["decay"], off, z["h0"], 8.0)
        return (o["h"][0] * dh).sum() + (o["h_last"][0] * dl).sum()

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    got = float((f64(grad) * v).sum())
    scale = np.sqrt(((f64(grad) * v) ** 2).sum())
    assert abs(got - want) <= 1e-5 * max(scale, abs(want)) + 1e-7


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S,C", [(1, 1), (3, 33), (64, 256), (5000, 7)])
def test_single_tokens(tbe, S, C, kind):
    """One token of each sequence: the definition, and the same state as a jagged batch of length-1 sequences."""
    d = make(S, S, C, kind, S + C, lengths=[1] * S)
    state = d["h0"].clone()
    h = tbe.tbe_gated_scan_step(d["x"], d["recur"], d["gate"], d["decay"], state)
    ref = ref_of(d, back=False)
    check(h, ref["h"], kind, "h")
    check(state, ref["h_last"], "f32", "state")


def test_prefill_then_single_tokens_equals_the_whole(tbe):
    d = make(204, 2, 40, "f32", 14, lengths=[102, 102])
    whole = tbe.tbe_gated_scan(d["x"], d["recur"], d["gate"], d["decay"], d["offsets"], h0=d["h0"])
    split = lambda t: t.reshape(2, 102, -1)  # noqa: E731
    head = [split(d[k])[:, :100].reshape(200, -1).contiguous() for k in ("x", "recur", "gate")]
    part = tbe.tbe_gated_scan(*head, d["decay"], torch.tensor([0, 100, 200], device="cuda"), h0=d["h0"])
    state = part.h_last.clone()
    ref = ref_of(d, back=False)
    for t in (100, 101):
        h = tbe.tbe_gated_scan_step(*[split(d[k])[:, t].contiguous() for k in ("x", "recur", "gate")], d["decay"], state)
        check(h, tuple(a.reshape(2, 102, -1)[:, t] for a in ref["h"]), "f32", "h")
    check(state, ref["h_last"], "f32", "state")
    check(whole.h_last, ref["h_last"], "f32", "h_last")


def test_more_than_2_to_31_elements(tbe):
    """Rows beyond 2^31 elements of the projection: the last sequence equals a batch of its own."""
    C, N, tail = 512, 1_500_000, 300
    proj = torch.zeros(N, 3 * C, dtype=torch.bfloat16, device="cuda")
    proj[-tail:] = torch.randn(tail, 3 * C, device="cuda")
    decay = torch.full((C,), -4.0, device="cuda")
    off = torch.tensor([0, N - tail, N], device="cuda")
    parts = lambda p: (p[:, :C], p[:, C:2 * C], p[:, 2 * C:])  # noqa: E731
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = tbe.tbe_gated_scan(*parts(proj), decay, off, want_states=True, dev_status=st)
    dh = torch.zeros(N, C, dtype=torch.bfloat16, device="cuda")
    dh[-tail:] = 1
    d = torch.empty_like(proj)
    tbe.tbe_gated_scan_backward(dh, *parts(proj), decay, off, f.states, out=parts(d), dev_status=st)
    small = proj[-tail:].contiguous()
    own = torch.tensor([0, tail], device="cuda")
    g = tbe.tbe_gated_scan(*parts(small), decay, own, want_states=True)
    e = torch.empty_like(small)
    tbe.tbe_gated_scan_backward(dh[-tail:].contiguous(), *parts(small), decay, own, g.states, out=parts(e))
    assert int(st) == 0
    assert torch.allclose(f.h[-tail:].float(), g.h.float(), rtol=2 ** -7, atol=1e-6)  # tiles cut elsewhere: one bf16 step
    assert torch.allclose(d[-tail:].float(), e.float(), rtol=2 ** -7, atol=1e-6)
    assert not f.h[:N - tail].any() and not d[:N - tail].any()


@pytest.mark.parametrize("offsets", [[1, 5, 10], [0, 7, 9], [0, 8, 5], [0, -3, 10], [0, 99, 10]])
def test_broken_offsets_are_reported(tbe, offsets):
    """Accesses stay in bounds by construction (every use of an offset is checked against its tile)."""
    d = make(10, 2, 4, "f32", 2, lengths=[5, 5])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tbe.tbe_gated_scan(d["x"], d["recur"], d["gate"], d["decay"], torch.tensor(offsets, device="cuda"), dev_status=st)
    assert int(st) & tbe.TBE_DEV_BAD_OFFSETS


def test_refusals(tbe):
    d = make(10, 2, 4, "f32", 2, lengths=[5, 5])
    ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]

    def refused(i, bad):
        a = list(ins)
        a[i] = bad
        with pytest.raises(tbe.TBEError):
            tbe.tbe_gated_scan(*a)

    refused(0, ins[0].cpu())
    refused(0, ins[0].double())
    refused(1, ins[1].half())
    refused(1, ins[1][:9])
    refused(2, ins[2].t().contiguous().t())  # columns apart
    refused(2, ins[2][:1].expand(10, 4))  # rows that overlap
    refused(3, ins[3].half())
    refused(3, ins[3][:3])
    refused(4, ins[4].float())
    refused(4, ins[4][:0])
    for kw in ({"h0": d["h0"][:1]}, {"h0": d["h0"].half()}, {"out": torch.empty(10, 3, device="cuda")},
               {"sharpness": float("nan")}, {"sharpness": -1.0}, {"dev_status": torch.zeros(1, device="cuda")}):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_gated_scan(*ins, **kw)
    f = tbe.tbe_gated_scan(*ins, want_states=True)
    for bad in (None, f.states[:, :3], f.states.half()):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_gated_scan_backward(d["dh"], *ins, bad)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_gated_scan_backward(d["dh"][:, :3], *ins, f.states)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_gated_scan_step(*ins[:4], d["h0"])  # ten tokens, two states


def pool_of(t):
    """The handle of the stream whose memory a tensor lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def test_calls_on_a_given_stream_keep_their_buffers(tbe):
    """``stream=``: what a call allocates is the given stream's memory, and is not handed out again before that
    stream, and the caller's, are through with it."""
    data = [make(40_000, 3, 96, "bf16", 30 + i, lengths=[30_000, 0, 10_000]) for i in range(2)]
    want = [run(tbe, d) for d in data]
    sides = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = []
    for d, side in zip(data, sides):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # the calls wait behind it, so that both streams' kernels run together
        ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]
        f = tbe.tbe_gated_scan(*ins, h0=d["h0"], want_states=True, stream=side)
        got.append((f, tbe.tbe_gated_scan_backward(d["dh"], *ins, f.states, h0=d["h0"], dh_last=d["dh_last"], stream=side)))
        junk = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(8, 26) for _ in range(3)]
        del junk
    torch.cuda.synchronize()
    for (f0, b0), (f, b), side in zip(want, got, sides):
        for p, q in zip((*f0, *b0), (*f, *b)):
            assert torch.equal(p, q)
            assert pool_of(q) == side.cuda_stream != torch.cuda.current_stream().cuda_stream
    state = data[0]["h0"].clone()
    ins = [data[0][k][:3] for k in ("x", "recur", "gate")] + [data[0]["decay"]]
    torch.cuda.synchronize()
    h = tbe.tbe_gated_scan_step(*ins, state, stream=sides[0])
    torch.cuda.synchronize()
    assert pool_of(h) == sides[0].cuda_stream
    torch.cuda._sleep(40_000_000)  # the current stream may still read f.h
    f = got[0][0].h
    at = f.data_ptr()
    got[0] = None
    del p, q, f0, b0, b, f
    with torch.cuda.stream(sides[0]):
        again = [torch.empty(40_000, 96, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    assert at not in [t.data_ptr() for t in again]
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("N", [100, 1500, 20_000])
def test_nan_gate_stays_out_of_what_does_not_depend_on_it(tbe, N, kind):
    """gate[t] enters h from t on, and of the gradients dx[t], dgate[t] and what h enters: drecur from t on.  The
    others are as in the reference (channels that forget slowly: both gates from one reciprocal)."""
    C, ch, start, end = 40, 3, N // 4, N - N // 5
    d = make(N, 3, C, kind, 20, lengths=[start, end - start, N - end])
    d["decay"].clamp_(max=-4.5)
    ref = ref_of(d)
    at = start + (end - start) // 3
    d["gate"][at, ch] = float("nan")
    f, b = run(tbe, d)
    hit = {name: np.zeros((N, C), bool) for name in ("h", "dx", "drecur", "dgate")}
    hit["h"][at:end, ch] = hit["drecur"][at:end, ch] = True
    hit["dx"][at, ch] = hit["dgate"][at, ch] = True
    for name, got in (("h", f.h), ("dx", b.dx), ("drecur", b.drecur), ("dgate", b.dgate)):
        got = got.double().cpu().numpy()
        assert np.isnan(got[hit[name]]).all(), name
        value, err = (a[~hit[name]] for a in ref[name])
        check(torch.from_numpy(got[~hit[name]]), (value, err), kind, name)
    other = [c for c in range(C) if c != ch]
    check(b.ddecay[other], tuple(a[other] for a in ref["ddecay"]), "f32", "ddecay")
    check(b.dh0, ref["dh0"], "f32", "dh0")


def test_arguments_without_a_truth_value(tbe):
    """A flag that cannot be told true or false raises what asking it raises."""
    d = make(10, 2, 4, "f32", 2, lengths=[5, 5])
    ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]
    with pytest.raises(ValueError):
        tbe.tbe_gated_scan(*ins, want_states=np.zeros(2))
    logits, labels = torch.zeros(4, 5, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    with pytest.raises(ValueError):
        tbe.tbe_preference_loss(logits, labels, off, torch.zeros(2, device="cuda"), want_grad=np.zeros(2))


def test_out_of_memory_is_told_as_such(tbe):
    """An output that does not fit raises what torch.empty raises, and the next call works."""
    torch.cuda.empty_cache()
    d = make(4096, 2, 2048, "f32", 2, h0=False, lengths=[2048, 2048])
    ins = [d[k] for k in ("x", "recur", "gate", "decay", "offsets")]
    want = tbe.tbe_gated_scan(*ins).h.clone()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (4 << 20)) / total)
        with pytest.raises(torch.OutOfMemoryError):
            held = [tbe.tbe_gated_scan(*ins) for _ in range(64)]  # 32 MB each, more than freed memory holds
        held = None
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.equal(tbe.tbe_gated_scan(*ins).h, want)
