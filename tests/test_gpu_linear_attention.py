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
         "offsets": torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), device="cuda"),
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
@pytest.mark.parametrize("d", [1, 7, 33, 63, 65, 100, 127])
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
