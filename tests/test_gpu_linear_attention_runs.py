"""Linear attention where a run of the token axis takes several tiles of 128 tokens: states kept from tile to tile, sums of
several tiles, values that are no numbers among them.

The definition is taken in 64 bits by blocks of 64 tokens, products that the causal mask leaves out not added at all.
Bounds as in test_gpu_linear_attention.py: half a step of the
type for the products of a tile or the state as it is read, a few hundred steps of 2^-23 for fp32 sums and powers.
"""

import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import table_embedding_bags_gb300 as tbe  # noqa: E402

pytestmark = pytest.mark.gpu

DT = {"f16": torch.float16, "bf16": torch.bfloat16}
TILE = 128


def tiles_of_a_run(N, H, d, passes):
    """How many tiles each block takes one after the other: as many blocks as the GPU holds at once share them out."""
    tiles = -(-N // TILE)
    blocks = (2 if d <= 64 else 1) * torch.cuda.get_device_properties(0).multi_processor_count
    return -(-tiles // max(1, blocks // (H * passes)))


def forward(q, k, v, decay, offsets, s0, scale, behind=False):
    """o [N, H, d] and the last states in 64 bits; `behind`: the decay comes behind the read."""
    N, H, d = q.shape
    o = torch.zeros_like(q)
    last = torch.zeros(len(offsets) - 1, H, d, d, dtype=q.dtype, device=q.device) if s0 is None else s0.clone()
    step = 64
    n = torch.arange(step, device=q.device, dtype=q.dtype)
    late = 1 if behind else 0
    power = lambda e: torch.exp(-decay.view(H, *[1] * e.dim()) * e)  # noqa: E731
    for s in range(len(offsets) - 1):
        state = last[s]
        for t in range(offsets[s], offsets[s + 1], step):
            m = min(step, offsets[s + 1] - t)
            a, b, c = (x[t:t + m].transpose(0, 1) for x in (q, k, v))
            apart = n[:m, None] - n[None, :m]
            w = torch.where(apart >= 0, (a @ b.transpose(1, 2)) * power(apart.clamp(min=0)), 0.0)
            bad = ~c.isfinite()
            x = w @ torch.where(bad, 0.0, c) + power(n[:m] + 1 - late)[..., None] * (a @ state)
            for h, i, j in bad.nonzero().tolist():  # (times 0 they would be NaN for tokens before them)
                x[h, i:, j] += w[h, i:, i] * c[h, i, j]
            o[t:t + m] = scale * x.transpose(0, 1)
            state = power(torch.tensor(float(m), device=q.device, dtype=q.dtype))[..., None, None] * state + \
                (b * power(m - 1 - n[:m] + late)[..., None]).transpose(1, 2) @ c
        last[s] = state
    return o, last


def backward(do, q, k, v, decay, offsets, s0, ds_last, scale):
    turned = [offsets[-1] - x for x in reversed(offsets)]
    flip = lambda x: None if x is None else x.flip(0)  # noqa: E731
    t = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    dq, _ = forward(do, v, k, decay, offsets, t(s0), scale)
    dk, _ = forward(flip(v), flip(do) * scale, flip(q), decay, turned, flip(t(ds_last)), 1.0, True)
    dv, ds0 = forward(flip(k), flip(q) * scale, flip(do), decay, turned, flip(ds_last), 1.0, True)
    return dq, dk.flip(0), dv.flip(0), ds0.flip(0)


def make(lengths, H, d, kind, seed, state, layout="slices"):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    N, S = sum(lengths), len(lengths)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if layout == "slices":
        q, k, v = normal(N, 3, H, d).to(DT[kind]).unbind(1)
    else:  # rows that tensor copies cannot read
        q, k, v = (normal(N, H, d + 1).to(DT[kind])[:, :, :d] for _ in range(3))
    return {"q": q, "k": k, "v": v, "do": normal(N, H, d).to(DT[kind]),
            "decay": torch.logspace(-3.5, 0.3, H, device="cuda"),
            "offsets": torch.tensor(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64), device="cuda"),
            "s0": normal(S, H, d, d) if state else None, "ds_last": normal(S, H, d, d) if state else None}


def both(c, scale=0.3, want_last=True):
    f = tbe.tbe_linear_attention(c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"], scale=scale, want_last=want_last)
    b = tbe.tbe_linear_attention_backward(c["do"], c["q"], c["k"], c["v"], c["decay"], c["offsets"], s0=c["s0"],
                                          ds_last=c["ds_last"], scale=scale)
    return f, b


def wanted(c, scale=0.3, magnitudes=False):
    x = {n: None if c[n] is None else c[n].double() for n in ("q", "k", "v", "do", "s0", "ds_last")}
    if magnitudes:
        x = {n: None if t is None else t.abs() for n, t in x.items()}
    decay, offsets = c["decay"].double(), c["offsets"].tolist()
    o, last = forward(x["q"], x["k"], x["v"], decay, offsets, x["s0"], scale)
    return o, last, *backward(x["do"], x["q"], x["k"], x["v"], decay, offsets, x["s0"], x["ds_last"], scale)


def close(got, want, size, half, fp32, what, where=None):
    off = (got.double() - want).abs()
    tol = (half + fp32) * size + half * want.abs() + (2.0**-24 if half == 2.0**-11 else 1e-37) + 2.0**-30 * size.max()
    ratio = off / tol
    if where is not None:
        ratio = ratio[where]
    assert (ratio <= 1).all(), f"{what}: worst {ratio.max().item():.3g} of the bound"


LENGTHS = {
    "long": [10_007],
    "cross": [3000, 1, 0, 2500, 128, 0, 4000, 500],
    "short": [20, 0, 300, 70] * 25,
    "whole tiles": [1280, 2560, 128, 128, 1024, 4096],
}


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", list(LENGTHS))
@pytest.mark.parametrize("state", [False, True])
def test_runs_of_several_tiles(name, d, kind, state):
    lengths, H = LENGTHS[name], 16
    N = sum(lengths)
    assert tiles_of_a_run(N, H, d, 1) >= 3 and tiles_of_a_run(N, H, d, 3) >= 3
    c = make(lengths, H, d, kind, 1 + d, state)
    f, b = both(c, want_last=state)
    want, size = wanted(c), wanted(c, magnitudes=True)
    half = torch.finfo(DT[kind]).eps / 2
    fp32 = (d + 128 + max(lengths) / 16) * 2.0**-22 + (0.0 if state else 2.0**-15)  # (states in two terms of bf16)
    for got, w, z, what in zip((f.o, *b[:3]), (want[0], *want[2:5]), (size[0], *size[2:5]), ("o", "dq", "dk", "dv")):
        close(got, w, z, half, fp32, what)
    if state:
        close(f.s_last, want[1], size[1], 0.0, fp32, "s_last")
        close(b.ds0, want[5], size[5], 0.0, fp32, "ds0")
    g, e = both(c, want_last=state)
    assert all(torch.equal(x, y) for x, y in zip((f.o, *b[:3]), (g.o, *e[:3])))


@pytest.mark.parametrize("d", [40, 100])
def test_runs_of_several_tiles_by_smaller_copies(d):
    """Widths that are filled up, rows that tensor copies cannot read."""
    c = make(LENGTHS["cross"], 16, d, "bf16", 2, True, layout="off")
    assert tiles_of_a_run(sum(LENGTHS["cross"]), 16, d, 1) >= 3
    f, b = both(c)
    want, size = wanted(c), wanted(c, magnitudes=True)
    fp32 = (d + 128 + 4000 / 16) * 2.0**-22
    for got, w, z, what in zip((f.o, *b[:3]), (want[0], *want[2:5]), (size[0], *size[2:5]), ("o", "dq", "dk", "dv")):
        close(got, w, z, 2.0**-8, fp32, what)
    close(f.s_last, want[1], size[1], 0.0, fp32, "s_last")
    close(b.ds0, want[5], size[5], 0.0, fp32, "ds0")




def finite_where_the_definition_is(got, want, size, half, fp32, what):
    """Where the definition's output is finite, so is the kernel's, and right."""
    ok = want.isfinite()
    assert ok.any() and not ok.all(), what
    close(torch.where(ok, got.double(), 0.0), torch.where(ok, want, 0.0), size, half, fp32, what)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 100])
@pytest.mark.parametrize("name", ["s0", "v", "k", "ds_last", "do", "q"])
def test_an_infinity_in_a_state_leaves_the_others_their_digits(name, d, kind):
    """In a state that comes in, or in what is added to it first: the power of two that fp16 operands are moved by comes from
    their finite values.  (An infinite key or query makes a row of the state infinite, a value a column.)"""
    c = make([700, 300], 16, d, kind, 4, True)
    size = wanted(c, magnitudes=True)
    x = dict(c)
    x[name] = c[name].clone()
    if name in ("s0", "ds_last"):
        x[name][0, 1, 3, 5] = math.inf
        x[name][1, 2, 7, 9] = -math.inf
    else:
        first = (0, 700) if name in "vk" else (699, 999)
        x[name][first[0], 1, 5] = math.inf
        x[name][first[1], 0, 9] = -math.inf
    f, b = both(x)
    want = wanted(x)
    fp32 = (d + 128 + 700 / 16) * 2.0**-22
    half = torch.finfo(DT[kind]).eps / 2
    if name in ("s0", "v", "k"):
        finite_where_the_definition_is(f.s_last, want[1], size[1], 0.0, fp32, "s_last")
    else:
        finite_where_the_definition_is(b.ds0, want[5], size[5], 0.0, fp32, "ds0")
    if name in ("s0", "v"):
        finite_where_the_definition_is(f.o, want[0], size[0], half, fp32, "o")
    if name in ("ds_last", "do"):
        finite_where_the_definition_is(b.dv, want[4], size[4], half, fp32, "dv")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("d", [64, 100])
@pytest.mark.parametrize("layout", ["slices", "off"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("state", [False, True])
@pytest.mark.parametrize("lengths,tokens", [([128], [127]), ([300], [0, 50, 130, 299]), ([40, 60, 0, 90], [70, 189]),
                                            ([2000, 3001], [1999, 2300, 4000])])
def test_what_is_no_number_is_not_seen_before_its_token(lengths, tokens, value, state, layout, d, kind):
    """Single entries of the values that are no numbers: other columns, and tokens before (behind, for dk and dv), are
    as the definition has them."""
    H = 2 if sum(lengths) < 1000 else 16
    c = make(lengths, H, d, kind, 3, state, layout)
    size = wanted(c, magnitudes=True)
    half = torch.finfo(DT[kind]).eps / 2
    fp32 = (d + 128 + max(lengths) / 16) * 2.0**-22 + 2.0**-15
    # the operand that takes the values' place: v for o, k for dq, q for dk, do for dv
    for name, i in (("v", 0), ("k", 2), ("q", 3), ("do", 4)):
        x = dict(c)
        x[name] = c[name].clone()
        for j, t in enumerate(tokens):
            x[name][t, 1, 7 * j + 3] = value
        f, b = both(x, want_last=state)
        want = wanted(x)
        finite_where_the_definition_is((f.o, None, *b)[i], want[i], size[i], half, fp32, name)
        if state and name in ("v", "do"):
            j = 1 if name == "v" else 5
            finite_where_the_definition_is(f.s_last if name == "v" else b.ds0, want[j], size[j], 0.0, fp32, name + "'s state")


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("lengths", [[300, 500], [1] * 200, [4000, 2000]])
def test_a_head_of_nothing_but_nan(lengths, kind):
    """Every value of one head, or every third one: the other heads stay as they are, bit for bit."""
    c = make(lengths, 16 if sum(lengths) > 1000 else 2, 64, kind, 5, False)
    f, b = both(c, want_last=False)
    for every in (1, 3):
        x = {**c, "v": c["v"].clone(), "do": c["do"].clone()}
        x["v"][::every, 1] = math.nan
        x["do"][::every, 1] = math.nan
        g, e = both(x, want_last=False)
        others = [h for h in range(c["q"].shape[1]) if h != 1]
        assert all(torch.equal(p[:, others], q[:, others]) for p, q in zip((f.o, *b[:3]), (g.o, *e[:3])))
        assert g.o[::every, 1].isnan().all() and e.dv[::every, 1].isnan().all()
        first = np.concatenate([[0], np.cumsum(lengths)])
        for s, n in enumerate(lengths):  # up to its sequence's first such token an output is the clean one
            at = -int(first[s]) % every
            assert torch.equal(g.o[first[s]:first[s] + min(at, n), 1], f.o[first[s]:first[s] + min(at, n), 1])
            assert g.o[first[s]:first[s] + min(at, n), 1].isfinite().all()


@pytest.mark.parametrize("order", ["slices", "slices of heads", "heads first"])
def test_outputs_between_the_inputs(order):
    """All of a call's rows in one buffer: what lies between is neither refused nor touched."""
    c = make([300, 77], 3, 40, "bf16", 6, False)
    want, grads = both(c, want_last=False)
    N, H, d = c["q"].shape
    if order == "slices":
        room = torch.zeros(N, 9, H, d, dtype=torch.bfloat16, device="cuda").unbind(1)
    elif order == "slices of heads":
        room = torch.zeros(N, H, 9, d, dtype=torch.bfloat16, device="cuda").unbind(2)
    else:
        room = [x.transpose(0, 1) for x in torch.zeros(H, 9, N, d, dtype=torch.bfloat16, device="cuda").unbind(1)]
    q, k, v, do, o, dq, dk, dv, last = room
    for x, name in zip((q, k, v, do), ("q", "k", "v", "do")):
        x.copy_(c[name])
    last.fill_(7)
    f = tbe.tbe_linear_attention(q, k, v, c["decay"], c["offsets"], scale=0.3, out=o)
    b = tbe.tbe_linear_attention_backward(do, q, k, v, c["decay"], c["offsets"], scale=0.3, out=(dq, dk, dv))
    assert torch.equal(f.o, want.o) and all(torch.equal(x, y) for x, y in zip(b[:3], grads[:3])) and (last == 7).all()
    for out in ((dq, dk, dq), (q, dk, dv), (dq, dk, do)):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_linear_attention_backward(do, q, k, v, c["decay"], c["offsets"], scale=0.3, out=out)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_linear_attention(q, k, v, c["decay"], c["offsets"], out=v)
