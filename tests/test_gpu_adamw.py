"""AdamW over a list of tensors against its definition in 64 bits (GPU).

Bounds: a moment is three roundings of its terms (2^-22 of their sizes); the
update passes a square root and a division of two units each and three more
roundings (2^-20 of its size); the weight adds its own rounding and half a
unit of its type.  8-bit states are compared code by code with a numpy
float32 restatement (one rounding per operation on both sides), and as
values with the 64-bit definition to half a code.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BLOCK = 256
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HYPER = {"learning_rate": 3e-3, "beta1": 0.9, "beta2": 0.99, "eps": 1e-8, "weight_decay": 0.1, "step": 7}
SIZES = [1, 255, 256, 257, 0, 5000, 64, 2048, 3, 70_001]
F = np.float32


@pytest.fixture(scope="module")
def tbe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import table_embedding_bags_gb300 as m

    m.load_library()
    return m


def tensors(sizes, kind, scale, seed, misaligned=False):
    rng = np.random.default_rng(seed)
    flat = torch.from_numpy((rng.standard_normal(sum(sizes) + 1) * scale).astype(F)).to("cuda", DT[kind])
    views = flat[1:].split(list(sizes)) if misaligned else [v.clone() for v in flat[1:].split(list(sizes))]
    return list(views)


def padded(sizes):
    return sum(-(-n // BLOCK) * BLOCK for n in sizes)


def slices(sizes):
    at, out = 0, []
    for n in sizes:
        out.append(slice(at, at + n))
        at += -(-n // BLOCK) * BLOCK
    return out


def state32(sizes, seed):
    rng = np.random.default_rng(seed)
    m, v = np.zeros(padded(sizes), F), np.zeros(padded(sizes), F)
    for s in slices(sizes):
        m[s] = rng.standard_normal(s.stop - s.start) * 1e-3
        v[s] = rng.standard_normal(s.stop - s.start) ** 2 * 1e-6
    return m, v


def want64(p, g, m, v, h, scale=1.0):
    """New weight, moments and their error bounds, in float64."""
    g = g * scale
    m1, v1 = h["beta1"] * m + (1 - h["beta1"]) * g, h["beta2"] * v + (1 - h["beta2"]) * g * g
    em = 2.0 ** -22 * (np.abs(m) + np.abs(g))
    ev = 2.0 ** -22 * (v + g * g)
    root = np.sqrt(v1 / (1 - h["beta2"] ** h["step"])) + h["eps"]
    step = h["learning_rate"] / (1 - h["beta1"] ** h["step"]) * m1 / root
    p1 = (1 - h["learning_rate"] * h["weight_decay"]) * p - step
    with np.errstate(divide="ignore", invalid="ignore"):
        ep = np.abs(step) * 2.0 ** -20 + np.abs(step) * np.where(v1 > 0, ev / np.where(v1 > 0, v1, 1), 0) \
            + h["learning_rate"] / (1 - h["beta1"] ** h["step"]) * em / root + 2.0 ** -22 * np.abs(p)
    return (p1, ep), (m1, em), (v1, ev)


def near(got, want, kind, what):
    value, err = want
    tol = 2 * err + HALF_ULP[kind] * 1.01 * (np.abs(value) + err) + (2.0 ** -25 if kind == "f16" else 1e-44)
    off = np.abs(got.astype(np.float64) - value)
    assert np.all(off <= tol), f"{what}: worst {np.nanmax(off / tol):.3g} of the bound"


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


@pytest.mark.parametrize("misaligned", [False, True])
@pytest.mark.parametrize("pk,gk", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32"), ("f32", "f16")])
def test_32_bit_states(tbe, pk, gk, misaligned):
    p, g = tensors(SIZES, pk, 0.05, 1, misaligned), tensors(SIZES, gk, 1e-3, 2, misaligned)
    m, v = state32(SIZES, 3)
    state = {"exp_avg": torch.from_numpy(m.copy()).cuda(), "exp_avg_sq": torch.from_numpy(v.copy()).cuda()}
    before = [f64(t) for t in p]
    plan = tbe.AdamWPlan(p, g, state=state)
    assert plan.slices == slices(SIZES)
    scale = torch.tensor([0.37], device="cuda")
    tbe.tbe_adamw_step(plan, grad_scale=scale, **HYPER)
    m1, v1 = plan.exp_avg.cpu().numpy(), plan.exp_avg_sq.cpu().numpy()
    for i, s in enumerate(slices(SIZES)):
        wp, wm, wv = want64(before[i], f64(g[i]), m[s].astype(np.float64), v[s].astype(np.float64), HYPER, float(F(0.37)))
        near(f64(p[i]), wp, pk, f"weight {i}")
        near(m1[s], wm, "f32", f"exp_avg {i}")
        near(v1[s], wv, "f32", f"exp_avg_sq {i}")
        s = slice(s.stop, -(-s.stop // BLOCK) * BLOCK)
        assert not m1[s].any() and not v1[s].any()  # the padding


def levels(count, power):
    return np.array([((k - 0.5) / count) ** power for k in range(1, count + 1)]).astype(F)


def quantise(x, count, power):
    """Codes and scales of blocks of float32 values, one rounding per operation."""
    x = x.reshape(-1, BLOCK)
    top = np.abs(x).max(1)
    top = np.where(top >= np.finfo(F).tiny, top, F(0))
    with np.errstate(divide="ignore"):
        inv = np.where(top > 0, F(1) / top, F(0)).astype(F)
    y = (np.abs(x) * inv[:, None]).astype(F)
    code = np.searchsorted(levels(count, power), y, side="right")
    return code, top, y


def dequantise8(qm, qv, sm, sv):
    q = qm.astype(F).reshape(-1, BLOCK)
    m = (q * np.abs(q)) * (sm * F(1 / 127 ** 2))[:, None]
    z = qv.astype(F).reshape(-1, BLOCK)
    z = z * z
    v = (z * z) * (sv * F(1 / 255 ** 4))[:, None]
    return m.reshape(-1), v.reshape(-1)


def step8(g, qm, qv, sm, sv, h):
    m, v = dequantise8(qm, qv, sm, sv)
    m = m * F(h["beta1"]) + g * F(1 - h["beta1"])
    v = v * F(h["beta2"]) + (g * g) * F(1 - h["beta2"])
    code, top, _ = quantise(m, 127, 2)
    qm = (code * np.sign(m).reshape(-1, BLOCK)).astype(np.int8).reshape(-1)
    zcode, ztop, y = quantise(v, 255, 4)
    zcode = np.maximum(zcode, y > 0)
    return m, v, qm, zcode.astype(np.uint8).reshape(-1), top.astype(F), ztop.astype(F)


def state8(sizes, seed):
    rng = np.random.default_rng(seed)
    n = padded(sizes)
    qm, qv = np.zeros(n, np.int8), np.zeros(n, np.uint8)
    for s in slices(sizes):
        qm[s] = rng.integers(-127, 128, s.stop - s.start)
        qv[s] = rng.integers(0, 256, s.stop - s.start)
    sm = (10.0 ** rng.uniform(-7, -2, n // BLOCK)).astype(F)
    sv = (10.0 ** rng.uniform(-14, -5, n // BLOCK)).astype(F)
    return qm, qv, sm, sv


def plan8(tbe, p, g, st):
    names = ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    return tbe.AdamWPlan(p, g, state_bits=8, state={k: torch.from_numpy(a.copy()).cuda() for k, a in zip(names, st)})


def codes(plan):
    return [t.cpu().numpy() for t in (plan.exp_avg, plan.exp_avg_sq, plan.exp_avg_scale, plan.exp_avg_sq_scale)]


def flat_padded(ts, sizes):
    out = np.zeros(padded(sizes), F)
    for t, s in zip(ts, slices(sizes)):
        out[s] = t.float().cpu().numpy().reshape(-1)
    return out


@pytest.mark.parametrize("misaligned", [False, True])
@pytest.mark.parametrize("pk,gk", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16")])
def test_8_bit_states(tbe, pk, gk, misaligned):
    """Three steps: codes and scales equal the restatement's bit for bit, weights within their bounds."""
    p, g = tensors(SIZES, pk, 0.05, 4, misaligned), tensors(SIZES, gk, 1e-3, 5, misaligned)
    g[5].view(-1)[::3] = 0
    st = state8(SIZES, 6)
    plan = plan8(tbe, p, g, st)
    for step in range(3):
        h = {**HYPER, "step": 50 + step}
        before = [f64(t) for t in p]
        m, v, *new = step8(flat_padded(g, SIZES), *st, h)
        tbe.tbe_adamw_step(plan, **h)
        for name, got, want in zip(("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"), codes(plan), new):
            assert np.array_equal(got, want), f"{name}: {np.sum(got != want)} differ in step {step}"
        dm, dv = dequantise8(*st)
        vm, vv = tbe.tbe_adamw_state(plan)
        for i, s in enumerate(slices(SIZES)):
            wp, wm, wv = want64(before[i], f64(g[i]), dm[s].astype(np.float64), dv[s].astype(np.float64), h)
            near(f64(p[i]), wp, pk, f"weight {i}")
            # half a code in the root: |sqrt(x) - sqrt(y)| <= (0.5 / 127) sqrt(scale), + rounding
            top = np.repeat(new[2], BLOCK)[s].astype(np.float64)
            got = vm.cpu().numpy()[s].astype(np.float64)
            assert np.all(np.abs(np.sqrt(np.abs(got)) - np.sqrt(np.abs(wm[0]))) <= (0.5 / 127 + 1e-5) * np.sqrt(top))
            assert np.all((got == 0) | (np.sign(got) == np.sign(wm[0])))
            top = np.repeat(new[3], BLOCK)[s].astype(np.float64)
            got = vv.cpu().numpy()[s].astype(np.float64)
            low = got ** 0.25 - wv[0] ** 0.25
            assert np.all(np.abs(low) <= (1.0 / 255 + 1e-5) * top ** 0.25)  # up to a whole code above zero
            assert np.all((got > 0) == (wv[0] > 0))
        want_m, want_v = dequantise8(*new)
        assert np.array_equal(vm.cpu().numpy(), want_m) and np.array_equal(vv.cpu().numpy(), want_v)
        st = new


def test_codes_next_to_every_level(tbe):
    """Moments one unit in the last place on either side of every level take the right code."""
    rows_m, rows_v = levels(127, 2), levels(255, 4)
    blocks = []
    for lv in (rows_m, rows_v):
        lv = lv.astype(F)
        near_ = np.concatenate([np.nextafter(lv, F(0)), lv, np.nextafter(lv, F(1))])
        for part in np.array_split(near_, -(-len(near_) // 255)):
            b = np.zeros(BLOCK, F)
            b[0] = 1
            b[1:1 + len(part)] = part
            blocks.append(b)
    g = np.concatenate(blocks)
    n = len(g)
    h = {**HYPER, "beta1": 0.0, "beta2": 0.0}
    for values in (g, np.sqrt(g)):  # as first moments, and squared as second ones
        values = values.astype(F)
        values[1::2] *= -1
        zero = (np.zeros(n, np.int8), np.zeros(n, np.uint8), np.zeros(n // BLOCK, F), np.zeros(n // BLOCK, F))
        plan = plan8(tbe, [torch.zeros(n, device="cuda")], [torch.from_numpy(values).cuda()], zero)
        tbe.tbe_adamw_step(plan, **h)
        for got, want in zip(codes(plan), step8(values, *zero, h)[2:]):
            assert np.array_equal(got, want)


def test_from_zero_follows_the_textbook(tbe):
    """Ten steps from zero states, against the 64-bit recursion; 8-bit states stay within a few percent of it."""
    n, rng = 1000, np.random.default_rng(8)
    w0 = rng.standard_normal(n).astype(F)
    grads = rng.standard_normal((10, n)).astype(F)
    w, m, v = w0.astype(np.float64), np.zeros(n), np.zeros(n)
    for t in range(1, 11):
        (w, _), (m, _), (v, _) = want64(w, grads[t - 1].astype(np.float64), m, v, {**HYPER, "step": t})
    moved = np.linalg.norm(w - w0)
    for bits, bound in ((32, 1e-5), (8, 0.05)):
        p, g = torch.from_numpy(w0.copy()).cuda(), torch.zeros(n, device="cuda")
        plan = tbe.AdamWPlan([p], [g], state_bits=bits)
        for t in range(1, 11):
            g.copy_(torch.from_numpy(grads[t - 1]))
            tbe.tbe_adamw_step(plan, **{**HYPER, "step": t})
        assert np.linalg.norm(f64(p) - w) <= bound * moved


@pytest.mark.parametrize("bits", [8, 32])
def test_skip_changes_nothing(tbe, bits):
    p, g = tensors([300, 20], "f32", 1, 9), tensors([300, 20], "f32", 1, 10)
    plan = tbe.AdamWPlan(p, g, state_bits=bits)
    tbe.tbe_adamw_step(plan, **HYPER)
    kept = [t.clone() for t in (*p, *tbe.tbe_adamw_state(plan))]
    skip = torch.ones(1, dtype=torch.int32, device="cuda")
    tbe.tbe_adamw_step(plan, skip=skip, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip(kept, (*p, *tbe.tbe_adamw_state(plan))))
    skip.zero_()
    tbe.tbe_adamw_step(plan, skip=skip, **HYPER)
    assert not torch.equal(kept[0], p[0])


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_gradients(tbe, bad):
    """32 bits: the element alone is lost.  8 bits: its block of states reads back as NaN, the next block is whole."""
    for bits in (32, 8):
        p, g = torch.ones(700, device="cuda"), torch.ones(700, device="cuda")
        g[300] = bad
        plan = tbe.AdamWPlan([p], [g], state_bits=bits)
        tbe.tbe_adamw_step(plan, **{**HYPER, "step": 1})
        m, v = (t.cpu() for t in tbe.tbe_adamw_state(plan))
        hit = torch.zeros(m.numel(), dtype=torch.bool)
        hit[256:512 if bits == 8 else 0] = True
        hit[300] = True
        if bits == 8:
            assert torch.isnan(m[hit]).all() and torch.isnan(v[hit]).all()
        else:
            assert not torch.isfinite(m[300]) and not torch.isfinite(v[300])
        assert torch.isfinite(m[~hit]).all() and torch.isfinite(v[~hit]).all()
        ok = torch.ones(700, dtype=torch.bool)
        ok[300] = False
        assert torch.isfinite(p.cpu()[ok]).all() and not torch.isfinite(p.cpu()[300])


def test_zero_and_tiny_states(tbe):
    """Zero gradients on zero states move nothing but the decay; blocks too small to scale are held as zero."""
    p, g = torch.ones(512, device="cuda"), torch.zeros(512, device="cuda")
    g[256:] = 1e-38
    plan = tbe.AdamWPlan([p], [g], state_bits=8)
    tbe.tbe_adamw_step(plan, **{**HYPER, "eps": 1e-8, "step": 1})
    assert torch.isfinite(p).all()
    assert torch.equal(p[:256], torch.full((256,), float(F(1 - 3e-4)), device="cuda"))
    m, v = tbe.tbe_adamw_state(plan)
    assert not m.any() and not v.any() and torch.isfinite(m).all()


def test_mixed_list_rebind_and_streams(tbe):
    """Types mixed over the list, new gradients by rebind, a step on another stream."""
    sizes = [300, 4096, 17, 256]
    kinds = ["f32", "bf16", "f16", "bf16"]
    p = [tensors([n], k, 0.1, i)[0] for i, (n, k) in enumerate(zip(sizes, kinds))]
    g = [tensors([n], k, 0.1, i + 9)[0] for i, (n, k) in enumerate(zip(sizes, kinds[::-1]))]
    plan = tbe.AdamWPlan(p, [torch.zeros_like(t) for t in g])
    plan.rebind(grads=g)
    before = [f64(t) for t in p]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tbe.tbe_adamw_step(plan, stream=side, **HYPER)
    torch.cuda.current_stream().wait_stream(side)
    for i, k in enumerate(kinds):
        wp, _, _ = want64(before[i], f64(g[i]), 0.0 * before[i], 0.0 * before[i], HYPER)
        near(f64(p[i]), wp, k, f"weight {i}")


def test_many_small_tensors(tbe):
    """More tensors than a tile has blocks, empty ones among them."""
    sizes = [i % 5 for i in range(2000)]
    p, g = tensors(sizes, "f32", 1, 11), tensors(sizes, "f32", 1, 12)
    before = [f64(t) for t in p]
    tbe.tbe_adamw_step(tbe.AdamWPlan(p, g), **HYPER)
    for i in range(2000):
        near(f64(p[i]), want64(before[i], f64(g[i]), 0 * before[i], 0 * before[i], HYPER)[0], "f32", f"weight {i}")


def test_more_than_2_to_31_elements(tbe):
    """One tensor of 2.2e9 elements: its last block moves as a small tensor's."""
    n, tail = 2_200_000_321, 1000
    p, g = torch.zeros(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    p[-tail:], g[-tail:] = 1, 0.01
    plan = tbe.AdamWPlan([p], [g], state_bits=8)
    tbe.tbe_adamw_step(plan, **HYPER)
    want = want64(1.0, float(g[-1]), 0.0, 0.0, HYPER)[0][0]
    assert torch.allclose(p[-tail:].float(), torch.full((tail,), want, device="cuda"), rtol=2 ** -8)
    assert int((p[:-tail] != 0).sum()) == 0
    codes_ = plan.exp_avg[n - tail:n]
    assert (codes_ > 0).all() and not plan.exp_avg[n:].any()


def test_refusals(tbe):
    p, g = [torch.ones(10, device="cuda")], [torch.ones(10, device="cuda")]
    E = tbe.TBEError
    for bad_p, bad_g in ((p, []), ([], []), (p, [g[0][:9]]), (p, [g[0].double()]), ([p[0].cpu()], g), (p, [g[0].cpu()]),
                         ([torch.ones(20, device="cuda")[::2]], g)):
        with pytest.raises(E):
            tbe.AdamWPlan(bad_p, bad_g)
    with pytest.raises(E):
        tbe.AdamWPlan(p, g, state_bits=16)
    for state in ({}, {"exp_avg": torch.zeros(256, device="cuda")},
                  {"exp_avg": torch.zeros(255, device="cuda"), "exp_avg_sq": torch.zeros(256, device="cuda")},
                  {"exp_avg": torch.zeros(256), "exp_avg_sq": torch.zeros(256)}):
        with pytest.raises(E):
            tbe.AdamWPlan(p, g, state=state)
    plan = tbe.AdamWPlan(p, g)
    for k, v in (("step", 0), ("beta1", 1.0), ("beta2", -0.1), ("eps", -1e-8), ("eps", float("nan")),
                 ("learning_rate", float("inf")), ("weight_decay", float("nan"))):
        with pytest.raises(E):
            tbe.tbe_adamw_step(plan, **{**HYPER, k: v})
    for kw in ({"grad_scale": torch.ones(1)}, {"grad_scale": torch.ones(2, device="cuda")},
               {"skip": torch.ones(1, device="cuda")}):
        with pytest.raises(E):
            tbe.tbe_adamw_step(plan, **HYPER, **kw)
    assert (p[0] == 1).all()


def pool_of(t):
    """The handle of the stream whose memory a tensor lies in."""
    at = t.data_ptr()
    return next(s["stream"] for s in torch.cuda.memory_snapshot() if s["address"] <= at < s["address"] + s["total_size"])


def churn():
    """Takes and writes freed memory of the current stream, of all sizes."""
    return [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(8, 24) for _ in range(4)]


@pytest.mark.parametrize("bits", [8, 32])
def test_steps_on_another_stream_keep_what_the_plan_holds(tbe, bits):
    """A plan that takes other gradients, or ends, while a step on another stream still reads its table of addresses,
    its old gradients and its states."""
    p, g = tensors(SIZES, "bf16", 0.05, 21), tensors(SIZES, "bf16", 1e-2, 22)
    q = [t.clone() for t in p]
    other = tbe.AdamWPlan(q, g, state_bits=bits)
    for step in (1, 2):
        tbe.tbe_adamw_step(other, **{**HYPER, "step": step})
    side = torch.cuda.Stream()
    plan = tbe.AdamWPlan(p, g, state_bits=bits)
    torch.cuda.synchronize()
    held = {plan._meta.data_ptr(), plan.exp_avg.data_ptr(), *(t.data_ptr() for t in g if t.numel())}
    with torch.cuda.stream(side):
        torch.cuda._sleep(60_000_000)  # the steps wait behind it
    tbe.tbe_adamw_step(plan, stream=side, **{**HYPER, "step": 1})
    fresh = [t.clone() for t in g]
    side.wait_stream(torch.cuda.current_stream())
    plan.rebind(grads=fresh)
    side.wait_stream(torch.cuda.current_stream())
    del g, other
    junk = churn()
    tbe.tbe_adamw_step(plan, stream=side, **{**HYPER, "step": 2})
    del plan, fresh
    junk += churn()
    assert not held & {t.data_ptr() for t in junk}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(p, q))


def test_a_plan_on_a_given_stream(tbe):
    """``stream=`` at the plan's creation: its table and states are that stream's memory, written in its order; so
    are the values of 8-bit states read on a given stream."""
    p, g = tensors(SIZES, "f32", 0.05, 23), tensors(SIZES, "f32", 1e-2, 24)
    q = [t.clone() for t in p]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    plan = tbe.AdamWPlan(p, g, state_bits=8, stream=side)
    tbe.tbe_adamw_step(plan, stream=side, **HYPER)
    values = tbe.tbe_adamw_state(plan, stream=side)
    torch.cuda.synchronize()
    for t in (plan._meta, plan.exp_avg, plan.exp_avg_sq, plan.exp_avg_scale, *values):
        assert pool_of(t) == side.cuda_stream
    same = tbe.AdamWPlan(q, g, state_bits=8)
    tbe.tbe_adamw_step(same, **HYPER)
    assert all(torch.equal(a, b) for a, b in zip((*p, *values), (*q, *tbe.tbe_adamw_state(same))))


@pytest.mark.parametrize("misaligned", [False, True])
def test_codes_of_tiny_moments(tbe, misaligned):
    """Second moments down to 2^-126, and first moments below 1e-34 beside second ones of zero: codes and scales of
    whole aligned blocks and of single elements equal the restatement's bit for bit, zeros among them."""
    rng = np.random.default_rng(13)
    size = 10.0 ** np.repeat(np.concatenate([np.arange(-11, -20, -0.5), np.arange(-32, -38, -0.5)]), BLOCK)
    values = (rng.standard_normal(len(size)) * size).astype(F)
    values[rng.random(len(size)) < 0.2] = 0
    values[3 * BLOCK:3 * BLOCK + 8] = 0  # nothing but zeros in a lane's eight elements
    n = len(values)
    g = torch.from_numpy(np.concatenate([[F(0)], values])).cuda()
    g = g[1:] if misaligned else g[1:].clone()
    zero = (np.zeros(n, np.int8), np.zeros(n, np.uint8), np.zeros(n // BLOCK, F), np.zeros(n // BLOCK, F))
    plan = plan8(tbe, [torch.zeros(n, device="cuda")], [g], zero)
    tbe.tbe_adamw_step(plan, **HYPER)
    _, v, *want = step8(values, *zero, HYPER)
    for name, got, exp in zip(("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"), codes(plan), want):
        assert np.array_equal(got, exp), f"{name}: {np.sum(got != exp)} differ"
    held = np.repeat(codes(plan)[3] > 0, BLOCK)
    assert (codes(plan)[1][held & (v > 0)] > 0).all()


@pytest.mark.parametrize("misaligned", [False, True])
def test_small_scales_stand_for_their_values(tbe, misaligned):
    """Scales down to the smallest normal number: what codes stand for, read back and in a step.  Bounds: five
    roundings of 2^-24, of which one may be of a number up to 2^-4 below the normal ones (2^-20), and half the
    smallest number (2^-150)."""
    rng = np.random.default_rng(14)
    scales = np.concatenate([2.0 ** np.arange(-125, -60.0), [2.0 ** -125 * 1.7, 1e-36, 1e-3, 1e30]]).astype(F)
    blocks = len(scales)
    n = blocks * BLOCK
    qm, qv = rng.integers(-127, 128, n).astype(np.int8), rng.integers(0, 256, n).astype(np.uint8)
    qm[::BLOCK], qv[::BLOCK] = 127, 255
    room = torch.zeros(n + 1, device="cuda")
    p, g = (room[1:], torch.zeros(n + 1, device="cuda")[1:]) if misaligned else (room[:n], torch.zeros(n, device="cuda"))
    plan = plan8(tbe, [p], [g], (qm, qv, scales, scales))
    s = np.repeat(scales, BLOCK).astype(np.float64)
    want_m = np.sign(qm) * (np.abs(qm) / 127.0) ** 2 * s
    want_v = (qv / 255.0) ** 4 * s
    for got, want in zip(tbe.tbe_adamw_state(plan), (want_m, want_v)):
        assert np.all(np.abs(f64(got) - want) <= 2.0 ** -19 * np.abs(want) + 2.0 ** -149)
    tbe.tbe_adamw_step(plan, **HYPER)  # no gradients: the largest moments shrink by the betas
    _, _, sm, sv = codes(plan)
    for got, beta in ((sm, HYPER["beta1"]), (sv, HYPER["beta2"])):
        want = beta * scales.astype(np.float64)
        on = want >= 1.001 * np.finfo(F).tiny
        assert np.all(np.abs(got[on] - want[on]) <= 2.0 ** -19 * want[on])


def test_a_missing_gradient_is_refused(tbe):
    """What a parameter that took no part in the loss has for its gradient: None."""
    p = [torch.ones(10, device="cuda"), torch.ones(4, device="cuda")]
    with pytest.raises(tbe.TBEError, match="gradient 1"):
        tbe.AdamWPlan(p, [torch.ones(10, device="cuda"), None])
    with pytest.raises(tbe.TBEError, match="parameter 0"):
        tbe.AdamWPlan([None, p[1]], p)
    plan = tbe.AdamWPlan(p, [torch.ones_like(t) for t in p])
    with pytest.raises(tbe.TBEError, match="gradient 0"):
        plan.rebind(grads=[None, p[1]])
    tbe.tbe_adamw_step(plan, **HYPER)  # still bound to what it had
    assert (p[0] != 1).all()


def test_rebind_takes_as_many_tensors_as_the_plan_has(tbe):
    p = [torch.ones(10, device="cuda"), torch.ones(4, device="cuda")]
    plan = tbe.AdamWPlan(p, [torch.ones_like(t) for t in p])
    for bad in (p[:1], p + p[:1]):
        with pytest.raises(tbe.TBEError, match="2 tensors"):
            plan.rebind(params=bad, grads=[torch.ones_like(t) for t in bad])
    tbe.tbe_adamw_step(plan, **HYPER)  # still bound to what it had
    assert all((t != 1).all() for t in p)


@pytest.mark.parametrize("kinds", [(("bf16", "f32"),), (("f32", "bf16"),), (("f16", "f32"),), (("f32", "f16"),),
                                   (("bf16", "f16"),), (("f16", "bf16"),),
                                   (("bf16", "f32"), ("f32", "f32"), ("f16", "f16"), ("f32", "bf16"))])
@pytest.mark.parametrize("misaligned", [False, True])
def test_8_bit_states_of_other_types(tbe, kinds, misaligned):
    """Parameters and gradients of unlike types, one pair of types for the list or mixed over it: codes and scales
    equal the restatement's bit for bit, weights within their bounds."""
    pk = [kinds[i % len(kinds)][0] for i in range(len(SIZES))]
    gk = [kinds[i % len(kinds)][1] for i in range(len(SIZES))]
    p = [tensors([n], k, 0.05, 40 + i, misaligned)[0] for i, (n, k) in enumerate(zip(SIZES, pk))]
    g = [tensors([n], k, 1e-3, 60 + i, misaligned)[0] for i, (n, k) in enumerate(zip(SIZES, gk))]
    st = state8(SIZES, 15)
    plan = plan8(tbe, p, g, st)
    for step in range(2):
        h = {**HYPER, "step": 50 + step}
        before = [f64(t) for t in p]
        new = step8(flat_padded(g, SIZES), *st, h)[2:]
        tbe.tbe_adamw_step(plan, **h)
        for name, got, want in zip(("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"), codes(plan), new):
            assert np.array_equal(got, want), f"{name}: {np.sum(got != want)} differ in step {step}"
        dm, dv = dequantise8(*st)
        for i, s in enumerate(slices(SIZES)):
            wp, _, _ = want64(before[i], f64(g[i]), dm[s].astype(np.float64), dv[s].astype(np.float64), h)
            near(f64(p[i]), wp, pk[i], f"weight {i}")
        st = new
