"""Preference loss over catalogue logits against its definition in 64 bits (GPU).

Bounds.  A row's log-sum adds exponentials whose arguments are rounded to
2^-23 of their size (at most 64 here) and whose values to 2^-21, in fp32
sums of depth below 2^7: its error is below 2^-16 + 2^-22 |lse|.  A sequence
adds its tokens' errors; d, the loss and the coefficients follow from there,
and dlogits adds half a unit of its type.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
SUBNORMAL = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tbe():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import table_embedding_bags_gb300 as m

    m.load_library()
    return m


def make(P, N, V, kind, seed, pad=0, lengths=None, ignore=0.2):
    rng = np.random.default_rng(seed)
    if lengths is None:
        lengths = rng.multinomial(N, rng.dirichlet(np.full(2 * P, 1.5)))
    logits = torch.from_numpy(rng.normal(0, 2, (N, V + pad)).astype(np.float32)).to("cuda", DT[kind])[:, :V]
    labels = rng.integers(0, V, N)
    labels[rng.random(N) < ignore] = -1
    return {"logits": logits, "labels": torch.from_numpy(labels).cuda(),
            "offsets": torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int64)).cuda(),
            "ref_logps": torch.from_numpy((-np.asarray(lengths) * np.log(V) + rng.normal(0, 3, 2 * P)).astype(np.float32)).cuda()}


def reference(d, beta, eps, scale=1.0):
    x = d["logits"].double().cpu().numpy()
    y, off = d["labels"].cpu().numpy(), d["offsets"].cpu().numpy()
    ref = d["ref_logps"].double().cpu().numpy()
    N, V = x.shape
    P = len(ref) // 2
    with np.errstate(divide="ignore", invalid="ignore"):
        top = x.max(1, keepdims=True)
        top = np.where(np.isneginf(top), 0, top)
        lse = (top + np.log(np.exp(x - top).sum(1, keepdims=True)))[:, 0]
    part = (y >= 0) & (y < V) & ~np.isneginf(lse)
    err = np.where(part, 2.0 ** -16 + 2.0 ** -22 * np.abs(np.where(part, lse, 0)), 0)
    lp = np.zeros(N)
    lp[part] = x[part, y[part]] - lse[part]
    s = np.array([lp[off[q]:off[q + 1]].sum() for q in range(2 * P)])
    es = np.array([err[off[q]:off[q + 1]].sum() + 2.0 ** -22 * np.abs(lp[off[q]:off[q + 1]]).sum() for q in range(2 * P)])
    d_ = beta * ((s[:P] - ref[:P]) - (s[P:] - ref[P:]))
    size = np.abs(s) + np.abs(ref)
    ed = abs(beta) * (es[:P] + es[P:]) + 2.0 ** -22 * abs(beta) * (size[:P] + size[P:])
    each = (1 - eps) * np.logaddexp(0, -d_) + eps * np.logaddexp(0, d_)
    out = {"loss": (each.mean(), ed.mean() + 2.0 ** -20 * np.abs(each).mean()), "seq_logps": (s, es), "margins": (d_, ed)}
    sig = lambda v: 1 / (1 + np.exp(-v))  # noqa: E731
    slope = beta / P * (eps * sig(d_) - (1 - eps) * sig(-d_))
    eslope = abs(beta) / P * (ed + 2.0 ** -20)
    where = np.repeat(np.arange(2 * P), np.diff(off))
    c = np.concatenate([slope, -slope])[where] * part * scale
    ec = np.concatenate([eslope, eslope])[where] * part * abs(scale)
    safe = np.where(part, lse, 0)[:, None]
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.where(part[:, None], np.exp(np.where(part[:, None], x, 0) - safe), 0)
    hot = np.zeros((N, V))
    hot[np.flatnonzero(part), y[part]] = 1
    g = c[:, None] * (hot - p)
    gap = np.minimum(np.abs(np.where(np.isfinite(x), x, 0) - safe), 1e30)
    eg = ec[:, None] * (hot + p) + np.abs(c)[:, None] * p * (2 * err[:, None] + 2.0 ** -22 * gap + 2.0 ** -19) \
        + 2.0 ** -23 * np.abs(c)[:, None] * hot
    out["dlogits"] = g, eg
    return out


def check(got, ref, kind, what):
    value, err = ref
    got = got.detach().double().cpu().numpy()
    tol = 2 * err + HALF_ULP[kind] * 1.01 * (np.abs(value) + err) + SUBNORMAL[kind] + 1e-37
    off = np.abs(got - value)
    assert np.all(off <= tol), f"{what}: worst {np.max(off / tol):.3g} of the bound"


def check_all(tbe, d, kind, beta=0.1, eps=0.05, scale=1.0):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = tbe.tbe_preference_loss(**d, beta=beta, label_smoothing=eps, want_grad=True, grad_scale=scale, dev_status=st)
    ref = reference(d, beta, eps, scale)
    for name in ("loss", "seq_logps", "margins"):
        check(getattr(r, name), ref[name], "f32", name)
    check(r.dlogits, ref["dlogits"], kind, "dlogits")
    assert r.dlogits.stride() == d["logits"].stride()
    return r, int(st)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("P,N,V,pad", [(1, 2, 1, 0), (1, 1, 7, 0), (3, 20, 50, 3), (40, 300, 1000, 0), (2, 9, 1025, 0),
                                       (300, 700, 130, 5), (5, 60, 5003, 0), (1, 5, 40_001, 7), (70, 1300, 2049, 0)])
def test_loss_and_gradient(tbe, P, N, V, pad, kind):
    """Rows by warp, by block and cut over blocks; odd widths (rows that start off a vector), empty sequences."""
    _, st = check_all(tbe, make(P, N, V, kind, P + V, pad), kind)
    assert st == 0


@pytest.mark.parametrize("beta,eps,scale", [(1.0, 0.0, 1.0), (0.5, 1.0, -3.0), (0.0, 0.3, 1.0), (-0.2, 0.5, 128.0)])
def test_parameters(tbe, beta, eps, scale):
    check_all(tbe, make(6, 80, 300, "f32", 4), "f32", beta, eps, scale)


def test_large_margins(tbe):
    """|d| in the hundreds: the loss grows linearly and the coefficient saturates, nothing overflows."""
    d = make(4, 40, 64, "f32", 5)
    d["ref_logps"] += torch.tensor([3e3, -3e3, 500, -500, 0, 0, 0, 0], device="cuda")
    r, _ = check_all(tbe, d, "f32", 1.0, 0.1)
    assert torch.isfinite(r.loss) and torch.isfinite(r.dlogits).all()


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("V", [200, 3000, 9000])
def test_masked_entries(tbe, V, kind):
    """Entries of -inf and of the type's lowest value: probability 0; a row whose entries are all -inf takes no
    part; a row of lowest values is an even choice."""
    d = make(3, 30, V, kind, 6, ignore=0.0)
    low = torch.finfo(DT[kind]).min
    x, y = d["logits"], d["labels"]
    keep = torch.nn.functional.one_hot(y, V).bool()
    x.masked_fill_((torch.rand(30, V, device="cuda") < 0.5) & ~keep, float("-inf"))
    x[4:8].masked_fill_((torch.rand(4, V, device="cuda") < 0.9) & ~keep[4:8], low)
    x[10] = float("-inf")
    x[11] = low
    x[12] = float("-inf")
    x[12, y[12]] = 1.5  # a single choice
    r, st = check_all(tbe, d, kind)
    assert st == 0
    assert not r.dlogits[10].any() and torch.isfinite(r.dlogits).all() and torch.isfinite(r.loss)
    assert torch.isneginf(r.lse[10])


def test_nan_stays_in_its_pair(tbe):
    d = make(4, 48, 1500, "f32", 7, lengths=[6] * 8, ignore=0.0)
    clean = tbe.tbe_preference_loss(**d, want_grad=True)
    d["logits"][8, 700] = float("nan")  # pair 1, preferred
    r = tbe.tbe_preference_loss(**d, want_grad=True)
    assert torch.isnan(r.loss) and torch.isnan(r.margins[1])
    rows = torch.tensor([n for n in range(48) if n // 6 not in (1, 5)], device="cuda")
    assert torch.equal(r.dlogits[rows], clean.dlogits[rows])
    assert torch.equal(r.margins[[0, 2, 3]], clean.margins[[0, 2, 3]])


def test_labels_outside_the_catalogue(tbe):
    d = make(2, 16, 90, "f32", 8, ignore=0.0)
    d["labels"][3], d["labels"][5], d["labels"][9] = 90, 1 << 40, -7
    r, st = check_all(tbe, d, "f32")
    assert st == tbe.TBE_DEV_BAD_INDEX
    assert not r.dlogits[[3, 5, 9]].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [100, 5000])
def test_in_place_backward_alone_and_other_strides(tbe, V, kind):
    d = make(3, 33, V, kind, 9, pad=8)
    r = tbe.tbe_preference_loss(**d, want_grad=True, grad_scale=2.0)
    only = tbe.tbe_preference_loss(**d)
    assert only.dlogits is None and torch.equal(only.loss, r.loss) and torch.equal(only.coef, r.coef)
    assert torch.equal(tbe.tbe_preference_loss_backward(**d, saved=only, grad_scale=2.0), r.dlogits)
    room = torch.full((33, V + 3), 9.0, device="cuda", dtype=DT[kind])  # rows that start elsewhere than the logits'
    tbe.tbe_preference_loss(**d, dlogits=room[:, 1:V + 1], grad_scale=2.0)
    assert torch.equal(room[:, 1:V + 1], r.dlogits) and (room[:, [0, V + 1, V + 2]] == 9).all()
    whole = d["logits"]
    tbe.tbe_preference_loss(**d, dlogits=whole, grad_scale=2.0)
    assert torch.equal(whole, r.dlogits)


def test_results_do_not_depend_on_timing_or_stream(tbe):
    d = make(50, 900, 7001, "bf16", 10)
    first = tbe.tbe_preference_loss(**d, want_grad=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        with torch.cuda.stream(side):
            r = tbe.tbe_preference_loss(**d, want_grad=True)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(first, r))


def test_gradient_against_differences(tbe):
    """<dlogits, v> against the central difference of the 64-bit loss along v."""
    d = make(3, 40, 70, "f32", 11)
    r = tbe.tbe_preference_loss(**d, beta=0.4, label_smoothing=0.1, want_grad=True)
    v = np.random.default_rng(1).standard_normal((40, 70))
    x = d["logits"].double()

    def loss(step):
        return reference({**d, "logits": x + step * torch.from_numpy(v).cuda()}, 0.4, 0.1)["loss"][0]

    want = (loss(1e-5) - loss(-1e-5)) / 2e-5
    g = r.dlogits.double().cpu().numpy()
    assert abs((g * v).sum() - want) <= 1e-5 * np.sqrt(((g * v) ** 2).sum()) + 1e-8


def test_more_than_2_to_31_logits(tbe):
    """The last pair of a batch of 2.3e9 logits equals a batch of its own."""
    V, N = 100_000, 23_000
    logits = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    logits[-4:] = torch.randn(4, V, device="cuda")
    labels = torch.full((N,), -1, device="cuda")
    labels[-4:] = torch.tensor([0, 5, V - 1, 77], device="cuda")
    offsets = torch.tensor([0, 0, N - 2, N - 2, N], device="cuda")  # preferred: none, N - 2; rejected: none, 2
    ref = torch.tensor([0.0, -20.0, 0.0, -25.0], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = tbe.tbe_preference_loss(logits, labels, offsets, ref, want_grad=True, dev_status=st)
    assert int(st) == 0
    small = {"logits": logits[-4:].clone(), "labels": labels[-4:].clone(),
             "offsets": torch.tensor([0, 0, 2, 2, 4], device="cuda"), "ref_logps": ref}
    want = reference(small, 0.1, 0.0)
    check(r.loss, want["loss"], "f32", "loss")
    check(r.dlogits[-4:], want["dlogits"], "bf16", "dlogits")
    assert not r.dlogits[:-4].any()


@pytest.mark.parametrize("offsets", [[1, 3, 6], [0, 3, 5], [0, 5, 4], [0, -2, 6], [0, 60, 6]])
def test_broken_offsets_are_reported(tbe, offsets):
    d = make(1, 6, 30, "f32", 12, lengths=[3, 3])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tbe.tbe_preference_loss(**{**d, "offsets": torch.tensor(offsets, device="cuda")}, want_grad=True, dev_status=st)
    assert int(st) & tbe.TBE_DEV_BAD_OFFSETS


def test_refusals(tbe):
    d = make(2, 10, 20, "f32", 13)
    bad = [("logits", d["logits"].cpu()), ("logits", d["logits"].double()), ("logits", d["logits"][:, :0]),
           ("logits", d["logits"].t()), ("logits", d["logits"][:1].expand(10, 20)), ("labels", d["labels"][:9]),
           ("labels", d["labels"].int()), ("offsets", d["offsets"][:4]), ("offsets", d["offsets"].int()),
           ("ref_logps", d["ref_logps"][:3]), ("ref_logps", d["ref_logps"].double()), ("beta", float("inf")),
           ("label_smoothing", 1.5), ("label_smoothing", float("nan")), ("dlogits", d["logits"].half()),
           ("dlogits", torch.empty(10, 19, device="cuda")), ("dev_status", torch.zeros(1, device="cuda"))]
    for key, value in bad:
        with pytest.raises(tbe.TBEError):
            tbe.tbe_preference_loss(**{**d, key: value}, want_grad=True)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_preference_loss(**d, want_grad=True, grad_scale=float("nan"))


@pytest.mark.parametrize("V", [100, 7001])
def test_calls_on_a_given_stream_keep_their_buffers(tbe, V):
    """``stream=``: results and workspace are the given stream's memory, whatever is allocated and written on the
    current stream behind the call."""
    data = [make(50, 900, V, "bf16", 30 + i) for i in range(2)]
    want = [tbe.tbe_preference_loss(**d, want_grad=True) for d in data]
    sides = [torch.cuda.Stream() for _ in data]
    torch.cuda.synchronize()
    got = []
    for d, side in zip(data, sides):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)  # the calls wait behind it, so that both streams' kernels run together
        grad = tbe.tbe_preference_loss(**d, want_grad=True, stream=side).dlogits  # the rest goes back at once
        r = tbe.tbe_preference_loss(**d, stream=side)
        got.append((grad, r, tbe.tbe_preference_loss_backward(**d, saved=r, stream=side)))
        junk = [torch.full((1 << k,), 255, dtype=torch.uint8, device="cuda") for k in range(8, 26) for _ in range(3)]
        del junk
    torch.cuda.synchronize()
    pools = torch.cuda.memory_snapshot()
    for w, (grad, r, alone), side in zip(want, got, sides):
        assert torch.equal(grad, w.dlogits) and torch.equal(alone, w.dlogits)
        assert torch.equal(r.loss, w.loss) and torch.equal(r.seq_logps, w.seq_logps) and torch.equal(r.coef, w.coef)
        for t in (grad, alone, r.loss):
            owner = [s["stream"] for s in pools if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
            assert owner == [side.cuda_stream]


@pytest.mark.parametrize("V", [90, 9000])
@pytest.mark.parametrize("eps,seq,want", [(0.0, 1, 0.0), (0.0, 0, np.inf), (1.0, 0, 0.0), (1.0, 1, np.inf),
                                          (0.1, 0, np.inf), (0.1, 1, np.inf)])
def test_masked_labels(tbe, V, eps, seq, want):
    """A label whose logit is -inf in one sequence of a pair: its margin is infinite, its loss 0 or infinite by the
    definition (a term of weight 0 counts as 0), the other pairs are as they were."""
    d = make(3, 60, V, "f32", 14, lengths=[10] * 6, ignore=0.0)
    clean = tbe.tbe_preference_loss(**d, label_smoothing=eps, want_grad=True)
    row = (seq * 3 + 1) * 10 + 4  # pair 1
    d["logits"][row, d["labels"][row]] = float("-inf")
    r = tbe.tbe_preference_loss(**d, label_smoothing=eps, want_grad=True)
    m = clean.margins.double().cpu().numpy()
    each = (1 - eps) * np.logaddexp(0, -m) + eps * np.logaddexp(0, m)
    each[1] = want
    assert float(r.margins[1]) == (-np.inf if seq == 0 else np.inf)
    assert torch.equal(r.margins[[0, 2]], clean.margins[[0, 2]])
    got = float(r.loss)
    assert got == np.inf if want == np.inf else abs(got - each.mean()) <= 2.0 ** -20 * each.mean()
    assert torch.isfinite(r.dlogits).all()
    other = torch.tensor([n for n in range(60) if n // 10 % 3 != 1], device="cuda")
    assert torch.equal(r.dlogits[other], clean.dlogits[other])


@pytest.mark.parametrize("kind,shift", [("f32", 1e4), ("f32", -3e5), ("f32", None), ("f16", None), ("bf16", None)])
@pytest.mark.parametrize("N,V", [(30, 200), (30, 9000), (40, 20_011), (200, 3000)])
def test_logits_far_from_zero(tbe, N, V, kind, shift):
    """Logits that share a large shift, and rows of nothing but the type's lowest value (shift None): probabilities
    do not depend on the size of the log-sum.  Bounds: exponentials and their sum 2^-16 in all (as above), arguments
    2^-22 of the distance to the log-sum, half a unit of the type; coefficients as the call returned them."""
    d = make(3, N, V, kind, 15, ignore=0.0)
    if shift is None:
        d["logits"][2::3] = torch.finfo(DT[kind]).min
    else:
        d["logits"] += shift
    r = tbe.tbe_preference_loss(**d, want_grad=True)
    x = d["logits"].double().cpu().numpy()
    top = x.max(1, keepdims=True)
    log_s = np.log(np.exp(x - top).sum(1, keepdims=True))
    gap = (x - top) - log_s
    y, off = d["labels"].cpu().numpy(), d["offsets"].cpu().numpy()
    hot = np.zeros_like(x)
    hot[np.arange(N), y] = 1
    lp = gap[np.arange(N), y]
    e = 2.0 ** -16 + 2.0 ** -22 * (np.abs(lp) + 2 * log_s[:, 0])
    s = np.array([lp[off[q]:off[q + 1]].sum() for q in range(6)])
    es = np.array([e[off[q]:off[q + 1]].sum() + 2.0 ** -22 * np.abs(lp[off[q]:off[q + 1]]).sum() for q in range(6)])
    check(r.seq_logps, (s, es / 2), "f32", "seq_logps")
    c = r.coef.double().cpu().numpy()[:, None]
    g = c * (hot - np.exp(gap))
    eg = np.abs(c) * (np.exp(gap) * (2.0 ** -16 + 2.0 ** -22 * np.abs(gap)) + 2.0 ** -22 * hot)
    check(r.dlogits, (g, eg / 2), kind, "dlogits")
    only = tbe.tbe_preference_loss(**d)
    assert torch.equal(tbe.tbe_preference_loss_backward(**d, saved=only), r.dlogits)


def test_gradient_of_a_narrow_view_of_a_wide_tensor(tbe):
    """The gradient's memory goes by the view, not by the tensor it was cut from."""
    wide = torch.randn(64, 1_000_000, device="cuda")
    d = make(2, 64, 100, "f32", 16)
    d["logits"] = wide[:, 5:105]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    r = tbe.tbe_preference_loss(**d, want_grad=True)
    alone = tbe.tbe_preference_loss_backward(**d, saved=r)
    assert torch.cuda.max_memory_allocated() - before < 1 << 20
    check(r.dlogits, reference(d, 0.1, 0.0)["dlogits"], "f32", "dlogits")
    assert torch.equal(alone, r.dlogits)


@pytest.mark.parametrize("kind", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("first,width", [(0, 4100), (1, 4100), (3, 4101), (5, 100_000)])
def test_new_gradients_lie_like_the_logits(tbe, kind, first, width):
    """Rows of a new gradient start at the same place of a 16-byte piece as the logits' rows, also where those start
    inside a row of a wider tensor."""
    d = make(2, 20, 4000, kind, 17)
    wide = torch.zeros(20, width, device="cuda", dtype=DT[kind])
    wide[:, first:first + 4000] = d["logits"]
    d["logits"] = wide[:, first:first + 4000]
    r, _ = check_all_but_strides(tbe, d, kind)
    alone = tbe.tbe_preference_loss_backward(**d, saved=tbe.tbe_preference_loss(**d, label_smoothing=0.05))
    assert torch.equal(alone, r.dlogits)
    for g in (r.dlogits, alone):
        for n in range(20):
            assert (g[n].data_ptr() - d["logits"][n].data_ptr()) % 16 == 0


def check_all_but_strides(tbe, d, kind):
    r = tbe.tbe_preference_loss(**d, label_smoothing=0.05, want_grad=True)
    ref = reference(d, 0.1, 0.05)
    for name in ("loss", "seq_logps", "margins"):
        check(getattr(r, name), ref[name], "f32", name)
    check(r.dlogits, ref["dlogits"], kind, "dlogits")
    return r, 0


@pytest.mark.parametrize("P,N,V,pad,kind", [(1, 6, 100_000, 0, "f32"), (1, 3, 99_999, 0, "f32"), (3, 40, 100_003, 5, "bf16"),
                                            (2, 13, 70_001, 0, "f16"), (5, 310, 16_390, 3, "bf16"),
                                            (4, 60, 20_000, 0, "f32"), (2, 300, 17_000, 1, "f16")])
def test_few_long_rows(tbe, P, N, V, pad, kind):
    """Batches above the small path's limit whose rows are cut over blocks of 256 threads, or just not."""
    _, st = check_all(tbe, make(P, N, V, kind, P + N, pad), kind)
    assert st == 0


@pytest.mark.parametrize("P,N,V,small", [(10, 256, 8, True), (10, 257, 8, False), (4, 256, 1024, True), (3, 16, 4000, True),
                                         (3, 17, 4000, False), (256, 250, 40, True), (257, 250, 40, False),
                                         (50, 20_000, 13, False), (5, 128, 2000, False)])
def test_one_cluster_takes_what_it_does_in_one_round(tbe, P, N, V, small):
    """Many short rows, or more than a few long ones, go to the kernels that use the whole GPU."""
    d = make(P, N, V, "f32", 18)
    tbe.trace_enable(True)
    try:
        tbe.tbe_preference_loss(**d, want_grad=True)
        stages = [name for name, _ in tbe.trace_read()]
    finally:
        tbe.trace_enable(False)
    assert ("preference_small" in stages) == small and ("preference_rows" in stages) != small
    check_all(tbe, d, "f32")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("V", [200, 9000])
def test_c_entry_of_the_gradient_from_lse_and_coef_alone(tbe, V, kind):
    """Without lse_low a row's probabilities carry the rounding of lse: 2^-24 of it (and as much again for the sum it
    is the log of), on top of the bounds of test_logits_far_from_zero."""
    import ctypes

    class Inputs(ctypes.Structure):
        _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64), ("labels", ctypes.c_void_p),
                    ("offsets", ctypes.c_void_p), ("ref_logps", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                    ("vocab", ctypes.c_int32), ("pairs", ctypes.c_int32), ("dtype", ctypes.c_int32),
                    ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float)]

    d = make(3, 30, V, kind, 19)
    d["logits"] += 100
    r = tbe.tbe_preference_loss(**d, want_grad=True)
    x = d["logits"]
    a = Inputs(x.data_ptr(), x.stride(0), d["labels"].data_ptr(), d["offsets"].data_ptr(), d["ref_logps"].data_ptr(), 30, V,
               3, {"f32": tbe.TBE_F32, "bf16": tbe.TBE_BF16}[kind], 0.1, 0.0)
    lib, stream = tbe.load_library(), torch.cuda.current_stream().cuda_stream
    lse, coef, low = r.lse.clone(), r.coef.clone(), r.lse_low.clone()
    got, same = torch.full_like(x, 7), torch.full_like(x, 7)
    assert lib.tbe_preference_loss_backward(ctypes.byref(a), lse.data_ptr(), coef.data_ptr(), 1.0, got.data_ptr(),
                                            x.stride(0), stream) == tbe.TBE_OK
    assert lib.tbe_preference_loss_backward_low(ctypes.byref(a), lse.data_ptr(), low.data_ptr(), coef.data_ptr(), 1.0,
                                                same.data_ptr(), x.stride(0), stream) == tbe.TBE_OK
    assert torch.equal(same, r.dlogits)
    z = x.double()
    gap = (z - torch.logsumexp(z, 1, keepdim=True)).cpu().numpy()
    y = d["labels"].cpu().numpy()
    hot = np.zeros_like(gap)
    hot[np.flatnonzero(y >= 0), y[y >= 0]] = 1
    c = coef.double().cpu().numpy()[:, None]
    e = np.abs(c) * (np.exp(gap) * (2.0 ** -16 + 2.0 ** -22 * np.abs(gap) + 2.0 ** -23 * 110) + 2.0 ** -22 * hot)
    check(got, (c * (hot - np.exp(gap)), e / 2), kind, "dlogits")
