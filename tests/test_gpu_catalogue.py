"""Cross entropy over a catalogue's table against its definition in 64 bits."""

import math

import pytest

torch = pytest.importorskip("torch")

import table_embedding_bags_gb300 as tbe  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def make(N, V, D, dtype, seed=0, hidden_pad=0, weights_pad=0, masked=0.1, spread=2.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    hidden = normal(N, D + hidden_pad).to(dtype)[:, hidden_pad // 2:hidden_pad // 2 + D]
    weights = (normal(V, D + weights_pad) * spread / math.sqrt(D)).to(dtype)[:, weights_pad // 2:weights_pad // 2 + D]
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda")
    labels[torch.rand(N, generator=gen, device="cuda") < masked] = -1
    return hidden, weights, labels


def definition(hidden, weights, labels, logit_scale=1.0, grad_scale=1.0):
    """The formulas in 64 bits, and how far the outputs may be off: see check()."""
    rows = torch.nonzero((labels >= 0) & (labels < weights.shape[0])).squeeze(1)
    h, w, y = hidden[rows].double(), weights.double(), labels[rows]
    x = logit_scale * (h @ w.T)
    size = abs(logit_scale) * (h.abs() @ w.abs().T)
    lse = torch.logsumexp(x, 1)
    at = torch.arange(len(rows), device="cuda")
    loss = lse - x[at, y]
    count = max(1, len(rows))
    p = torch.exp(x - lse[:, None])
    g = p.clone()
    g[at, y] -= 1
    f = grad_scale * logit_scale / count
    N = hidden.shape[0]
    r = {"rows": rows, "lse": torch.zeros(N, dtype=torch.float64, device="cuda").index_copy(0, rows, lse),
         "token_loss": torch.zeros(N, dtype=torch.float64, device="cuda").index_copy(0, rows, loss),
         "loss": loss.sum() / count}
    r["dhidden"] = torch.zeros(N, h.shape[1], dtype=torch.float64, device="cuda").index_copy(0, rows, f * (g @ w))
    r["dweights"] = f * (g.T @ h)
    # a logit: D exact products summed in fp32 (a step of 2^-23 each allows for truncation), then a few roundings
    dx = (h.shape[1] + 4) * 2.0**-23 * (size.amax(1) if len(rows) else size.sum(1)) + 2.0**-22 * (1 + lse.abs())
    half = torch.finfo(hidden.dtype).eps / 2
    # g: half a step of its type, the logit's error times p; a floor where fp16 (held 2^14 times larger) is subnormal
    err = half * g.abs() + 4 * dx[:, None] * p + 2.0**-38
    terms = len(rows) + weights.shape[0]
    err = err + g.abs() * terms * 2.0**-23  # the sum's own
    r["tol_x"] = torch.zeros(N, dtype=torch.float64, device="cuda").index_copy(0, rows, 2 * dx)
    f = abs(f)
    r["tol_dhidden"] = torch.zeros_like(r["dhidden"]).index_copy(0, rows, f * (err @ w.abs()))
    r["tol_dweights"] = f * (err.T @ h.abs())
    return r


def check(got, want, grads=True):
    assert got.lse.isfinite().all()
    assert ((got.lse.double() - want["lse"]).abs() <= want["tol_x"]).all()
    assert ((got.token_loss.double() - want["token_loss"]).abs() <= want["tol_x"]).all()
    n = max(1, len(want["rows"]))
    # (the mean of so many fp32 numbers, summed by 8 and then by 32 lanes)
    assert abs(got.loss.item() - want["loss"].item()) <= (want["tol_x"].sum() / n + 2.0**-20 * (want["token_loss"].abs().sum() / n)).item()
    if not grads:
        assert got.dhidden is None and got.dweights is None
        return
    check_grads(got.dhidden, got.dweights, want)


def check_grads(dhidden, dweights, want):
    for name, t in (("dhidden", dhidden), ("dweights", dweights)):
        w = want[name]
        tiny = torch.finfo(t.dtype).smallest_normal * torch.finfo(t.dtype).eps
        tol = want["tol_" + name] + torch.finfo(t.dtype).eps / 2 * w.abs() + tiny
        off = (t.double() - w).abs()
        assert (off <= tol).all(), (name, (off / tol).max().item())


@pytest.mark.parametrize("N,V,D,dtype,kind", [
    (1, 1, 1, "bf16", {}),
    (1, 50, 16, "f16", {"masked": 0.0}),
    (8, 1000, 64, "bf16", {}),
    (129, 257, 65, "f16", {}),
    (128, 256, 64, "bf16", {"masked": 0.0}),
    (300, 1000, 128, "f16", {"hidden_pad": 24}),
    (517, 3001, 72, "bf16", {"weights_pad": 8, "hidden_pad": 2}),
    (1000, 777, 250, "f16", {"hidden_pad": 13}),
    (640, 5000, 257, "bf16", {"weights_pad": 3}),
    (2500, 4097, 320, "bf16", {}),
    (40, 30011, 512, "f16", {}),
    (1500, 130, 600, "bf16", {}),
])
def test_loss_and_gradients(N, V, D, dtype, kind):
    hidden, weights, labels = make(N, V, D, TYPES[dtype], seed=N + V, **kind)
    scale = 1.0 if dtype == "bf16" else 1024.0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=0.7, want_grad=True, grad_scale=scale,
                                 dev_status=status)
    want = definition(hidden, weights, labels, 0.7, scale)
    assert status.item() == 0
    check(got, want)
    assert (got.dhidden[labels < 0] == 0).all()
    alone = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=0.7)
    check(alone, want, grads=False)
    assert torch.equal(alone.token_loss, got.token_loss) and torch.equal(alone.loss, got.loss)
    dh, dw = tbe.tbe_catalogue_loss_backward(hidden, weights, labels, got.lse, logit_scale=0.7, grad_scale=scale)
    check_grads(dh, dw, want)


def test_more_than_one_piece_of_the_vocabulary():
    # 4,096 rows take the vocabulary by 8,192
    hidden, weights, labels = make(4000, 20000, 96, torch.bfloat16, seed=3)
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    check(got, definition(hidden, weights, labels))
    again = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    assert torch.equal(got.dhidden, again.dhidden) and torch.equal(got.dweights, again.dweights)
    assert torch.equal(got.token_loss, again.token_loss) and torch.equal(got.loss, again.loss)


# ---------------------------------------------------------------------------
# values and sizes at the edges
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -65504.0])
def test_rows_without_a_label_are_not_looked_at(dtype, value):
    hidden, weights, labels = make(300, 700, 80, TYPES[dtype], seed=5, masked=0.4)
    want = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    hidden[labels < 0] = value
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert not got.dhidden[labels < 0].any() and not got.lse[labels < 0].any()


@pytest.mark.parametrize("N,V,D", [(1, 5, 3), (300, 700, 64)])
def test_no_token_takes_part(N, V, D):
    hidden, weights, labels = make(N, V, D, torch.bfloat16)
    hidden.fill_(float("nan"))
    labels.fill_(-100)
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    assert all(not t.any() for t in got)
    dh, dw = tbe.tbe_catalogue_loss_backward(hidden, weights, labels, got.lse)
    assert not dh.any() and not dw.any()


def test_labels_outside_the_table_are_reported():
    hidden, weights, labels = make(200, 90, 64, torch.bfloat16, seed=6)
    labels[[0, 7, 150]] = torch.tensor([90, 1 << 40, 91], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True, dev_status=status)
    assert status.item() == tbe.TBE_DEV_BAD_INDEX
    check(got, definition(hidden, weights, labels))


@pytest.mark.parametrize("scale", [-0.5, 0.0, 30.0])
def test_logit_scale(scale):
    hidden, weights, labels = make(150, 1000, 64, torch.bfloat16, seed=7)
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale, want_grad=True)
    check(got, definition(hidden, weights, labels, scale))


def test_a_logit_that_stands_out():
    """Losses near 0, where the log-sum all but equals the label's logit, keep their digits."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    weights = torch.randn(500, 64, generator=gen, device="cuda").bfloat16()
    labels = torch.randint(0, 500, (64,), generator=gen, device="cuda")
    hidden = (weights[labels].float() * 0.3).bfloat16()
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    want = definition(hidden, weights, labels)
    check(got, want)
    small = want["token_loss"] < 1e-3
    assert small.any()
    # The sum is 1 + s: some 16 additions at 1 (8 in a chunk of 32, 4 chunks, halves, tiles) of 2^-24 each, the label's own
    # exponential (2^-22) and the logarithm (2^-23) add up to less than 2^-19; the logits' errors (2^-20 of sizes below
    # 2^6) move s by 2^-14 of it.  Against that, 2^-24 of the log-sums of 10 to 40 would be up to 2^-18.
    off = (got.token_loss.double() - want["token_loss"]).abs()
    assert (off <= 2.0**-19 + 2.0**-13 * want["token_loss"])[small].all()


def test_what_is_no_number_in_a_row_that_takes_part():
    hidden, weights, labels = make(300, 400, 64, torch.bfloat16, seed=9, masked=0.0)
    hidden[17, 3] = float("nan")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    assert got.loss.isnan() and got.token_loss[17].isnan() and got.dhidden[17].isnan().all()
    others = torch.arange(300, device="cuda") != 17
    assert got.token_loss[others].isfinite().all() and got.dhidden[others].isfinite().all() and got.dweights.isnan().any()


@pytest.mark.parametrize("N,V,D", [(20000, 50, 8), (3, 70000, 24), (255, 255, 128), (257, 513, 192), (64, 2048, 1024)])
def test_long_and_flat(N, V, D):
    hidden, weights, labels = make(N, V, D, torch.bfloat16, seed=10)
    check(tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True), definition(hidden, weights, labels))


@pytest.mark.parametrize("D,pad", [(64, 0), (96, 5), (33, 1)])
def test_given_gradients_and_what_lies_between(D, pad):
    hidden, weights, labels = make(200, 300, D, torch.float16, seed=11)
    want = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True, grad_scale=256.0)
    dh = torch.full((200, D + 2 * pad), 7.0, dtype=torch.float16, device="cuda")
    dw = torch.full((300, D + 3 * pad), 7.0, dtype=torch.float16, device="cuda")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, grad_scale=256.0, dhidden=dh[:, pad:pad + D],
                                 dweights=dw[:, 2 * pad:2 * pad + D])
    assert torch.equal(got.dhidden, want.dhidden) and torch.equal(got.dweights, want.dweights)
    assert (dh[:, :pad] == 7).all() and (dh[:, pad + D:] == 7).all()
    assert (dw[:, :2 * pad] == 7).all() and (dw[:, 2 * pad + D:] == 7).all()


def test_streams_and_graphs():
    a, b = make(500, 3000, 64, torch.bfloat16, seed=12), make(500, 3000, 64, torch.bfloat16, seed=13, masked=0.5)
    want = [tbe.tbe_catalogue_loss(*x, want_grad=True) for x in (a, b)]

    def same(x, y):
        assert all(torch.equal(p, q) for p, q in zip(x, y))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        there = tbe.tbe_catalogue_loss(*b, want_grad=True)
    here = tbe.tbe_catalogue_loss(*a, want_grad=True)
    torch.cuda.current_stream().wait_stream(side)
    same(here, want[0])
    same(there, want[1])
    given = tbe.tbe_catalogue_loss(*b, want_grad=True, stream=side)
    side.synchronize()
    same(given, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = tbe.tbe_catalogue_loss(*a, want_grad=True)
    graph.replay()
    same(captured, want[0])
    for x, y in zip(a, b):  # other rows take part
        x.copy_(y)
    graph.replay()
    same(captured, want[1])


def test_refusals():
    hidden, weights, labels = make(50, 60, 64, torch.bfloat16)

    def refused(h=hidden, w=weights, y=labels, **more):
        with pytest.raises(tbe.TBEError):
            tbe.tbe_catalogue_loss(h, w, y, want_grad=True, **more)

    refused(h=hidden.cpu())
    refused(h=hidden.float(), w=weights.float())
    refused(h=hidden.half())
    refused(h=hidden[:, :32])
    refused(h=hidden[:0], y=labels[:0])
    refused(h=hidden.view(50, 8, 8))
    refused(w=weights[:0])
    refused(w=weights.cpu())
    refused(w=weights.t().contiguous().t())
    refused(y=labels.int())
    refused(y=labels[:-1])
    refused(y=labels.cpu())
    refused(logit_scale=float("nan"))
    refused(grad_scale=float("inf"))
    refused(dhidden=hidden)
    refused(dweights=weights)
    refused(dhidden=torch.empty(50, 64, device="cuda"))
    refused(dweights=torch.empty(60, 63, dtype=torch.bfloat16, device="cuda"))
    room = torch.empty(200, 64, dtype=torch.bfloat16, device="cuda")
    refused(dhidden=room[:50], dweights=room[40:100])
    refused(dev_status=torch.zeros(1, device="cuda"))
    with pytest.raises(tbe.TBEError):
        tbe.tbe_catalogue_loss_backward(hidden, weights, labels, None)
    with pytest.raises(tbe.TBEError):
        tbe.tbe_catalogue_loss_backward(hidden, weights, labels, torch.zeros(49, device="cuda"))


@pytest.mark.parametrize("N,V,D,scale", [(1, 32768, 64, 1.0), (33, 40001, 72, -0.5), (64, 33000, 200, 20.0), (64, 100003, 128, 1.0),
                                         (65, 33000, 64, 1.0), (32, 32767, 64, 1.0)])
def test_few_tokens_over_many_rows(N, V, D, scale):
    """Up to 64 tokens over 32,768 rows or more: the log-sums of a token are kept by many threads, whose own maxima need
    not be the largest."""
    hidden, weights, labels = make(N, V, D, torch.bfloat16, seed=14, masked=0.2 if N > 1 else 0.0)
    labels[-1] = V - 1
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale, want_grad=True)
    check(got, definition(hidden, weights, labels, scale))
    alone = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale)
    assert torch.equal(alone.loss, got.loss) and torch.equal(alone.lse, got.lse)


def test_few_tokens_and_logits_that_grow():
    """Each tile's logits lie far above those before it."""
    gen = torch.Generator(device="cuda").manual_seed(15)
    weights = torch.randn(40000, 64, generator=gen, device="cuda") * torch.linspace(0.01, 3, 40000, device="cuda")[:, None]
    hidden = torch.randn(20, 64, generator=gen, device="cuda").bfloat16()
    labels = torch.randint(0, 40000, (20,), generator=gen, device="cuda")
    for w in (weights.bfloat16(), weights.flip(0).bfloat16()):
        check(tbe.tbe_catalogue_loss(hidden, w, labels, want_grad=True), definition(hidden, w, labels))


def test_few_tokens_what_is_no_number():
    hidden, weights, labels = make(40, 40000, 64, torch.bfloat16, seed=16, masked=0.0)
    hidden[7] = float("nan")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels)
    others = torch.arange(40, device="cuda") != 7
    assert got.token_loss[7].isnan() and got.loss.isnan() and got.token_loss[others].isfinite().all()
