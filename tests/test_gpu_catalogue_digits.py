"""Cross entropy over a catalogue where digits are easily lost: tokens that are all but learnt, and logits that are no
finite numbers.

Bounds.  A logit is D exact products summed in fp32 (a step of 2^-23 of the sum of magnitudes each, as sums may be cut
off): e = (D + 4) 2^-23 size.  With r = sum over the other rows of exp(x_v - x_y), a token's loss is log(1 + r) and its
label's share of the gradient -r / (1 + r).  Every term of r is off by at most 2 e of its size (two logits), 2^-22 (its
exponential, by five joins of partial sums as many again) and fewer than 64 additions of 2^-24 each: 2 e + 2^-17 in all,
of r's own size, however small it is.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import table_embedding_bags_gb300 as tbe  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def learnt(N, V, D, kind, seed, scale=1.0):
    """Tokens whose hidden rows are their label's row times 0.2 to 1: losses from about 1 down to 1e-9."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    weights = torch.randn(V, D, generator=gen, device="cuda").to(TYPES[kind])
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda")
    by = torch.linspace(0.2, 1.0, N, device="cuda")[:, None] / scale
    hidden = (weights[labels].float() * by).to(TYPES[kind])
    return hidden, weights, labels


def wanted(hidden, weights, labels, scale):
    """r, and how far it may be off relative to itself."""
    h, w = hidden.double(), weights.double()
    at = torch.arange(len(labels), device="cuda")
    x = scale * (h @ w.T)
    size = abs(scale) * (h.abs() @ w.abs().T).amax(1)
    p = torch.exp(x - x[at, labels][:, None])  # relative to the label's
    p[at, labels] = 0
    off = 2 * (h.shape[1] + 4) * 2.0**-23 * size + 2.0**-17
    return p, p.sum(1), off


CASES = [(64, 500, 64, 1.0), (64, 40000, 64, 1.0), (40, 33000, 100, -2.0), (300, 3000, 64, 0.5), (1, 32768, 48, 1.0)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("N,V,D,scale", CASES)
def test_losses_near_zero(N, V, D, scale, kind):
    hidden, weights, labels = learnt(N, V, D, kind, 1, scale)
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale)
    _, r, off = wanted(hidden, weights, labels, scale)
    want = torch.log1p(r)
    if N > 1:
        assert (want < 1e-5).sum() >= N // 8
    # the logarithm and the scale to natural units: 2^-22
    bound = (off + 2.0**-21) * want
    worst = ((got.token_loss.double() - want).abs() / bound).max().item()
    assert worst <= 1, worst
    assert abs(got.loss.item() - want.mean().item()) <= ((bound.mean() + 2.0**-20 * want.mean()).item())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("call", ["with the loss", "alone"])
@pytest.mark.parametrize("N,V,D,scale", CASES)
def test_gradients_of_tokens_that_are_nearly_learnt(N, V, D, scale, call, kind):
    """A bound of each entry of g by its own size, the label's among them: r / (1 + r), not 1."""
    hidden, weights, labels = learnt(N, V, D, kind, 2, scale)
    up = 2.0**12
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale, want_grad=True, grad_scale=up)
    dh, dw = got.dhidden, got.dweights
    if call == "alone":
        dh, dw = tbe.tbe_catalogue_loss_backward(hidden, weights, labels, got.lse, logit_scale=scale, grad_scale=up,
                                                 token_loss=got.token_loss)
    p, r, off = wanted(hidden, weights, labels, scale)
    g = p / (1 + r)[:, None]
    g[torch.arange(N, device="cuda"), labels] = -r / (1 + r)
    h, w = hidden.double(), weights.double()
    half = torch.finfo(TYPES[kind]).eps / 2
    # half a step of its type; what r is off by, once for itself and once for 1 + r; the log-sum's rounding (which stays
    # below 2^-22 of 64); the products' own sums; fp16's smallest numbers
    lse = torch.log1p(r) + scale * (h * w[labels]).sum(1)
    each = half + 2 * off[:, None] + 2.0**-21 * (1 + lse.abs())[:, None]
    f = up * abs(scale) / N
    for t, want, bound in ((dh, up * scale / N * (g @ w), f * ((each + V * 2.0**-23) * g.abs() + 2.0**-38) @ w.abs()),
                           (dw, up * scale / N * (g.T @ h), f * ((each + N * 2.0**-23) * g.abs() + 2.0**-38).T @ h.abs())):
        bound = bound + half * want.abs() + torch.finfo(t.dtype).smallest_normal * torch.finfo(t.dtype).eps
        worst = ((t.double() - want).abs() / bound).max().item()
        assert worst <= 1, worst


def by_formula(hidden, weights, labels, scale=1.0):
    x = scale * (hidden.double() @ weights.double().T)
    lse = torch.logsumexp(x, 1)
    return lse, lse - x[torch.arange(len(labels), device="cuda"), labels], torch.exp(x - lse[:, None])


def alike(a, b):
    """The same infinities and NaN in the same places."""
    a, b = a.double(), b.double()
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a == math.inf, b == math.inf) and torch.equal(a == -math.inf, b == -math.inf)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("V,scale", [(700, 1.0), (700, -0.5), (40000, 1.0), (40000, -0.5)])
def test_logits_that_are_no_finite_numbers(V, scale, kind):
    """Infinities in a row of the table (logits of either sign), in hidden rows, and NaN, as the formulas have them."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    N, D = 40, 64
    weights = torch.randn(V, D, generator=gen, device="cuda").to(TYPES[kind])
    hidden = torch.randn(N, D, generator=gen, device="cuda").to(TYPES[kind])
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda")
    weights[V // 3, 5] = math.inf
    labels[:6] = V // 3
    hidden[7, 5] = 0.0  # a logit of 0 * inf
    hidden[9] = math.inf  # logits of inf - inf
    hidden[11, 2] = math.nan
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale, want_grad=True)
    lse, loss, p = by_formula(hidden, weights, labels, scale)
    assert (lse == math.inf).any() and lse.isfinite().any() and lse.isnan().any()
    assert alike(got.lse, lse) and alike(got.token_loss, loss) and got.loss.isnan()
    ok = lse.isfinite() & loss.isfinite()
    assert torch.allclose(got.lse[ok].double(), lse[ok], rtol=1e-4) and torch.allclose(got.token_loss[ok].double(), loss[ok], rtol=1e-3, atol=1e-3)
    g = p.clone()
    g[torch.arange(N, device="cuda"), labels] -= 1
    assert alike(got.dhidden, (g @ weights.double()) * scale)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("V", [3, 700, 40000])
def test_logits_of_nothing(V, kind):
    """Rows whose logits are all -inf, or all but the label's, or where only the label's is -inf."""
    weights = torch.ones(V, 16, device="cuda").to(TYPES[kind])
    hidden = torch.zeros(2, 16, device="cuda").to(TYPES[kind])
    hidden[:, 0] = torch.tensor([1.0, 2.0])
    weights[:, 0] = -math.inf
    got = tbe.tbe_catalogue_loss(hidden, weights, torch.tensor([0, V - 1], device="cuda"))
    assert (got.lse == -math.inf).all() and got.token_loss.isnan().all()
    one = torch.full((V, 16), -math.inf, device="cuda").to(TYPES[kind])
    one[1] = 1
    h = torch.full((2, 16), 0.25, device="cuda").to(TYPES[kind])
    got = tbe.tbe_catalogue_loss(h, one, torch.tensor([1, 2], device="cuda"), want_grad=True)
    assert torch.allclose(got.lse, torch.full((2,), 4.0, device="cuda"), rtol=2.0**-22)
    assert got.token_loss[0] == 0 and got.token_loss[1] == math.inf and got.loss == math.inf
    assert torch.equal(got.dweights[1], (-h[0] + h[0] + h[1]) / 2) and torch.equal(got.dweights[2], -h[1] / 2)


@pytest.mark.parametrize("V", [3, 700, 40000])
def test_one_row_and_no_scale(V):
    gen = torch.Generator(device="cuda").manual_seed(4)
    weights, hidden = torch.randn(V, 32, generator=gen, device="cuda").bfloat16(), torch.randn(9, 32, generator=gen, device="cuda").bfloat16()
    labels = torch.randint(0, V, (9,), generator=gen, device="cuda")
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=0.0)
    assert torch.allclose(got.token_loss, torch.full((9,), math.log(V), device="cuda"), rtol=2.0**-20)
    one = tbe.tbe_catalogue_loss(hidden, weights[:1], torch.zeros_like(labels))
    x = (hidden.double() @ weights[:1].double().T).squeeze(1)
    assert not one.token_loss.any()
    assert torch.allclose(one.lse.double(), x, rtol=2.0**-18, atol=2.0**-18)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_one_row_has_no_gradient(kind):
    gen = torch.Generator(device="cuda").manual_seed(6)
    weights, hidden = (torch.randn(n, 32, generator=gen, device="cuda").to(TYPES[kind]) for n in (1, 9))
    got = tbe.tbe_catalogue_loss(hidden, weights, torch.zeros(9, dtype=torch.int64, device="cuda"), want_grad=True)
    assert not got.dhidden.any() and not got.dweights.any()


@pytest.mark.parametrize("N,V,D,scale", [(33, 40001, 72, -0.5), (64, 100003, 128, 1.0), (1, 32768, 64, 0.0)])
def test_few_tokens_in_half_precision(N, V, D, scale):
    from test_gpu_catalogue import check, definition, make

    hidden, weights, labels = make(N, V, D, torch.float16, seed=5, masked=0.2 if N > 1 else 0.0)
    labels[-1] = V - 1
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, logit_scale=scale, want_grad=True, grad_scale=256.0)
    check(got, definition(hidden, weights, labels, scale, 256.0))
