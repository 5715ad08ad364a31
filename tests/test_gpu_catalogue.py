"""Cross entropy over a catalogue's table against its definition in 64 bits."""

import math

import pytest
import torch

import table_embedding_bags_gb300 as tbe

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
