"""The example's training step: the operators run together, and its gradients (GPU).

The loss starts at log 2 (the model is its own reference) and falls.  One
step's gradients are compared with torch autograd in float64 through a plain
form of the same model: bf16 rounds the rows, the projection, the states, the
logits and their gradients once each (2^-9), so relative errors of the
gradients stay below a few of those (0.03)."""

import math
import os
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import sequence_preference as m

    return m


@pytest.mark.parametrize("state_bits", [32, 8])
def test_the_loss_falls(example, state_bits):
    losses = example.train(steps=40, items=500, pairs=24, state_bits=state_bits)
    assert abs(losses[0] - math.log(2)) < 1e-3
    assert losses[-1] < 0.3 * losses[0]
    assert all(math.isfinite(v) for v in losses)


def plain_loss(table, w_in, w_out, decay, ids, labels, offsets, ref, beta):
    H = decay.numel()
    x, r, g = (table[ids] @ w_in).split(H, dim=1)
    a = torch.exp(-8 * torch.nn.functional.softplus(decay) * torch.sigmoid(r))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(g) * x
    logps, off = [], offsets.tolist()
    for q in range(len(off) - 1):
        h, hs = torch.zeros(H, dtype=torch.float64, device="cuda"), []
        for t in range(off[q], off[q + 1]):
            h = a[t] * h + b[t]
            hs.append(h)
        lp = torch.log_softmax(torch.stack(hs) @ w_out, dim=1)
        y = labels[off[q]:off[q + 1]]
        keep = (y >= 0).nonzero()[:, 0]
        logps.append(lp[keep, y[keep]].sum())
    s = torch.stack(logps)
    P = len(logps) // 2
    d = beta * ((s[:P] - ref[:P]) - (s[P:] - ref[P:]))
    return torch.nn.functional.softplus(-d).mean()


def test_gradients_of_one_step(example):
    model = example.Model(items=60, dim=16, hidden=24, seed=3)
    ids, labels, offsets = example.make_pairs(60, 5, seed=4, mean_length=6)
    ref = torch.randn(10, device="cuda") * 3 - 12
    leaves = [t.double().clone().requires_grad_() for t in (model.table, *model.params)]
    loss = plain_loss(*leaves, ids, labels, offsets, ref.double(), 0.2)
    loss.backward()
    before = model.table.clone()
    got = model.step(ids, labels, offsets, ref, beta=0.2, table_rate=1.0)
    assert abs(float(got) - float(loss)) < 0.02 * float(loss) + 1e-3
    for g, leaf, name in zip(model.grads, leaves[1:], ("w_in", "w_out", "decay")):
        rel = float((g.double() - leaf.grad).norm() / leaf.grad.norm())
        assert rel < 0.03, f"{name}: {rel}"
    # exact row-wise Adagrad from zero momentum moves each row that was read by rate * g / (sqrt(mean g^2) + eps)
    G = leaves[0].grad
    moved = (before.double() - model.table.double())
    want = G / (G.square().mean(1, keepdim=True).sqrt() + 1e-6)
    rows = G.abs().amax(1) > 1e-4
    assert rows.any() and not moved[G.abs().amax(1) == 0].any()
    assert float((moved - want)[rows].norm() / want[rows].norm()) < 0.05
