"""Table, linear attention and catalogue loss run together (GPU): a step's gradients against torch autograd in 64 bits,
and single events against the whole history.

bf16 rounds the rows' projection, the products and states of the attention, its outputs, the probabilities and every
gradient that passes on once each (2^-9 of their size, rarely adding up), so relative errors stay below a few of those
(0.03, as in the other example's test)."""

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
    import next_item as m

    return m


def plain_hidden(model, table, proj, ids, offsets):
    H, d = model.heads, model.head_dim
    q, k, v = (table[ids] @ proj).view(-1, 3, H, d).unbind(1)
    gamma = torch.exp(-model.decay.double())[:, None, None]
    out = []
    for s in range(len(offsets) - 1):
        state = torch.zeros(H, d, d, dtype=torch.float64, device="cuda")
        for t in range(offsets[s], offsets[s + 1]):
            state = gamma * state + k[t][:, :, None] * v[t][:, None, :]
            out.append(model.scale * torch.einsum("hi,hij->hj", q[t], state).reshape(-1))
    return torch.stack(out)


def test_gradients_of_one_step(example):
    model = example.Model(items=90, heads=3, head_dim=24, seed=3)
    ids, labels, offsets = example.make_histories(90, 7, seed=4, mean_length=9)
    table, proj = (p.double().clone().requires_grad_() for p in model.params)
    hidden = plain_hidden(model, table, proj, ids, offsets.tolist())
    want = torch.nn.functional.cross_entropy(hidden @ table.T, labels, ignore_index=-1)
    want.backward()
    got = model.gradients(ids, labels, offsets)
    assert abs(got.item() - want.item()) < 0.01 * want.item()
    for g, leaf, name in zip(model.grads, (table, proj), ("table", "projection")):
        rel = float((g.double() - leaf.grad).norm() / leaf.grad.norm())
        assert rel < 0.03, f"{name}: {rel}"


def test_it_runs(example):
    model, loss = example.train(steps=3, items=300, users=40)
    assert loss == loss and all(bool(p.isfinite().all()) for p in model.params) and model.steps == 3


def test_events_one_by_one(example):
    """A history read whole, and read up to its last three events, which then come one at a time."""
    model = example.Model(items=200, seed=5)
    users, n = 9, 40
    ids = torch.randint(0, 200, (users, n), device="cuda")
    offsets = lambda k: torch.arange(0, users * k + 1, k, device="cuda")  # noqa: E731
    whole, state = model.read(ids.reshape(-1), offsets(n))
    whole = whole.view(users, n, -1)
    _, running = model.read(ids[:, :n - 3].reshape(-1), offsets(n - 3))
    for t in range(n - 3, n):
        got = model.event(ids[:, t], running)
        assert float((got - whole[:, t]).norm() / whole[:, t].norm()) < 2.0**-7
    assert float((running - state).norm() / state.norm()) < 1e-5
