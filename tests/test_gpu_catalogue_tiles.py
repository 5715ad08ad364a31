"""Cross entropy over a catalogue: gradients between other tensors' columns."""

import pytest

torch = pytest.importorskip("torch")

import table_embedding_bags_gb300 as tbe  # noqa: E402
from test_gpu_catalogue import make  # noqa: E402

pytestmark = pytest.mark.gpu


def test_gradients_between_other_columns():
    hidden, weights, labels = make(300, 700, 64, torch.bfloat16, seed=20)
    want = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True)
    rows, table = (torch.full((n, 192), 7.0, dtype=torch.bfloat16, device="cuda") for n in (300, 700))
    rows[:, :64], table[:, 128:] = hidden, weights
    got = tbe.tbe_catalogue_loss(rows[:, :64], table[:, 128:], labels, dhidden=rows[:, 64:128], dweights=table[:, :64])
    assert torch.equal(got.dhidden, want.dhidden) and torch.equal(got.dweights, want.dweights)
    assert torch.equal(rows[:, :64], hidden) and torch.equal(table[:, 128:], weights)
    assert (rows[:, 128:] == 7).all() and (table[:, 64:128] == 7).all()
    with pytest.raises(tbe.TBEError):
        tbe.tbe_catalogue_loss(rows[:, :64], table[:, 128:], labels, dhidden=rows[:, 63:127], dweights=table[:, :64])
