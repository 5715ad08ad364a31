"""Cross entropy over a catalogue: many tiles to a pair of blocks, many pieces of the vocabulary, gradients between other
tensors' columns.  The definition and its bounds are those of test_gpu_catalogue.py."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

import table_embedding_bags_gb300 as tbe  # noqa: E402
from test_gpu_catalogue import check, check_grads, definition, make  # noqa: E402
from test_more_operators_abi import Catalogue  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


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


def same_again(hidden, weights, labels, first, times=4, **more):
    for _ in range(times):
        got = tbe.tbe_catalogue_loss(hidden, weights, labels, **more)
        assert all(x is None and y is None or torch.equal(x, y) for x, y in zip(got, first))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,V,D", [(6000, 60000, 16), (300, 400_000, 64), (30_000, 300, 16)])
def test_many_tiles_to_a_pair(N, V, D, dtype):
    """A pair's places for tiles are used again many times, by short tiles."""
    hidden, weights, labels = make(N, V, D, TYPES[dtype], seed=21)
    tiles = -(-N // 256) * -(-V // 256)
    if V > 300:
        assert tiles >= 8 * 4 * torch.cuda.get_device_properties(0).multi_processor_count // 2
    got = tbe.tbe_catalogue_loss(hidden, weights, labels)
    check(got, definition(hidden, weights, labels), grads=False)
    same_again(hidden, weights, labels, got)
    grads = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True, grad_scale=512.0)
    check(grads, definition(hidden, weights, labels, grad_scale=512.0))
    same_again(hidden, weights, labels, grads, want_grad=True, grad_scale=512.0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("N,V,D", [(8000, 30_000, 96), (8192, 32_769, 64)])
def test_many_pieces_of_the_vocabulary(N, V, D, dtype):
    """Four pieces at least, the last one short: both buffers of g are written again behind what reads them, and one
    launch makes a piece while it multiplies the one before."""
    hidden, weights, labels = make(N, V, D, TYPES[dtype], seed=22)
    kind = tbe.TBE_F16 if dtype == "f16" else tbe.TBE_BF16
    a = Catalogue(hidden.data_ptr(), weights.data_ptr(), labels.data_ptr(), D, D, N, V, D, kind, 1.0)
    # two buffers of a piece's g are part of the workspace: were they a third of the vocabulary wide, it would be larger
    rows = -(-N // 256) * 256
    assert tbe.load_library().tbe_catalogue_workspace_bytes(ctypes.byref(a), 1) < 4 * rows * V // 3
    want = definition(hidden, weights, labels, grad_scale=512.0)
    got = tbe.tbe_catalogue_loss(hidden, weights, labels, want_grad=True, grad_scale=512.0)
    check(got, want)
    same_again(hidden, weights, labels, got, want_grad=True, grad_scale=512.0)
    dh, dw = tbe.tbe_catalogue_loss_backward(hidden, weights, labels, got.lse, grad_scale=512.0, token_loss=got.token_loss)
    check_grads(dh, dw, want)
