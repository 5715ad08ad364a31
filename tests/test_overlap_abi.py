"""Outputs that share memory with inputs, or with each other, are refused by the C entries of linear attention and the
catalogue loss (CPU only: host memory stands in for the device's; no call here reaches a launch)."""

import ctypes
import itertools

import pytest

import table_embedding_bags_gb300 as tbe
from table_embedding_bags_gb300.build import build
from test_more_operators_abi import Catalogue, Linear, LinearGrads

INVALID = tbe.TBE_ERR_INVALID_ARG


@pytest.fixture(scope="module")
def lib():
    build()
    return tbe.load_library()


@pytest.fixture(scope="module")
def base():
    room = (ctypes.c_uint8 * (4 << 20))()
    at = (ctypes.addressof(room) + 255) // 256 * 256
    yield lambda n: at + n * 131072
    del room


N, H, D, S = 64, 4, 16, 64  # rows of 16 elements, 8 KB in all
STATE = 4 * S * H * D * D


def linear(base, q=None, k=None, v=None, stride=H * D, head=D, s0=None):
    return Linear(N, S, H, D, tbe.TBE_BF16, 0, 1.0, q or base(0), k or base(1), v or base(2), stride, stride, stride, head, head,
                  head, base(3), base(4), s0)


def forward(lib, a, o, stride=H * D, head=D, last=None):
    return lib.tbe_linear_attention(ctypes.byref(a), o, stride, head, last, None, 0, None, None)


def backward(lib, a, do, dq, dk, dv, stride=H * D, head=D, ds_last=None, ds0=None):
    g = LinearGrads(dq, dk, dv, stride, stride, stride, head, head, head, ds0)
    return lib.tbe_linear_attention_backward(ctypes.byref(a), do, H * D, D, ds_last, ctypes.byref(g), None, 0, None, None)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("by", [0, 2, 30, 2 * H * D, 2 * (N * H * D - 1), -2, -2 * (N * H * D - 1)])
def test_output_over_an_input(lib, base, which, by):
    assert forward(lib, linear(base), base(which) + by + (0 if by >= 0 else 0)) == INVALID
    for grads in itertools.permutations([base(5), base(6), base(which) + by]):
        assert backward(lib, linear(base), base(7), *grads) == INVALID
    one = linear(base)
    assert lib.tbe_linear_attention_step(ctypes.byref(one), base(8), base(which) + by, H * D, D, None) == INVALID


def test_output_over_other_inputs(lib, base):
    s0 = base(8)
    a = linear(base, s0=s0)
    for at in (base(3), base(4) + 8 * S, s0 + STATE - 2):  # decay, offsets, states
        assert forward(lib, a, at) == INVALID
        assert backward(lib, a, base(7), base(5), at, base(6)) == INVALID
    assert backward(lib, linear(base), base(7), base(5), base(6), base(7) + 64) == INVALID  # dO
    assert backward(lib, linear(base), base(7), base(5), base(6), base(20), ds_last=base(20)) == INVALID
    assert lib.tbe_linear_attention_step(ctypes.byref(linear(base)), s0, s0 + 64, H * D, D, None) == INVALID
    assert lib.tbe_linear_attention_step(ctypes.byref(linear(base)), base(1) - 64, base(5), H * D, D, None) == INVALID
    for state in (base(0), base(5), base(4)):  # last states over q, o and offsets
        assert forward(lib, linear(base), base(5), last=state) == INVALID
    for state in (base(7), base(5), base(6) - STATE + 4):
        assert backward(lib, linear(base), base(7), base(5), base(6), base(20), ds0=state) == INVALID


def test_outputs_over_each_other(lib, base):
    for grads in ((5, 5, 6), (5, 6, 5), (6, 5, 5)):
        assert backward(lib, linear(base), base(7), *(base(n) for n in grads)) == INVALID


def test_rows_that_lie_between_others(lib, base):
    """Slices of one buffer: refused where any element is shared, whatever the order of tokens and heads."""
    wide = 4 * H * D
    q, k, v = (base(0) + 2 * n * H * D for n in range(3))
    a = linear(base, q, k, v, stride=wide)
    for o in (q + 2 * D, k, v + 2 * (H - 1) * D, v + 30, v + 2 * wide, base(0) + 2 * 4 * H * D - 2):
        assert forward(lib, a, o, stride=wide) == INVALID
    # heads that lie between the keys' heads, one element too far
    a = linear(base, base(0), base(0) + 2 * D, base(0) + 4 * D, stride=4 * H * D, head=4 * D)
    for by in (3 * D + 1, 3 * D - 1):
        assert forward(lib, a, base(0) + 2 * by, stride=4 * H * D, head=4 * D) == INVALID
    # heads first
    a = linear(base, stride=D, head=N * D)
    assert forward(lib, a, base(1) + 2 * N * D, stride=D, head=N * D) == INVALID
    assert forward(lib, a, base(1), stride=H * D, head=D) == INVALID


def catalogue(lib, base, dh, dw, dhs, dws, hidden=None, hs=32, labels=None):
    a = Catalogue(hidden or base(0), base(1), labels or base(2), hs, 32, 50, 60, 32, tbe.TBE_F16, 1.0)
    f = base(3)
    return lib.tbe_catalogue_loss(ctypes.byref(a), f, f, f, dh, dhs, dw, dws, 1.0, base(8), 16, None, None)


def test_catalogue_gradients_between_other_rows(lib, base):
    """Columns of one wider tensor are no overlap (the workspace given here is too small: that is what is found next)."""
    passed = tbe.TBE_ERR_WORKSPACE
    assert catalogue(lib, base, base(0) + 64, base(5), 64, 32, hs=64) == passed
    assert catalogue(lib, base, base(5), base(5) + 64, 64, 64) == passed
    for by in (62, 66, 0, 130):
        assert catalogue(lib, base, base(0) + by, base(5), 64, 32, hs=64) == INVALID
    assert catalogue(lib, base, base(5), base(5) + 62, 64, 64) == INVALID
    assert catalogue(lib, base, base(2) + 398, base(5), 32, 32) == INVALID  # the last label
    assert catalogue(lib, base, base(2) + 400, base(5), 32, 32) == passed


def test_catalogue_gradients_on_their_own(lib, base):
    a = Catalogue(base(0), base(1), base(2), 32, 32, 50, 60, 32, tbe.TBE_F16, 1.0)
    full = lambda lse, loss, dh, dw: lib.tbe_catalogue_loss_backward_full(  # noqa: E731
        ctypes.byref(a), lse, loss, dh, 32, dw, 32, 1.0, base(8), 16, None, None)
    assert full(None, base(4), base(5), base(6)) == INVALID and full(base(3), base(4), None, base(6)) == INVALID
    assert full(base(3), None, base(5), base(6)) == tbe.TBE_ERR_WORKSPACE
    assert full(base(3), base(4), base(5), base(6)) == tbe.TBE_ERR_WORKSPACE
    assert full(base(5), base(4), base(5), base(6)) == INVALID and full(base(3), base(6), base(5), base(6)) == INVALID
