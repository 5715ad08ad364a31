"""Refusals of the C entries of linear attention and the catalogue loss, before anything is launched (CPU only: host
memory stands in for the device's; every call here is refused)."""

import ctypes

import pytest

import table_embedding_bags_gb300 as tbe
from table_embedding_bags_gb300.build import build

I64, I32, P, F = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_float


class Linear(ctypes.Structure):
    _fields_ = [("tokens", I64), ("sequences", I32), ("heads", I32), ("head_dim", I32), ("dtype", I32), ("offsets_i32", I32),
                ("scale", F), ("q", P), ("k", P), ("v", P), ("q_stride", I64), ("k_stride", I64), ("v_stride", I64),
                ("q_head_stride", I64), ("k_head_stride", I64), ("v_head_stride", I64), ("decay", P), ("offsets", P), ("s0", P)]


class LinearGrads(ctypes.Structure):
    _fields_ = [("dq", P), ("dk", P), ("dv", P), ("dq_stride", I64), ("dk_stride", I64), ("dv_stride", I64),
                ("dq_head_stride", I64), ("dk_head_stride", I64), ("dv_head_stride", I64), ("ds0", P)]


class Catalogue(ctypes.Structure):
    _fields_ = [("hidden", P), ("weights", P), ("labels", P), ("hidden_stride", I64), ("weights_stride", I64), ("tokens", I64),
                ("vocab", I32), ("width", I32), ("dtype", I32), ("logit_scale", F)]


@pytest.fixture(scope="module")
def lib():
    build()
    return tbe.load_library()


@pytest.fixture(scope="module")
def room():
    return (ctypes.c_uint8 * (1 << 20))()


def base(room, n):
    return (ctypes.addressof(room) + 255) // 256 * 256 + n * 65536


def linear(room, **other):
    a = dict(tokens=64, sequences=2, heads=2, head_dim=16, dtype=tbe.TBE_BF16, offsets_i32=0, scale=1.0, q=base(room, 0),
             k=base(room, 1), v=base(room, 2), q_stride=32, k_stride=32, v_stride=32, q_head_stride=16, k_head_stride=16,
             v_head_stride=16, decay=base(room, 3), offsets=base(room, 4), s0=None)
    a.update(other)
    return Linear(*[a[n] for n, _ in Linear._fields_])


INVALID, UNSUPPORTED = tbe.TBE_ERR_INVALID_ARG, tbe.TBE_ERR_UNSUPPORTED


@pytest.mark.parametrize("other,code", [
    (dict(dtype=7), INVALID), (dict(dtype=tbe.TBE_F32), UNSUPPORTED), (dict(tokens=-1), INVALID), (dict(heads=0), INVALID),
    (dict(head_dim=0), INVALID), (dict(head_dim=129, q_head_stride=129, k_head_stride=129, v_head_stride=129), UNSUPPORTED),
    (dict(tokens=1 << 36), UNSUPPORTED), (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(decay=None), INVALID), (dict(offsets=None), INVALID), (dict(sequences=0), INVALID), (dict(sequences=-1), INVALID),
    (dict(q_stride=31), INVALID), (dict(k_head_stride=15), INVALID), (dict(v_stride=16, v_head_stride=16), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(q=1), UNSUPPORTED), (dict(decay=2), UNSUPPORTED), (dict(s0=2), UNSUPPORTED)])
def test_linear_attention(lib, room, other, code):
    a = linear(room, **other)
    o = base(room, 5)
    assert lib.tbe_linear_attention(ctypes.byref(a), o, 32, 16, None, None, 0, None, None) == code
    g = LinearGrads(o, o, o, 32, 32, 32, 16, 16, 16, None)
    assert lib.tbe_linear_attention_backward(ctypes.byref(a), base(room, 6), 32, 16, None, ctypes.byref(g), None, 0, None,
                                             None) == code


def test_linear_attention_outputs_and_states(lib, room):
    o, s = base(room, 5), base(room, 6)
    size = 4 * 2 * 2 * 16 * 16
    call = lambda a, o, stride, head, last: lib.tbe_linear_attention(ctypes.byref(a), o, stride, head, last, None, 0, None, None)  # noqa: E731
    assert call(linear(room), None, 32, 16, None) == INVALID
    assert call(linear(room), o, 31, 16, None) == INVALID
    assert call(linear(room), o, 32, 15, None) == INVALID
    assert call(linear(room), o + 1, 32, 16, None) == UNSUPPORTED
    assert call(linear(room), o, 32, 16, s + 2) == UNSUPPORTED
    for last in (s, s + size - 4, s - size + 4):  # states that are read and written by different blocks
        assert call(linear(room, s0=s), o, 32, 16, last) == INVALID
    back = lambda a, do, dlast, g: lib.tbe_linear_attention_backward(ctypes.byref(a), do, 32, 16, dlast, ctypes.byref(g),  # noqa: E731
                                                                    None, 0, None, None)
    good = [o, o, o, 32, 32, 32, 16, 16, 16]
    assert back(linear(room), None, None, LinearGrads(*good, None)) == INVALID
    assert back(linear(room), o, None, LinearGrads(None, *good[1:], None)) == INVALID
    assert back(linear(room), o, None, LinearGrads(o, o + 1, *good[2:], None)) == UNSUPPORTED
    assert back(linear(room, s0=s), o, None, LinearGrads(*good, s + 4)) == INVALID
    assert back(linear(room), o, s, LinearGrads(*good, s)) == INVALID
    assert lib.tbe_linear_attention(None, o, 32, 16, None, None, 0, None, None) == INVALID
    assert lib.tbe_linear_attention_step(None, s, o, 32, 16, None) == INVALID
    for a in (linear(room), linear(room, sequences=64, s0=s)):  # a token for each sequence, no s0
        assert lib.tbe_linear_attention_step(ctypes.byref(a), s, o, 32, 16, None) == INVALID
    one = linear(room, sequences=64)
    assert lib.tbe_linear_attention_step(ctypes.byref(one), None, o, 32, 16, None) == INVALID
    assert lib.tbe_linear_attention_step(ctypes.byref(one), s + 2, o, 32, 16, None) == UNSUPPORTED
    assert lib.tbe_linear_attention_workspace_bytes(-1, 1, 1, 0) == 0
    assert lib.tbe_linear_attention_workspace_bytes(1, 1, 129, 0) == 0


def catalogue(room, **other):
    a = dict(hidden=base(room, 0), weights=base(room, 1), labels=base(room, 2), hidden_stride=32, weights_stride=32, tokens=50,
             vocab=60, width=32, dtype=tbe.TBE_F16, logit_scale=1.0)
    a.update(other)
    return Catalogue(*[a[n] for n, _ in Catalogue._fields_])


@pytest.mark.parametrize("other,code", [
    (dict(dtype=9), INVALID), (dict(dtype=tbe.TBE_F32), UNSUPPORTED), (dict(tokens=0), INVALID), (dict(vocab=0), INVALID),
    (dict(width=0), INVALID), (dict(tokens=(1 << 24) + 1), UNSUPPORTED), (dict(vocab=(1 << 30) + 1), UNSUPPORTED),
    (dict(tokens=1 << 24, vocab=1 << 23), UNSUPPORTED),
    (dict(width=(1 << 16) + 1, hidden_stride=1 << 17, weights_stride=1 << 17), UNSUPPORTED), (dict(hidden=None), INVALID),
    (dict(weights=None), INVALID), (dict(labels=None), INVALID), (dict(hidden_stride=31), INVALID),
    (dict(weights_stride=31), INVALID), (dict(logit_scale=float("inf")), INVALID), (dict(hidden=1), UNSUPPORTED),
    (dict(labels=4), UNSUPPORTED)])
def test_catalogue(lib, room, other, code):
    a, f, g, ws = catalogue(room, **other), base(room, 4), base(room, 6), base(room, 8)
    assert lib.tbe_catalogue_loss(ctypes.byref(a), f, f, f, None, 0, None, 0, 1.0, ws, 1 << 16, None, None) == code
    assert lib.tbe_catalogue_loss_backward(ctypes.byref(a), f, g, 32, g + 8192, 32, 1.0, ws, 1 << 16, None, None) == code
    assert lib.tbe_catalogue_workspace_bytes(ctypes.byref(a), 1) == 0


def test_catalogue_outputs_and_workspace(lib, room):
    a, f, ws = catalogue(room), base(room, 4), base(room, 8)
    h, w, g, e = a.hidden, a.weights, base(room, 6), base(room, 7)

    def call(loss=f, token=f, lse=f, dh=g, dhs=32, dw=e, dws=32, scale=1.0, work=ws, size=16):
        return lib.tbe_catalogue_loss(ctypes.byref(a), loss, token, lse, dh, dhs, dw, dws, scale, work, size, None, None)

    assert call() == tbe.TBE_ERR_WORKSPACE
    for missing in (dict(loss=None), dict(token=None), dict(lse=None), dict(dh=None), dict(dw=None), dict(work=None),
                    dict(dhs=31), dict(dws=31), dict(scale=float("nan"))):
        assert call(**missing) == INVALID, missing
    for overlapping in (dict(dh=h), dict(dw=w), dict(dh=w + 2), dict(dw=h + 100), dict(dh=g, dw=g + 64)):
        assert call(**overlapping) == INVALID, overlapping
    assert call(dh=g + 1) == UNSUPPORTED and call(work=ws + 16) == UNSUPPORTED
    assert lib.tbe_catalogue_loss(None, f, f, f, None, 0, None, 0, 1.0, ws, 16, None, None) == INVALID
    assert lib.tbe_catalogue_loss_backward(ctypes.byref(a), None, g, 32, e, 32, 1.0, ws, 16, None, None) == INVALID
    assert lib.tbe_catalogue_loss_backward(ctypes.byref(a), f, None, 32, e, 32, 1.0, ws, 16, None, None) == INVALID
    assert lib.tbe_catalogue_workspace_bytes(None, 0) == 0
