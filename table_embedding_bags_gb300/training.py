"""Python binding of the training operators beside the tables.

A gated recurrence over jagged sequences, a preference loss over catalogue
logits and an AdamW step over a list of tensors.  As in the package's
``__init__``: argument checks and marshalling only, names as in
``include/tbe.h``, outputs allocated where none are given, everything
enqueued on the current stream (or ``stream``).
"""

from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple

import numpy as np
import torch

import table_embedding_bags_gb300 as _tbe

TBE_SCAN_STEP = 8
TBE_ADAMW_BLOCK = 256

_DTYPE = {torch.float32: _tbe.TBE_F32, torch.float16: _tbe.TBE_F16, torch.bfloat16: _tbe.TBE_BF16}


# The argument structs of include/tbe.h that are made at every call, packed
# (native alignment): a ctypes.Structure costs several times as much to fill.
_SCAN_INPUTS = struct.Struct("@qiiiiPPPqqqPPPf0P")
_SCAN_GRADS = struct.Struct("@PPPqqqPP")
_PREFERENCE_INPUTS = struct.Struct("@PqPPPqiiiff0P")
_ADAMW = struct.Struct("@dddddq")


class _AdamWTensors(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("numel", ctypes.c_void_p),
                ("params", ctypes.c_void_p), ("grads", ctypes.c_void_p), ("param_dtype", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_void_p)]


def declare(lib):
    """Result and argument types of the library's training entry points."""
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    for name, res, args in [
        ("tbe_gated_scan_states", i64, [i64]),
        ("tbe_gated_scan_workspace_bytes", sz, [i64, i32, i32, i32]),
        ("tbe_gated_scan", ctypes.c_int, [P, P, i64, P, P, P, sz, P, P]),
        ("tbe_gated_scan_backward", ctypes.c_int, [P, P, i64, P, P, P, P, sz, P, P]),
        ("tbe_gated_scan_step", ctypes.c_int, [P, P, P, i64, P]),
        ("tbe_preference_workspace_bytes", sz, [i64, i32, i32, i32]),
        ("tbe_preference_loss", ctypes.c_int, [P, P, P, P, P, P, P, i64, f32, P, sz, P, P]),
        ("tbe_preference_loss_backward", ctypes.c_int, [P, P, P, f32, P, i64, P]),
        ("tbe_adamw_state_blocks", i64, [i32, P]),
        ("tbe_adamw_plan_device_bytes", sz, [i32, P, i32]),
        ("tbe_adamw_plan_create", ctypes.c_int, [P, P, sz, P, P]),
        ("tbe_adamw_plan_destroy", None, [P]),
        ("tbe_adamw_step", ctypes.c_int, [P, P, P, P, P, P, P, P, P]),
        ("tbe_adamw_state", ctypes.c_int, [P, P, P, P, P, P, P, P]),
    ]:
        getattr(lib, name).restype = res
        getattr(lib, name).argtypes = args


def _rows(t, rows, cols, dtype, dev, what):
    """Checks a [rows, cols] argument of ``dtype`` on CUDA device ``dev`` with
    consecutive columns; returns its row stride in elements (at least cols)."""
    if t.get_device() != dev or dev < 0:
        raise _tbe.TBEError(f"{what} must be a CUDA tensor on the device of the other arguments (got {t.device})")
    if t.dtype is not dtype:
        raise _tbe.TBEError(f"{what} has dtype {t.dtype}; expected {dtype}")
    if t.shape != (rows, cols):
        raise _tbe.TBEError(f"{what} has shape {tuple(t.shape)}; expected ({rows}, {cols})")
    stride, step = t.stride()
    if rows < 2:
        stride = cols
    if (step != 1 and cols > 1 and rows > 0) or stride < cols:
        raise _tbe.TBEError(f"{what} must have consecutive columns and rows that do not overlap")
    return stride


def _vector(t, shape, dtypes, dev, what):
    """Checks a contiguous argument of exactly ``shape``; returns its address."""
    if t is None:
        raise _tbe.TBEError(f"{what} is required")
    if t.get_device() != dev or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise _tbe.TBEError(f"{what} must be a contiguous {' or '.join(map(str, dtypes))} tensor of shape {shape} on "
                            f"CUDA device {dev} (got {t.dtype}, {tuple(t.shape)}, {t.device})")
    return t.data_ptr()


_F32 = (torch.float32,)
_I64 = (torch.int64,)
_I32 = (torch.int32,)
_IDS = (torch.int64, torch.int32)

# the current stream's handle as an integer, without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _run(fn, what, dev, stream, *args):
    """Calls ``fn(*args, stream)`` with CUDA device ``dev`` current."""
    handle = _raw_stream(dev) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() != dev:
        with torch.cuda.device(dev):
            rc = fn(*args, handle)
    else:
        rc = fn(*args, handle)
    if rc != _tbe.TBE_OK:
        _tbe._check(rc, what)


@functools.lru_cache(maxsize=4096)
def _scan_workspace(N, C, dtype, backward, dev):
    with torch.cuda.device(dev):
        return int(_tbe.load_library().tbe_gated_scan_workspace_bytes(N, C, _DTYPE[dtype], backward))


@functools.lru_cache(maxsize=4096)
def _preference_workspace(N, V, P, dtype, dev):
    with torch.cuda.device(dev):
        return int(_tbe.load_library().tbe_preference_workspace_bytes(N, V, P, _DTYPE[dtype]))


# ---------------------------------------------------------------------------
# gated recurrence
# ---------------------------------------------------------------------------

class GatedScan(NamedTuple):
    h: torch.Tensor  # [tokens, channels] in the inputs' dtype
    h_last: torch.Tensor  # fp32 [sequences, channels]
    states: torch.Tensor | None  # for tbe_gated_scan_backward


class GatedScanGrads(NamedTuple):
    dx: torch.Tensor
    drecur: torch.Tensor
    dgate: torch.Tensor
    ddecay: torch.Tensor  # fp32 [channels]
    dh0: torch.Tensor | None  # fp32 [sequences, channels]


def _scan_inputs(x, recur, gate, decay, sequences, offsets, h0, sharpness):
    """Checks what the three scan calls share; returns the packed struct, the
    sizes and the device."""
    dt = x.dtype
    if x.dim() != 2 or dt not in _DTYPE:
        raise _tbe.TBEError(f"x must be a [tokens, channels] tensor of float32, float16 or bfloat16 (got {x.dtype}, "
                            f"{tuple(x.shape)})")
    N, C = x.shape
    dev = x.get_device()
    sx = _rows(x, N, C, dt, dev, "x")
    sr = _rows(recur, N, C, dt, dev, "recur")
    sg = _rows(gate, N, C, dt, dev, "gate")
    d = _vector(decay, (C,), _F32, dev, "decay")
    h = 0 if h0 is None else _vector(h0, (sequences, C), _F32, dev, "h0")
    o, i32 = 0, 0
    if offsets is not None:
        o = _vector(offsets, (sequences + 1,), _IDS, dev, "offsets")
        i32 = int(offsets.dtype is torch.int32)
    packed = _SCAN_INPUTS.pack(N, sequences, C, _DTYPE[dt], i32, x.data_ptr(), recur.data_ptr(), gate.data_ptr(), sx,
                               sr, sg, d, o, h, sharpness)
    return packed, N, C, dt, dev


def _sequences(offsets):
    S = offsets.numel() - 1
    if S < 0:
        raise _tbe.TBEError("offsets must hold at least one entry")
    return S


def tbe_gated_scan(x, recur, gate, decay, offsets, h0=None, sharpness: float = 8.0, want_states=False, out=None,
                   dev_status=None, stream=None) -> GatedScan:
    """Gated linear recurrence over the jagged sequences of ``offsets``:
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t with
    a_t = exp(-sharpness softplus(decay) sigmoid(recur_t)).

    ``x``, ``recur`` and ``gate`` are [tokens, channels] (rows may be
    strided, so slices of one projection do); ``decay`` is fp32 [channels];
    ``offsets`` int64 or int32 [sequences + 1]; ``h0`` fp32 [sequences,
    channels].  ``want_states`` keeps what ``tbe_gated_scan_backward`` needs."""
    lib = _tbe.load_library()
    S = _sequences(offsets)
    a, N, C, dt, dev = _scan_inputs(x, recur, gate, decay, S, offsets, h0, sharpness)
    if out is None:
        h, h_stride = x.new_empty((N, C)), C
    else:
        h, h_stride = out, _rows(out, N, C, dt, dev, "out")
    st = None if dev_status is None else _vector(dev_status, (1,), _I32, dev, "dev_status")
    h_last = decay.new_empty((S, C))
    states = decay.new_empty((max(1, -(-N // TBE_SCAN_STEP)), C)) if want_states else None
    nbytes = _scan_workspace(N, C, dt, 0, dev)
    ws = decay.new_empty(nbytes // 4) if nbytes else None
    _run(lib.tbe_gated_scan, "tbe_gated_scan", dev, stream, a, h.data_ptr(), h_stride, h_last.data_ptr(),
         states.data_ptr() if want_states else None, ws.data_ptr() if nbytes else None, nbytes, st)
    return GatedScan(h, h_last, states)


def tbe_gated_scan_backward(dh, x, recur, gate, decay, offsets, states, h0=None, dh_last=None, sharpness: float = 8.0,
                            out=None, dev_status=None, stream=None) -> GatedScanGrads:
    """Gradients of sum(dh * h) + sum(dh_last * h_last), from the inputs of a
    ``tbe_gated_scan`` call and the ``states`` it kept.  ``out``: the three
    [tokens, channels] tensors to write dx, drecur and dgate to (rows may be
    strided).  dh0 is returned where ``h0`` was given."""
    lib = _tbe.load_library()
    S = _sequences(offsets)
    a, N, C, dt, dev = _scan_inputs(x, recur, gate, decay, S, offsets, h0, sharpness)
    dh_stride = _rows(dh, N, C, dt, dev, "dh")
    last = None if dh_last is None else _vector(dh_last, (S, C), _F32, dev, "dh_last")
    kept = _vector(states, (max(1, -(-N // TBE_SCAN_STEP)), C), _F32, dev, "states")
    st = None if dev_status is None else _vector(dev_status, (1,), _I32, dev, "dev_status")
    if out is None:
        dx, dr, dg = x.new_empty((N, C)), x.new_empty((N, C)), x.new_empty((N, C))
        strides = (C, C, C)
    else:
        dx, dr, dg = out
        strides = (_rows(dx, N, C, dt, dev, "dx"), _rows(dr, N, C, dt, dev, "drecur"), _rows(dg, N, C, dt, dev, "dgate"))
    ddecay = decay.new_empty(C)
    dh0 = None if h0 is None else decay.new_empty((S, C))
    g = _SCAN_GRADS.pack(dx.data_ptr(), dr.data_ptr(), dg.data_ptr(), *strides, ddecay.data_ptr(),
                         0 if dh0 is None else dh0.data_ptr())
    nbytes = _scan_workspace(N, C, dt, 1, dev)
    ws = decay.new_empty(nbytes // 4) if nbytes else None
    _run(lib.tbe_gated_scan_backward, "tbe_gated_scan_backward", dev, stream, a, dh.data_ptr(), dh_stride, last, kept, g,
         ws.data_ptr() if nbytes else None, nbytes, st)
    return GatedScanGrads(dx, dr, dg, ddecay, dh0)


def tbe_gated_scan_step(x, recur, gate, decay, state, sharpness: float = 8.0, out=None, stream=None):
    """One token of every sequence: ``state`` (fp32 [sequences, channels])
    moves on in place; returns h [sequences, channels] in x's dtype."""
    lib = _tbe.load_library()
    a, S, C, dt, dev = _scan_inputs(x, recur, gate, decay, x.shape[0], None, None, sharpness)
    s = _vector(state, (S, C), _F32, dev, "state")
    if out is None:
        h, h_stride = x.new_empty((S, C)), C
    else:
        h, h_stride = out, _rows(out, S, C, dt, dev, "out")
    _run(lib.tbe_gated_scan_step, "tbe_gated_scan_step", dev, stream, a, s, h.data_ptr(), h_stride)
    return h


# ---------------------------------------------------------------------------
# preference loss
# ---------------------------------------------------------------------------

class PreferenceLoss:
    """Results of ``tbe_preference_loss``, views of one fp32 buffer: ``loss``
    (scalar), ``seq_logps`` [2 * pairs], ``margins`` [pairs], ``lse`` and
    ``coef`` [tokens] (for ``tbe_preference_loss_backward``); and ``dlogits``
    (laid out like the logits) or None."""

    __slots__ = ("_room", "_pairs", "_tokens", "dlogits")

    def __init__(self, room, pairs, tokens, dlogits):
        self._room, self._pairs, self._tokens, self.dlogits = room, pairs, tokens, dlogits

    loss = property(lambda self: self._room[0])
    seq_logps = property(lambda self: self._room.narrow(0, 1, 2 * self._pairs))
    margins = property(lambda self: self._room.narrow(0, 1 + 2 * self._pairs, self._pairs))
    lse = property(lambda self: self._room.narrow(0, 1 + 3 * self._pairs, self._tokens))
    coef = property(lambda self: self._room.narrow(0, 1 + 3 * self._pairs + self._tokens, self._tokens))

    def __iter__(self):
        return iter((self.loss, self.seq_logps, self.margins, self.dlogits, self.lse, self.coef))


def _preference_inputs(logits, labels, offsets, ref_logps, beta, label_smoothing):
    dt = logits.dtype
    if logits.dim() != 2 or dt not in _DTYPE:
        raise _tbe.TBEError(f"logits must be a [tokens, vocab] tensor of float32, float16 or bfloat16 (got "
                            f"{logits.dtype}, {tuple(logits.shape)})")
    N, V = logits.shape
    dev = logits.get_device()
    stride = _rows(logits, N, V, dt, dev, "logits")
    if N < 1 or V < 1 or V >= 1 << 31:
        raise _tbe.TBEError("logits must have at least one row and one column (and fewer than 2^31 columns)")
    Q = ref_logps.numel()
    if Q < 2 or Q % 2:
        raise _tbe.TBEError("ref_logps must hold two sequences per pair")
    y = _vector(labels, (N,), _I64, dev, "labels")
    o = _vector(offsets, (Q + 1,), _I64, dev, "offsets")
    r = _vector(ref_logps, (Q,), _F32, dev, "ref_logps")
    packed = _PREFERENCE_INPUTS.pack(logits.data_ptr(), stride, y, o, r, N, V, Q // 2, _DTYPE[dt], beta, label_smoothing)
    return packed, N, V, Q // 2, stride, dt, dev


def _like_rows(logits, N, V, stride):
    """Room for the gradient with the logits' row stride, so that both rows
    start on the same alignment."""
    if stride == V:
        return logits.new_empty((N, V))
    return logits.new_empty((N, stride))[:, :V]


def tbe_preference_loss(logits, labels, offsets, ref_logps, beta: float = 0.1, label_smoothing: float = 0.0,
                        want_grad=False, grad_scale: float = 1.0, dlogits=None, dev_status=None,
                        stream=None) -> PreferenceLoss:
    """Preference loss of pairs of label sequences over ``logits`` [tokens,
    vocab]: the mean over pairs of -log sigmoid(d), d = beta times the
    difference of the preferred and the rejected sequence's log-ratio to
    ``ref_logps`` (with ``label_smoothing``).  ``offsets`` (int64 [2 * pairs +
    1]) lists the preferred sequences, then the rejected ones; a token whose
    label is negative takes no part.  ``want_grad`` (or a ``dlogits`` tensor,
    which may be ``logits``) adds grad_scale * d loss / d logits."""
    lib = _tbe.load_library()
    a, N, V, P, stride, dt, dev = _preference_inputs(logits, labels, offsets, ref_logps, beta, label_smoothing)
    d_stride = 0
    if dlogits is not None:
        d_stride = _rows(dlogits, N, V, dt, dev, "dlogits")
    elif want_grad:
        dlogits, d_stride = _like_rows(logits, N, V, stride), stride
    st = None if dev_status is None else _vector(dev_status, (1,), _I32, dev, "dev_status")
    # one allocation: the results, then the workspace on 256 bytes
    start = -(-4 * (1 + 3 * P + 2 * N) // 256) * 256
    nbytes = _preference_workspace(N, V, P, dt, dev)
    room = ref_logps.new_empty((start + nbytes) // 4)
    at = room.data_ptr()
    _run(lib.tbe_preference_loss, "tbe_preference_loss", dev, stream, a, at, at + 4, at + 4 + 8 * P, at + 4 + 12 * P,
         at + 4 + 12 * P + 4 * N, None if dlogits is None else dlogits.data_ptr(), d_stride, grad_scale, at + start,
         nbytes, st)
    return PreferenceLoss(room, P, N, dlogits)


def tbe_preference_loss_backward(logits, labels, offsets, ref_logps, saved: PreferenceLoss, grad_scale: float = 1.0,
                                 dlogits=None, stream=None):
    """grad_scale * d loss / d logits from the ``lse`` and ``coef`` of the
    ``tbe_preference_loss`` call on the same arguments."""
    lib = _tbe.load_library()
    a, N, V, _, stride, dt, dev = _preference_inputs(logits, labels, offsets, ref_logps, 1.0, 0.0)
    lse = _vector(saved.lse, (N,), _F32, dev, "saved.lse")
    coef = _vector(saved.coef, (N,), _F32, dev, "saved.coef")
    if dlogits is None:
        dlogits, d_stride = _like_rows(logits, N, V, stride), stride
    else:
        d_stride = _rows(dlogits, N, V, dt, dev, "dlogits")
    _run(lib.tbe_preference_loss_backward, "tbe_preference_loss_backward", dev, stream, a, lse, coef, grad_scale,
         dlogits.data_ptr(), d_stride)
    return dlogits


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

class AdamWPlan:
    """A list of parameters and their gradients with the optimizer's states.

    The plan holds the tensors' addresses: parameters and gradients are
    updated in place and must keep their storage (``rebind`` takes new ones).
    States are flat, ``exp_avg`` and ``exp_avg_sq`` with each tensor's part
    starting on a block of 256 elements (``slices[i]``): fp32 for
    ``state_bits`` 32, codes with one scale per block (``exp_avg_scale``,
    ``exp_avg_sq_scale``) for 8.  ``state``: a dict with those tensors, to go
    on from (they are used as they are, not copied)."""

    def __init__(self, params, grads, state_bits: int = 32, state=None, stream=None):
        params, grads = list(params), list(grads)
        if not params:
            raise _tbe.TBEError("AdamWPlan needs at least one tensor")
        if state_bits not in (8, 32):
            raise _tbe.TBEError(f"state_bits must be 8 or 32 (got {state_bits})")
        self.state_bits = state_bits
        self.device = params[0].device
        if self.device.type != "cuda":
            raise _tbe.TBEError(f"parameter 0 must be a CUDA tensor (got {self.device})")
        self.numel = np.array([p.numel() for p in params], dtype=np.int64)
        ends = np.cumsum(-(-self.numel // TBE_ADAMW_BLOCK))
        self.blocks = int(ends[-1])
        starts = np.concatenate([[0], ends[:-1]]) * TBE_ADAMW_BLOCK
        self.slices = [slice(int(s), int(s + n)) for s, n in zip(starts, self.numel)]
        self._h = ctypes.c_void_p()
        self._bind(params, grads, stream)
        want = {"exp_avg": torch.float32, "exp_avg_sq": torch.float32}
        if state_bits == 8:
            want = {"exp_avg": torch.int8, "exp_avg_sq": torch.uint8, "exp_avg_scale": torch.float32,
                    "exp_avg_sq_scale": torch.float32}
        for name, dt in want.items():
            n = self.blocks if name.endswith("scale") else self.blocks * TBE_ADAMW_BLOCK
            t = torch.zeros(n, dtype=dt, device=self.device) if state is None else state.get(name)
            _vector(t, (n,), (dt,), self.device.index, f"state[{name!r}]")
            setattr(self, name, t)
        if state_bits == 32:
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        self._state_addr = tuple(None if t is None else t.data_ptr() for t in (
            self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale))

    def _bind(self, params, grads, stream):
        n = len(params)
        if len(grads) != n:
            raise _tbe.TBEError(f"{n} parameters but {len(grads)} gradients")
        for what, tensors in (("parameter", params), ("gradient", grads)):
            for i, t in enumerate(tensors):
                if t.device != self.device or t.device.type != "cuda":
                    raise _tbe.TBEError(f"{what} {i} must be a CUDA tensor on {self.device} (got {t.device})")
                if t.dtype not in _DTYPE:
                    raise _tbe.TBEError(f"{what} {i} has dtype {t.dtype}; expected float32, float16 or bfloat16")
                if not t.is_contiguous() or t.numel() != self.numel[i]:
                    raise _tbe.TBEError(f"{what} {i} must be contiguous with {self.numel[i]} elements")
        lib = _tbe.load_library()
        p = np.array([t.data_ptr() for t in params], dtype=np.uint64)
        g = np.array([t.data_ptr() for t in grads], dtype=np.uint64)
        pd = np.array([_DTYPE[t.dtype] for t in params], dtype=np.int32)
        gd = np.array([_DTYPE[t.dtype] for t in grads], dtype=np.int32)
        nbytes = lib.tbe_adamw_plan_device_bytes(n, self.numel.ctypes.data, self.state_bits)
        if nbytes == 0:
            raise _tbe.TBEError("tbe_adamw_plan_device_bytes: sizes out of range")
        meta = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        L = _AdamWTensors(n, self.state_bits, self.numel.ctypes.data, p.ctypes.data, g.ctypes.data, pd.ctypes.data,
                          gd.ctypes.data)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _tbe._check(lib.tbe_adamw_plan_create(ctypes.byref(L), meta.data_ptr(), nbytes, _tbe._stream(stream),
                                                  ctypes.byref(h)), "tbe_adamw_plan_create")
        self._release()
        self._h, self._meta, self.params, self.grads = h, meta, params, grads

    def rebind(self, params=None, grads=None, stream=None):
        """Takes new parameter and/or gradient tensors (same sizes)."""
        self._bind(self.params if params is None else list(params), self.grads if grads is None else list(grads),
                   stream)

    def _release(self):
        if self._h.value and _tbe._lib is not None:
            _tbe._lib.tbe_adamw_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        if getattr(self, "_h", None) is not None:
            self._release()


def tbe_adamw_step(plan: AdamWPlan, step: int, learning_rate: float, beta1: float = 0.9, beta2: float = 0.999,
                   eps: float = 1e-8, weight_decay: float = 0.01, grad_scale=None, skip=None, stream=None):
    """One AdamW step, in place on the plan's parameters and states.
    ``step`` counts from 1.  ``grad_scale``: fp32 scalar on the device that
    multiplies every gradient; ``skip``: int32 scalar on the device, not 0
    where the step is to change nothing."""
    for t, dt, what in ((grad_scale, torch.float32, "grad_scale"), (skip, torch.int32, "skip")):
        if t is not None and (t.device != plan.device or t.dtype is not dt or t.numel() != 1):
            raise _tbe.TBEError(f"{what} must be one {dt} on {plan.device}")
    opt = _ADAMW.pack(learning_rate, beta1, beta2, eps, weight_decay, step)
    _run(_tbe.load_library().tbe_adamw_step, "tbe_adamw_step", plan.device.index, stream, plan._h, opt,
         *plan._state_addr, None if grad_scale is None else grad_scale.data_ptr(), None if skip is None else skip.data_ptr())


def tbe_adamw_state(plan: AdamWPlan, stream=None):
    """(exp_avg, exp_avg_sq) as fp32 values, flat as the plan lays them out:
    the states themselves for 32 bits, what the codes stand for for 8."""
    if plan.state_bits == 32:
        return plan.exp_avg, plan.exp_avg_sq
    m = torch.empty(plan.blocks * TBE_ADAMW_BLOCK, dtype=torch.float32, device=plan.device)
    v = torch.empty_like(m)
    _run(_tbe.load_library().tbe_adamw_state, "tbe_adamw_state", plan.device.index, stream, plan._h, *plan._state_addr,
         m.data_ptr(), v.data_ptr())
    return m, v
