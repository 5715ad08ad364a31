"""Python binding of the training operators beside the tables.

A gated recurrence over jagged sequences, a preference loss over catalogue
logits and an AdamW step over a list of tensors.  As in the package's
``__init__``: argument checks and marshalling only, names as in
``include/tbe.h``, outputs allocated where none are given, everything
enqueued on the current stream (or ``stream``).
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import numpy as np
import torch

import table_embedding_bags_gb300 as _tbe

TBE_SCAN_STEP = 8
TBE_ADAMW_BLOCK = 256

_DTYPE = {torch.float32: _tbe.TBE_F32, torch.float16: _tbe.TBE_F16, torch.bfloat16: _tbe.TBE_BF16}


class _ScanInputs(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("sequences", ctypes.c_int32), ("channels", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("offsets_i32", ctypes.c_int32), ("x", ctypes.c_void_p),
                ("recur", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("x_stride", ctypes.c_int64),
                ("recur_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64), ("decay", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("h0", ctypes.c_void_p), ("sharpness", ctypes.c_float)]


class _ScanGrads(ctypes.Structure):
    _fields_ = [("dx", ctypes.c_void_p), ("drecur", ctypes.c_void_p), ("dgate", ctypes.c_void_p),
                ("dx_stride", ctypes.c_int64), ("drecur_stride", ctypes.c_int64), ("dgate_stride", ctypes.c_int64),
                ("ddecay", ctypes.c_void_p), ("dh0", ctypes.c_void_p)]


class _PreferenceInputs(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("logits_stride", ctypes.c_int64), ("labels", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("ref_logps", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("vocab", ctypes.c_int32), ("pairs", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("beta", ctypes.c_float), ("label_smoothing", ctypes.c_float)]


class _AdamWTensors(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("numel", ctypes.c_void_p),
                ("params", ctypes.c_void_p), ("grads", ctypes.c_void_p), ("param_dtype", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_void_p)]


class _AdamW(ctypes.Structure):
    _fields_ = [("learning_rate", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


def declare(lib):
    """Result and argument types of the library's training entry points."""
    P, i32, i64, sz, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    for name, res, args in [
        ("tbe_gated_scan_states", i64, [i64]),
        ("tbe_gated_scan_workspace_bytes", sz, [i64, i32, i32]),
        ("tbe_gated_scan", ctypes.c_int, [P, P, i64, P, P, P, sz, P, P]),
        ("tbe_gated_scan_backward", ctypes.c_int, [P, P, i64, P, P, P, P, sz, P, P]),
        ("tbe_gated_scan_step", ctypes.c_int, [P, P, P, i64, P]),
        ("tbe_preference_workspace_bytes", sz, [i64, i32, i32]),
        ("tbe_preference_loss", ctypes.c_int, [P, P, P, P, P, P, P, i64, f32, P, sz, P, P]),
        ("tbe_preference_loss_backward", ctypes.c_int, [P, P, P, f32, P, i64, P]),
        ("tbe_adamw_state_blocks", i64, [i32, P]),
        ("tbe_adamw_plan_device_bytes", sz, [i32, P]),
        ("tbe_adamw_plan_create", ctypes.c_int, [P, P, sz, P, P]),
        ("tbe_adamw_plan_destroy", None, [P]),
        ("tbe_adamw_step", ctypes.c_int, [P, P, P, P, P, P, P, P, P]),
        ("tbe_adamw_state", ctypes.c_int, [P, P, P, P, P, P, P, P]),
    ]:
        getattr(lib, name).restype = res
        getattr(lib, name).argtypes = args


def _rows(t, rows, cols, dtype, device, what):
    """Checks a [rows, cols] argument of ``dtype`` on ``device`` with
    consecutive columns; returns its row stride in elements (at least cols)."""
    if t.device != device or device.type != "cuda":
        raise _tbe.TBEError(f"{what} must be a CUDA tensor on the device of the other arguments (got {t.device})")
    if t.dtype is not dtype:
        raise _tbe.TBEError(f"{what} has dtype {t.dtype}; expected {dtype}")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise _tbe.TBEError(f"{what} has shape {tuple(t.shape)}; expected ({rows}, {cols})")
    stride = t.stride(0) if rows > 1 else cols
    if (cols > 1 and rows > 0 and t.stride(1) != 1) or stride < cols:
        raise _tbe.TBEError(f"{what} must have consecutive columns and rows that do not overlap")
    return stride


def _vector(t, shape, dtypes, device, what, optional=False):
    """Checks a contiguous argument of exactly ``shape``."""
    if t is None:
        if optional:
            return
        raise _tbe.TBEError(f"{what} is required")
    if t.device != device or t.dtype not in dtypes or tuple(t.shape) != shape or not t.is_contiguous():
        raise _tbe.TBEError(f"{what} must be a contiguous {' or '.join(map(str, dtypes))} tensor of shape {shape} on "
                            f"{device} (got {t.dtype}, {tuple(t.shape)}, {t.device})")


def _addr(t):
    return None if t is None else t.data_ptr()


_F32 = (torch.float32,)
_I64 = (torch.int64,)
_I32 = (torch.int32,)
_IDS = (torch.int64, torch.int32)


def _run(fn, what, device, stream, *args):
    """Calls ``fn(*args, stream)`` with ``device`` current."""
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            rc = fn(*args, _tbe._stream(stream))
    else:
        rc = fn(*args, (torch.cuda.current_stream() if stream is None else stream).cuda_stream)
    if rc != _tbe.TBE_OK:
        _tbe._check(rc, what)


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
    if x.dim() != 2 or x.dtype not in _DTYPE:
        raise _tbe.TBEError(f"x must be a [tokens, channels] tensor of float32, float16 or bfloat16 (got {x.dtype}, "
                            f"{tuple(x.shape)})")
    N, C = x.shape
    dev, dt = x.device, x.dtype
    strides = [_rows(t, N, C, dt, dev, name) for t, name in ((x, "x"), (recur, "recur"), (gate, "gate"))]
    _vector(decay, (C,), _F32, dev, "decay")
    _vector(h0, (sequences, C), _F32, dev, "h0", optional=True)
    i32 = 0
    if offsets is not None:
        _vector(offsets, (sequences + 1,), _IDS, dev, "offsets")
        i32 = int(offsets.dtype is torch.int32)
    return _ScanInputs(N, sequences, C, _DTYPE[dt], i32, x.data_ptr(), recur.data_ptr(), gate.data_ptr(), *strides,
                       decay.data_ptr(), _addr(offsets), _addr(h0), float(sharpness))


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


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
    S = int(offsets.numel()) - 1
    if S < 0:
        raise _tbe.TBEError("offsets must hold at least one entry")
    a = _scan_inputs(x, recur, gate, decay, S, offsets, h0, sharpness)
    N, C, dev = a.tokens, a.channels, x.device
    h = torch.empty((N, C), dtype=x.dtype, device=dev) if out is None else out
    h_stride = C if out is None else _rows(out, N, C, x.dtype, dev, "out")
    _vector(dev_status, (1,), _I32, dev, "dev_status", optional=True)
    h_last = torch.empty((S, C), dtype=torch.float32, device=dev)
    states = None
    if want_states:
        states = torch.empty((lib.tbe_gated_scan_states(N), C), dtype=torch.float32, device=dev)
    nbytes = lib.tbe_gated_scan_workspace_bytes(N, C, 0)
    ws = _workspace(nbytes, dev)
    _run(lib.tbe_gated_scan, "tbe_gated_scan", dev, stream, ctypes.byref(a), h.data_ptr(), h_stride,
         h_last.data_ptr(), _addr(states), _addr(ws), nbytes, _addr(dev_status))
    return GatedScan(h, h_last, states)


def tbe_gated_scan_backward(dh, x, recur, gate, decay, offsets, states, h0=None, dh_last=None, sharpness: float = 8.0,
                            out=None, dev_status=None, stream=None) -> GatedScanGrads:
    """Gradients of sum(dh * h) + sum(dh_last * h_last), from the inputs of a
    ``tbe_gated_scan`` call and the ``states`` it kept.  ``out``: the three
    [tokens, channels] tensors to write dx, drecur and dgate to (rows may be
    strided).  dh0 is returned where ``h0`` was given."""
    lib = _tbe.load_library()
    S = int(offsets.numel()) - 1
    if S < 0:
        raise _tbe.TBEError("offsets must hold at least one entry")
    a = _scan_inputs(x, recur, gate, decay, S, offsets, h0, sharpness)
    N, C, dev, dt = a.tokens, a.channels, x.device, x.dtype
    dh_stride = _rows(dh, N, C, dt, dev, "dh")
    _vector(dh_last, (S, C), _F32, dev, "dh_last", optional=True)
    _vector(states, (lib.tbe_gated_scan_states(N), C), _F32, dev, "states")
    _vector(dev_status, (1,), _I32, dev, "dev_status", optional=True)
    if out is None:
        out = tuple(torch.empty((N, C), dtype=dt, device=dev) for _ in range(3))
    strides = [_rows(t, N, C, dt, dev, "out") for t in out]
    ddecay = torch.empty(C, dtype=torch.float32, device=dev)
    dh0 = None if h0 is None else torch.empty((S, C), dtype=torch.float32, device=dev)
    g = _ScanGrads(out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), *strides, ddecay.data_ptr(), _addr(dh0))
    nbytes = lib.tbe_gated_scan_workspace_bytes(N, C, 1)
    ws = _workspace(nbytes, dev)
    _run(lib.tbe_gated_scan_backward, "tbe_gated_scan_backward", dev, stream, ctypes.byref(a), dh.data_ptr(),
         dh_stride, _addr(dh_last), states.data_ptr(), ctypes.byref(g), _addr(ws), nbytes, _addr(dev_status))
    return GatedScanGrads(*out, ddecay, dh0)


def tbe_gated_scan_step(x, recur, gate, decay, state, sharpness: float = 8.0, out=None, stream=None):
    """One token of every sequence: ``state`` (fp32 [sequences, channels])
    moves on in place; returns h [sequences, channels] in x's dtype."""
    lib = _tbe.load_library()
    S = int(x.shape[0])
    a = _scan_inputs(x, recur, gate, decay, S, None, None, sharpness)
    C, dev = a.channels, x.device
    _vector(state, (S, C), _F32, dev, "state")
    h = torch.empty((S, C), dtype=x.dtype, device=dev) if out is None else out
    h_stride = C if out is None else _rows(out, S, C, x.dtype, dev, "out")
    _run(lib.tbe_gated_scan_step, "tbe_gated_scan_step", dev, stream, ctypes.byref(a), state.data_ptr(),
         h.data_ptr(), h_stride)
    return h


# ---------------------------------------------------------------------------
# preference loss
# ---------------------------------------------------------------------------

class PreferenceLoss(NamedTuple):
    loss: torch.Tensor  # fp32 scalar
    seq_logps: torch.Tensor  # fp32 [2 * pairs]
    margins: torch.Tensor  # fp32 [pairs]
    dlogits: torch.Tensor | None  # laid out like the logits
    lse: torch.Tensor  # fp32 [tokens]; with coef, for tbe_preference_loss_backward
    coef: torch.Tensor  # fp32 [tokens]


def _preference_inputs(logits, labels, offsets, ref_logps, beta, label_smoothing):
    if logits.dim() != 2 or logits.dtype not in _DTYPE:
        raise _tbe.TBEError(f"logits must be a [tokens, vocab] tensor of float32, float16 or bfloat16 (got "
                            f"{logits.dtype}, {tuple(logits.shape)})")
    N, V = logits.shape
    dev = logits.device
    stride = _rows(logits, N, V, logits.dtype, dev, "logits")
    if N < 1 or V < 1 or V >= 1 << 31:
        raise _tbe.TBEError("logits must have at least one row and one column (and fewer than 2^31 columns)")
    Q = int(ref_logps.numel())
    if Q < 2 or Q % 2:
        raise _tbe.TBEError("ref_logps must hold two sequences per pair")
    _vector(labels, (N,), _I64, dev, "labels")
    _vector(offsets, (Q + 1,), _I64, dev, "offsets")
    _vector(ref_logps, (Q,), _F32, dev, "ref_logps")
    return _PreferenceInputs(logits.data_ptr(), stride, labels.data_ptr(), offsets.data_ptr(), ref_logps.data_ptr(),
                             N, V, Q // 2, _DTYPE[logits.dtype], float(beta), float(label_smoothing))


def _like_rows(logits, stride):
    """Room for the gradient with the logits' row stride, so that both rows
    start on the same alignment."""
    N, V = logits.shape
    return torch.empty((N, stride), dtype=logits.dtype, device=logits.device)[:, :V]


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
    a = _preference_inputs(logits, labels, offsets, ref_logps, beta, label_smoothing)
    N, V, P, dev = a.tokens, a.vocab, a.pairs, logits.device
    d_stride = 0
    if dlogits is not None:
        d_stride = _rows(dlogits, N, V, logits.dtype, dev, "dlogits")
    elif want_grad:
        dlogits, d_stride = _like_rows(logits, a.logits_stride), a.logits_stride
    _vector(dev_status, (1,), _I32, dev, "dev_status", optional=True)
    loss, seq_logps, margins, lse, coef = torch.empty(1 + 3 * P + 2 * N, dtype=torch.float32, device=dev).split(
        [1, 2 * P, P, N, N])
    nbytes = lib.tbe_preference_workspace_bytes(N, V, P)
    ws = _workspace(nbytes, dev)
    _run(lib.tbe_preference_loss, "tbe_preference_loss", dev, stream, ctypes.byref(a), loss.data_ptr(),
         seq_logps.data_ptr(), margins.data_ptr(), lse.data_ptr(), coef.data_ptr(), _addr(dlogits), d_stride,
         float(grad_scale), ws.data_ptr(), nbytes, _addr(dev_status))
    return PreferenceLoss(loss.view(()), seq_logps, margins, dlogits, lse, coef)


def tbe_preference_loss_backward(logits, labels, offsets, ref_logps, saved: PreferenceLoss, grad_scale: float = 1.0,
                                 dlogits=None, stream=None):
    """grad_scale * d loss / d logits from the ``lse`` and ``coef`` of the
    ``tbe_preference_loss`` call on the same arguments."""
    lib = _tbe.load_library()
    a = _preference_inputs(logits, labels, offsets, ref_logps, 1.0, 0.0)
    N, V, dev = a.tokens, a.vocab, logits.device
    _vector(saved.lse, (N,), _F32, dev, "saved.lse")
    _vector(saved.coef, (N,), _F32, dev, "saved.coef")
    if dlogits is None:
        dlogits, d_stride = _like_rows(logits, a.logits_stride), a.logits_stride
    else:
        d_stride = _rows(dlogits, N, V, logits.dtype, dev, "dlogits")
    _run(lib.tbe_preference_loss_backward, "tbe_preference_loss_backward", dev, stream, ctypes.byref(a),
         saved.lse.data_ptr(), saved.coef.data_ptr(), float(grad_scale), dlogits.data_ptr(), d_stride)
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
            _vector(t, (n,), (dt,), self.device, f"state[{name!r}]")
            setattr(self, name, t)
        if state_bits == 32:
            self.exp_avg_scale = self.exp_avg_sq_scale = None

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
        nbytes = lib.tbe_adamw_plan_device_bytes(n, self.numel.ctypes.data)
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
    opt = _AdamW(learning_rate, beta1, beta2, eps, weight_decay, step)
    _run(_tbe.load_library().tbe_adamw_step, "tbe_adamw_step", plan.device, stream, plan._h, ctypes.byref(opt),
         plan.exp_avg.data_ptr(), plan.exp_avg_sq.data_ptr(), _addr(plan.exp_avg_scale),
         _addr(plan.exp_avg_sq_scale), _addr(grad_scale), _addr(skip))


def tbe_adamw_state(plan: AdamWPlan, stream=None):
    """(exp_avg, exp_avg_sq) as fp32 values, flat as the plan lays them out:
    the states themselves for 32 bits, what the codes stand for for 8."""
    if plan.state_bits == 32:
        return plan.exp_avg, plan.exp_avg_sq
    m = torch.empty(plan.blocks * TBE_ADAMW_BLOCK, dtype=torch.float32, device=plan.device)
    v = torch.empty_like(m)
    _run(_tbe.load_library().tbe_adamw_state, "tbe_adamw_state", plan.device, stream, plan._h,
         plan.exp_avg.data_ptr(), plan.exp_avg_sq.data_ptr(), plan.exp_avg_scale.data_ptr(),
         plan.exp_avg_sq_scale.data_ptr(), m.data_ptr(), v.data_ptr())
    return m, v
