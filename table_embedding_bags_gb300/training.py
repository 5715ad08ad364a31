"""Python binding of the training operators beside the tables.

A gated recurrence and linear attention over jagged sequences, a preference loss over catalogue
logits, cross entropy over a catalogue's table and an AdamW step over a list of
tensors.  As in the package's
``__init__``: argument checks and marshalling only, names as in
``include/tbe.h``, outputs allocated where none are given, everything
enqueued on the current stream (or ``stream``, whose own memory then holds
what the call allocates; the caller orders the streams, and keeps its tensors
alive, as under ``with torch.cuda.stream(stream)``).  The recurrences' and the
losses' checks are compiled (``csrc/marshal.cpp``): their smallest calls take
the GPU a few microseconds.
"""

from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple

import numpy as np
import torch

import table_embedding_bags_gb300 as _tbe

TBE_SCAN_STEP = _tbe.TBE_SCAN_STEP
TBE_ADAMW_BLOCK = _tbe.TBE_ADAMW_BLOCK

_DTYPE = {torch.float32: _tbe.TBE_F32, torch.float16: _tbe.TBE_F16, torch.bfloat16: _tbe.TBE_BF16}


# tbe_adamw of include/tbe.h, packed (native alignment)
_ADAMW = struct.Struct("@dddddq")


class _AdamWTensors(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("state_bits", ctypes.c_int32), ("numel", ctypes.c_void_p),
                ("params", ctypes.c_void_p), ("grads", ctypes.c_void_p), ("param_dtype", ctypes.c_void_p),
                ("grad_dtype", ctypes.c_void_p)]


def _vector(t, shape, dtype, device, what):
    """Checks a contiguous argument of exactly ``shape``."""
    if t is None or t.device != device or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        got = "None" if t is None else f"{t.dtype}, {tuple(t.shape)}, {t.device}"
        raise _tbe.TBEError(f"{what} must be a contiguous {dtype} tensor of shape {shape} on {device} (got {got})")


_compiled = None


def _marshal():
    """The compiled part, given the library's functions (no fallback: raises
    where it has not been built)."""
    global _compiled
    if _compiled is None:
        lib = _tbe.load_library()
        try:
            from table_embedding_bags_gb300 import _marshal as m
        except ImportError as e:
            raise _tbe.TBEError(f"the compiled binding is not built ({e}): build it with "
                                "table_embedding_bags_gb300.build.build()") from e
        m.init(_tbe.TBEError, {name: ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "tbe_gated_scan", "tbe_gated_scan_backward", "tbe_gated_scan_step", "tbe_gated_scan_states",
            "tbe_gated_scan_workspace_bytes", "tbe_preference_loss", "tbe_preference_loss_backward_low",
            "tbe_preference_workspace_bytes", "tbe_catalogue_loss", "tbe_catalogue_loss_backward_full",
            "tbe_catalogue_workspace_bytes", "tbe_linear_attention", "tbe_linear_attention_backward",
            "tbe_linear_attention_step", "tbe_linear_attention_workspace_bytes", "tbe_status_string")})
        _compiled = m
    return _compiled


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


def tbe_gated_scan(x, recur, gate, decay, offsets, h0=None, sharpness: float = 8.0, want_states=False, out=None,
                   dev_status=None, stream=None) -> GatedScan:
    """Gated linear recurrence over the jagged sequences of ``offsets``:
    h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(gate_t) x_t with
    a_t = exp(-sharpness softplus(decay) sigmoid(recur_t)).

    ``x``, ``recur`` and ``gate`` are [tokens, channels] (rows may be
    strided, so slices of one projection do); ``decay`` is fp32 [channels];
    ``offsets`` int64 or int32 [sequences + 1]; ``h0`` fp32 [sequences,
    channels].  ``want_states`` keeps what ``tbe_gated_scan_backward`` needs.
    ``out`` must not overlap an input."""
    m = _compiled or _marshal()
    return GatedScan(*m.gated_scan(x, recur, gate, decay, offsets, h0, sharpness, want_states, out, dev_status,
                                   None if stream is None else stream.cuda_stream))


def tbe_gated_scan_backward(dh, x, recur, gate, decay, offsets, states, h0=None, dh_last=None, sharpness: float = 8.0,
                            out=None, dev_status=None, stream=None) -> GatedScanGrads:
    """Gradients of sum(dh * h) + sum(dh_last * h_last), from the inputs of a
    ``tbe_gated_scan`` call and the ``states`` it kept.  ``out``: the three
    [tokens, channels] tensors to write dx, drecur and dgate to (rows may be
    strided; not overlapping an input).  dh0 is returned where ``h0`` was
    given."""
    m = _compiled or _marshal()
    return GatedScanGrads(*m.gated_scan_backward(dh, x, recur, gate, decay, offsets, states, h0, dh_last, sharpness, out,
                                                 dev_status, None if stream is None else stream.cuda_stream))


def tbe_gated_scan_step(x, recur, gate, decay, state, sharpness: float = 8.0, out=None, stream=None):
    """One token of every sequence: ``state`` (fp32 [sequences, channels])
    moves on in place; returns h [sequences, channels] in x's dtype."""
    m = _compiled or _marshal()
    return m.gated_scan_step(x, recur, gate, decay, state, sharpness, out,
                             None if stream is None else stream.cuda_stream)


# ---------------------------------------------------------------------------
# linear attention
# ---------------------------------------------------------------------------

class LinearAttention(NamedTuple):
    o: torch.Tensor  # [tokens, heads, head_dim] in the inputs' dtype
    s_last: torch.Tensor | None  # fp32 [sequences, heads, head_dim, head_dim]


class LinearAttentionGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    ds0: torch.Tensor | None  # fp32 [sequences, heads, head_dim, head_dim]


def tbe_linear_attention(q, k, v, decay, offsets, s0=None, scale: float = 1.0, want_last=False, out=None,
                         dev_status=None, stream=None) -> LinearAttention:
    """Causal linear attention with a decay for each head over the jagged
    sequences of ``offsets``: o_t = scale S_t^T q_t with S_t = exp(-decay)
    S_{t-1} + k_t v_t^T.

    ``q``, ``k`` and ``v`` are [tokens, heads, head_dim] in float16 or
    bfloat16 (tokens and heads may be strided, so slices of one projection
    do); ``decay`` is fp32 [heads]; ``offsets`` int64 or int32 [sequences +
    1]; ``s0`` fp32 [sequences, heads, head_dim, head_dim] (keys by values).
    ``want_last`` returns each sequence's last state.  An ``out`` that overlaps
    an input is refused."""
    m = _compiled or _marshal()
    return LinearAttention(*m.linear_attention(q, k, v, decay, offsets, s0, scale, want_last, out, dev_status,
                                               None if stream is None else stream.cuda_stream))


def tbe_linear_attention_backward(do, q, k, v, decay, offsets, s0=None, ds_last=None, scale: float = 1.0, out=None,
                                  dev_status=None, stream=None) -> LinearAttentionGrads:
    """Gradients of sum(do * o) + sum(ds_last * s_last) from the inputs of a
    ``tbe_linear_attention`` call.  ``out``: the three tensors to write dq, dk
    and dv to (strided as ``q`` may be; refused where they overlap an input
    or each other).  ds0 is returned where ``s0`` was given."""
    m = _compiled or _marshal()
    return LinearAttentionGrads(*m.linear_attention_backward(do, q, k, v, decay, offsets, s0, ds_last, scale, out,
                                                             dev_status, None if stream is None else stream.cuda_stream))


def tbe_linear_attention_step(q, k, v, decay, state, scale: float = 1.0, out=None, stream=None):
    """One token of every sequence: ``state`` (fp32 [sequences, heads,
    head_dim, head_dim]) moves on in place; returns o [sequences, heads,
    head_dim] in q's dtype."""
    m = _compiled or _marshal()
    return m.linear_attention_step(q, k, v, decay, state, scale, out, None if stream is None else stream.cuda_stream)


# ---------------------------------------------------------------------------
# preference loss
# ---------------------------------------------------------------------------

class PreferenceLoss:
    """Results of ``tbe_preference_loss``, views of one fp32 buffer: ``loss``
    (scalar), ``seq_logps`` [2 * pairs], ``margins`` [pairs], ``lse`` (with
    ``lse_low``, what its rounding left) and ``coef`` [tokens] (for
    ``tbe_preference_loss_backward``); and ``dlogits`` (with the logits' row
    stride, unless those are a narrow view of a wide tensor) or None."""

    __slots__ = ("_room", "_pairs", "_tokens", "dlogits")

    def __init__(self, room, pairs, tokens, dlogits):
        self._room, self._pairs, self._tokens, self.dlogits = room, pairs, tokens, dlogits

    loss = property(lambda self: self._room[0])
    seq_logps = property(lambda self: self._room.narrow(0, 1, 2 * self._pairs))
    margins = property(lambda self: self._room.narrow(0, 1 + 2 * self._pairs, self._pairs))
    lse = property(lambda self: self._room.narrow(0, 1 + 3 * self._pairs, self._tokens))
    coef = property(lambda self: self._room.narrow(0, 1 + 3 * self._pairs + self._tokens, self._tokens))
    # at the beginning of the workspace, which follows on a multiple of 256 bytes
    lse_low = property(lambda self: self._room.narrow(0, (1 + 3 * self._pairs + 2 * self._tokens + 63) // 64 * 64,
                                                      self._tokens))

    def __iter__(self):
        return iter((self.loss, self.seq_logps, self.margins, self.dlogits, self.lse, self.coef))


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
    m = _compiled or _marshal()
    room, dlogits = m.preference_loss(logits, labels, offsets, ref_logps, beta, label_smoothing, want_grad, grad_scale,
                                      dlogits, dev_status, None if stream is None else stream.cuda_stream)
    return PreferenceLoss(room, ref_logps.numel() // 2, logits.shape[0], dlogits)


def tbe_preference_loss_backward(logits, labels, offsets, ref_logps, saved: PreferenceLoss, grad_scale: float = 1.0,
                                 dlogits=None, stream=None):
    """grad_scale * d loss / d logits from what the ``tbe_preference_loss``
    call on the same arguments saved: its gradient bit for bit."""
    m = _compiled or _marshal()
    return m.preference_loss_backward(logits, labels, offsets, ref_logps, saved.lse, saved.lse_low, saved.coef, grad_scale,
                                      dlogits, None if stream is None else stream.cuda_stream)


# ---------------------------------------------------------------------------
# cross entropy over a catalogue
# ---------------------------------------------------------------------------

class CatalogueLoss(NamedTuple):
    loss: torch.Tensor  # fp32 scalar
    token_loss: torch.Tensor  # fp32 [tokens], 0 for tokens that take no part
    lse: torch.Tensor  # fp32 [tokens], likewise
    dhidden: torch.Tensor | None  # [tokens, width]
    dweights: torch.Tensor | None  # [vocab, width]


def tbe_catalogue_loss(hidden, weights, labels, logit_scale: float = 1.0, want_grad=False, grad_scale: float = 1.0,
                       dhidden=None, dweights=None, dev_status=None, stream=None) -> CatalogueLoss:
    """Softmax cross entropy of ``hidden`` [tokens, width] over every row of
    ``weights`` [vocab, width] (float16 or bfloat16, rows may be strided),
    logits = logit_scale * hidden @ weights.T, which are not kept: the mean
    over the tokens with a label in ``labels`` (int64; a negative one takes no
    part, whatever its hidden row holds).  ``want_grad`` (or tensors
    ``dhidden`` and ``dweights`` to write to) adds grad_scale times both
    gradients."""
    m = _compiled or _marshal()
    return CatalogueLoss(*m.catalogue_loss(hidden, weights, labels, logit_scale, want_grad, grad_scale, dhidden, dweights,
                                           dev_status, None if stream is None else stream.cuda_stream))


def tbe_catalogue_loss_backward(hidden, weights, labels, lse, logit_scale: float = 1.0, grad_scale: float = 1.0,
                                dhidden=None, dweights=None, dev_status=None, stream=None, token_loss=None):
    """(dhidden, dweights) from the ``lse`` and ``token_loss`` of a
    ``tbe_catalogue_loss`` call on the same arguments.  Without
    ``token_loss`` the gradients of tokens that are nearly learnt keep few
    digits (a probability less 1)."""
    m = _compiled or _marshal()
    return m.catalogue_loss_backward(hidden, weights, labels, lse, logit_scale, grad_scale, dhidden, dweights, dev_status,
                                     None if stream is None else stream.cuda_stream, token_loss)


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------

# the current stream's handle as an integer, without a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda dev: torch.cuda.current_stream(dev).cuda_stream)


class AdamWPlan:
    """A list of parameters and their gradients with the optimizer's states.

    The plan holds the tensors' addresses: parameters and gradients are
    updated in place and must keep their storage (``rebind`` takes new ones).
    States are flat, ``exp_avg`` and ``exp_avg_sq`` with each tensor's part
    starting on a block of 256 elements (``slices[i]``): fp32 for
    ``state_bits`` 32, codes with one scale per block (``exp_avg_scale``,
    ``exp_avg_sq_scale``) for 8.  ``state``: a dict with those tensors, to go
    on from (they are used as they are, not copied).  A step may go to another
    stream than the plan's (the caller orders the two): what the plan holds is
    then kept from reuse until that stream is through with it, also where the
    plan takes other tensors or ends before."""

    def __init__(self, params, grads, state_bits: int = 32, state=None, stream=None):
        params, grads = list(params), list(grads)
        if not params:
            raise _tbe.TBEError("AdamWPlan needs at least one tensor")
        if state_bits not in (8, 32):
            raise _tbe.TBEError(f"state_bits must be 8 or 32 (got {state_bits})")
        self._need_tensors("parameter", params)
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
        self._state_home, self._state_seen = self._home, set()
        want = {"exp_avg": torch.float32, "exp_avg_sq": torch.float32}
        if state_bits == 8:
            want = {"exp_avg": torch.int8, "exp_avg_sq": torch.uint8, "exp_avg_scale": torch.float32,
                    "exp_avg_sq_scale": torch.float32}
        for name, dt in want.items():
            n = self.blocks if name.endswith("scale") else self.blocks * TBE_ADAMW_BLOCK
            with torch.cuda.stream(stream):
                t = torch.zeros(n, dtype=dt, device=self.device) if state is None else state.get(name)
            _vector(t, (n,), dt, self.device, f"state[{name!r}]")
            setattr(self, name, t)
        if state_bits == 32:
            self.exp_avg_scale = self.exp_avg_sq_scale = None
        self._states = (self.exp_avg, self.exp_avg_sq, self.exp_avg_scale, self.exp_avg_sq_scale)
        self._state_addr = tuple(None if t is None else t.data_ptr() for t in self._states)

    @staticmethod
    def _need_tensors(what, tensors):
        for i, t in enumerate(tensors):
            if not isinstance(t, torch.Tensor):
                raise _tbe.TBEError(f"{what} {i} must be a tensor (got {t!r})")

    def _bind(self, params, grads, stream):
        n = len(params)
        if n != len(self.numel):
            raise _tbe.TBEError(f"the plan is for {len(self.numel)} tensors (got {n} parameters)")
        if len(grads) != n:
            raise _tbe.TBEError(f"{n} parameters but {len(grads)} gradients")
        for what, tensors in (("parameter", params), ("gradient", grads)):
            self._need_tensors(what, tensors)
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
        with torch.cuda.device(self.device):
            home = _tbe._stream(stream)
            with torch.cuda.stream(stream):
                meta = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        L = _AdamWTensors(n, self.state_bits, self.numel.ctypes.data, p.ctypes.data, g.ctypes.data, pd.ctypes.data,
                          gd.ctypes.data)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _tbe._check(lib.tbe_adamw_plan_create(ctypes.byref(L), meta.data_ptr(), nbytes, home, ctypes.byref(h)),
                        "tbe_adamw_plan_create")
        self._release()
        self._h, self._meta, self.params, self.grads = h, meta, params, grads
        self._home, self._seen = home.value or 0, set()  # the plan's stream, others that have read it

    def rebind(self, params=None, grads=None, stream=None):
        """Takes new parameter and/or gradient tensors (same sizes)."""
        self._bind(self.params if params is None else list(params), self.grads if grads is None else list(grads),
                   stream)

    def _call(self, name, stream, *args):
        """Calls an entry point of the plan with the plan's device current."""
        fn, dev = getattr(_tbe._lib, name), self.device.index
        handle = _raw_stream(dev) if stream is None else stream.cuda_stream
        if handle != self._home or handle != self._state_home:
            self._used_on(handle, torch.cuda.current_stream(dev) if stream is None else stream)
        if torch.cuda.current_device() != dev:
            with torch.cuda.device(dev):
                rc = fn(self._h, *args, handle)
        else:
            rc = fn(self._h, *args, handle)
        if rc != _tbe.TBE_OK:
            _tbe._check(rc, name)

    def _used_on(self, handle, stream):
        """Keeps the memory of what the plan holds from reuse until ``stream``
        is through with it (noted once per stream)."""
        for home, seen, tensors in ((self._home, self._seen, (self._meta, *self.params, *self.grads)),
                                    (self._state_home, self._state_seen, self._states)):
            if handle != home and handle not in seen:
                seen.add(handle)
                for t in tensors:
                    if t is not None:
                        t.record_stream(stream)

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
    plan._call("tbe_adamw_step", stream, opt, *plan._state_addr, None if grad_scale is None else grad_scale.data_ptr(),
               None if skip is None else skip.data_ptr())


def tbe_adamw_state(plan: AdamWPlan, stream=None):
    """(exp_avg, exp_avg_sq) as fp32 values, flat as the plan lays them out:
    the states themselves for 32 bits, what the codes stand for for 8."""
    if plan.state_bits == 32:
        return plan.exp_avg, plan.exp_avg_sq
    caller = torch.cuda.current_stream(plan.device)
    with torch.cuda.stream(stream):
        m = torch.empty(plan.blocks * TBE_ADAMW_BLOCK, dtype=torch.float32, device=plan.device)
        v = torch.empty_like(m)
    if stream is not None and stream != caller:  # the caller's own stream is as likely to use them
        m.record_stream(caller)
        v.record_stream(caller)
    plan._call("tbe_adamw_state", stream, *plan._state_addr, m.data_ptr(), v.data_ptr())
    return m, v
