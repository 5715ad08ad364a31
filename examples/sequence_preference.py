"""A training step of a sequence model over an embedding table, on synthetic data.

Users' histories are jagged sequences of item ids, two per pair: one that ends
in items the user preferred, one in items they did not.  A step

  1. looks the items up in the table           (tbe_forward, one id per bag),
  2. projects the rows and mixes each history  (tbe_gated_scan),
  3. scores the whole catalogue at each token  (a matrix product),
  4. compares the pairs' log-probabilities with those of the model it started
     from, and takes the gradient of the loss  (tbe_preference_loss),
  5. goes back through the recurrence          (tbe_gated_scan_backward),
  6. updates the table's rows that were read   (tbe_backward_update, exact
     row-wise Adagrad) and the dense parameters (tbe_adamw_step).

    python examples/sequence_preference.py [--steps 60] [--state-bits 8]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bags_gb300 as tbe  # noqa: E402


class Model:
    """Table, projection, recurrence and output layer, with their optimizer."""

    def __init__(self, items=2000, dim=64, hidden=96, state_bits=32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=g, device="cuda") / rows**0.5).bfloat16()

        self.items, self.dim, self.hidden = items, dim, hidden
        self.plan = tbe.Plan(1, [0, items], [0, dim], [0], [tbe.TBE_BF16], tbe.TBE_BF16)
        self.table = torch.randn(items, dim, generator=g, device="cuda").bfloat16()
        self.momentum = torch.zeros(items, device="cuda")
        self.w_in, self.w_out = weight(dim, 3 * hidden), weight(hidden, items)
        self.decay = torch.full((hidden,), -4.0, device="cuda")
        self.params = [self.w_in, self.w_out, self.decay]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.adamw = tbe.AdamWPlan(self.params, self.grads, state_bits=state_bits)
        self.steps = 0

    def forward(self, ids, offsets, keep):
        """Logits [tokens, items] and what the backward needs."""
        bags = torch.arange(ids.numel() + 1, device="cuda")  # one id per bag: the rows themselves
        rows = tbe.tbe_forward(self.plan, self.table.view(-1), ids, bags, ids.numel())
        proj = rows @ self.w_in
        parts = proj.split(self.hidden, dim=1)
        scan = tbe.tbe_gated_scan(*parts, self.decay, offsets, want_states=keep)
        return scan.h @ self.w_out, (bags, rows, proj, scan)

    def step(self, ids, labels, offsets, ref_logps, beta=0.2, learning_rate=2e-3, table_rate=0.05):
        """One step; returns the loss (on the device)."""
        logits, (bags, rows, proj, scan) = self.forward(ids, offsets, keep=True)
        out = tbe.tbe_preference_loss(logits, labels, offsets, ref_logps, beta=beta, dlogits=logits)  # in place
        dlogits = out.dlogits
        torch.mm(scan.h.t(), dlogits, out=self.grads[1])
        dh = dlogits @ self.w_out.t()
        dproj = torch.empty_like(proj)
        back = tbe.tbe_gated_scan_backward(dh, *proj.split(self.hidden, dim=1), self.decay, offsets, scan.states,
                                           out=dproj.split(self.hidden, dim=1))
        self.grads[2].copy_(back.ddecay)
        torch.mm(rows.t(), dproj, out=self.grads[0])
        drows = (dproj @ self.w_in.t()).float()
        tbe.tbe_backward_update(self.plan, self.table.view(-1), tbe.TBE_OPT_EXACT_ROWWISE_ADAGRAD, table_rate, drows, ids,
                                bags, ids.numel(), eps=1e-6, momentum=self.momentum)
        self.steps += 1
        tbe.tbe_adamw_step(self.adamw, self.steps, learning_rate)
        return out.loss


def make_pairs(items, pairs, seed=0, mean_length=20):
    """Histories of ``pairs`` users, twice (preferred, rejected), as ids and
    next-item labels; only the last three tokens are answered for.  Users of
    even items prefer even items."""
    rng = np.random.default_rng(seed)
    ids, labels, lengths = [], [], []
    for preferred in (True, False):
        user = np.random.default_rng(seed + 1)
        for _ in range(pairs):
            n, kind = max(5, user.poisson(mean_length)), user.integers(0, 2)
            history = 2 * user.integers(0, items // 2, n) + kind
            ending = 2 * rng.integers(0, items // 2, 3) + (kind if preferred else 1 - kind)
            tokens = np.concatenate([history, ending])
            target = np.concatenate([tokens[1:], [-1]])
            target[:n - 1] = -1
            ids.append(tokens[:-1])
            labels.append(target[:-1])
            lengths.append(len(tokens) - 1)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    return tuple(torch.from_numpy(np.concatenate(a) if isinstance(a, list) else a).cuda() for a in (ids, labels, offsets))


def train(steps=60, items=2000, pairs=64, state_bits=32, report=None):
    """Trains on one batch of pairs; returns the losses."""
    model = Model(items=items, state_bits=state_bits)
    ids, labels, offsets = make_pairs(items, pairs)
    logits, _ = model.forward(ids, offsets, keep=False)
    ref = torch.zeros(2 * pairs, device="cuda")
    ref = tbe.tbe_preference_loss(logits, labels, offsets, ref).seq_logps.clone()  # the model it starts from
    losses = []
    for k in range(steps):
        losses.append(model.step(ids, labels, offsets, ref).clone())
        if report and (k % 10 == 0 or k == steps - 1):
            report(f"step {k:3d}  loss {float(losses[-1]):.4f}")
    return [float(v) for v in losses]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    args = ap.parse_args()
    train(args.steps, state_bits=args.state_bits, report=print)
