"""Next-item prediction over jagged histories with one table for both ends, on synthetic data.

A step

  1. looks the histories' items up in the table     (tbe_forward, one id per bag),
  2. mixes each history                             (a projection, tbe_linear_attention),
  3. takes the softmax cross entropy over every row of the same table, with
     its gradients, without logits                  (tbe_catalogue_loss),
  4. goes back through the attention                (tbe_linear_attention_backward),
  5. sums the lookups' gradients by row             (tbe_backward),
  6. updates the table and the projection           (tbe_adamw_step).

Serving reads a history once (want_last) and then takes one event at a time
(tbe_linear_attention_step).

    python examples/next_item.py [--steps 60]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import table_embedding_bags_gb300 as tbe  # noqa: E402


class Model:
    """A table of items and one attention layer of ``heads`` heads as wide as its rows."""

    def __init__(self, items=2000, heads=4, head_dim=32, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.items, self.heads, self.head_dim, self.width = items, heads, head_dim, heads * head_dim
        self.scale = head_dim**-0.5
        self.plan = tbe.Plan(1, [0, items], [0, self.width], [0], [tbe.TBE_BF16], tbe.TBE_BF16)
        self.table = (torch.randn(items, self.width, generator=g, device="cuda") * self.width**-0.25).bfloat16()
        self.proj = (torch.randn(self.width, 3 * self.width, generator=g, device="cuda") * self.width**-0.5).bfloat16()
        self.decay = 2.0 ** -torch.arange(1, heads + 1, device="cuda", dtype=torch.float32)
        self.params = [self.table, self.proj]
        self.grads = [torch.zeros_like(p) for p in self.params]
        self.adamw = tbe.AdamWPlan(self.params, self.grads)
        self.steps = 0

    def qkv(self, ids):
        ids = ids.contiguous()
        bags = torch.arange(ids.numel() + 1, device="cuda")  # one id per bag: the rows themselves
        rows = tbe.tbe_forward(self.plan, self.table.view(-1), ids, bags, ids.numel())
        return rows, bags, (rows @ self.proj).view(-1, 3, self.heads, self.head_dim)

    def gradients(self, ids, labels, offsets):
        """Loss, and both parameters' gradients in ``grads``."""
        rows, bags, qkv = self.qkv(ids)
        q, k, v = qkv.unbind(1)
        f = tbe.tbe_linear_attention(q, k, v, self.decay, offsets, scale=self.scale)
        loss = tbe.tbe_catalogue_loss(f.o.view(-1, self.width), self.table, labels, want_grad=True)
        dqkv = torch.empty_like(qkv)
        tbe.tbe_linear_attention_backward(loss.dhidden.view_as(f.o), q, k, v, self.decay, offsets, scale=self.scale,
                                          out=dqkv.unbind(1))
        dqkv = dqkv.view(ids.numel(), -1)
        torch.mm(rows.t(), dqkv, out=self.grads[1])
        drows = (dqkv @ self.proj.t()).float()
        b = tbe.tbe_backward(self.plan, drows, ids, bags, ids.numel())
        n = int(b.unique_count[-1])
        lookups = b.row_grads[:n * self.width].view(n, self.width)
        self.grads[0].copy_(loss.dweights.float().index_add_(0, b.unique_rows[:n], lookups))
        return loss.loss

    def step(self, ids, labels, offsets, learning_rate=3e-3):
        loss = self.gradients(ids, labels, offsets)
        self.steps += 1
        tbe.tbe_adamw_step(self.adamw, self.steps, learning_rate)
        return loss

    def read(self, ids, offsets):
        """Hidden rows of whole histories, and the state that each leaves."""
        _, _, qkv = self.qkv(ids)
        f = tbe.tbe_linear_attention(*qkv.unbind(1), self.decay, offsets, scale=self.scale, want_last=True)
        return f.o.view(-1, self.width), f.s_last

    def event(self, ids, state):
        """Hidden rows after one more event of each history, whose state moves on."""
        _, _, qkv = self.qkv(ids)
        return tbe.tbe_linear_attention_step(*qkv.unbind(1), self.decay, state, scale=self.scale).view(-1, self.width)


def make_histories(items, users, seed=0, mean_length=20):
    """Ids, next-item labels (-1 behind the last) and offsets: users walk the items in steps of their own."""
    rng = np.random.default_rng(seed)
    ids, labels, lengths = [], [], []
    for _ in range(users):
        n = max(2, rng.poisson(mean_length))
        walk = (rng.integers(items) + rng.integers(1, 4) * np.arange(n)) % items
        ids.append(walk)
        labels.append(np.append(walk[1:], -1))
        lengths.append(n)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    return tuple(torch.from_numpy(np.asarray(a, dtype=np.int64)).cuda() for a in
                 (np.concatenate(ids), np.concatenate(labels), offsets))


def train(steps=60, items=2000, users=256, report=None):
    model = Model(items=items)
    batch = make_histories(items, users)
    for k in range(steps):
        loss = model.step(*batch)
        if report and (k % 10 == 0 or k == steps - 1):
            report(f"step {k:3d}  loss {float(loss):.4f}")
    return model, float(loss)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    train(ap.parse_args().steps, report=print)
