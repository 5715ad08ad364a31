"""More operators of a sequence model beside the embedding tables, as cases to be measured and compared.

The two ends of a next-item model over jagged user histories:

* ``attention``: causal linear attention with a decay for each head over jagged sequences (prefill, training pass,
  single tokens),
* ``catalogue``: softmax cross entropy of hidden rows over every row of a catalogue's table, without keeping the logits
  (evaluation, and loss with both gradients).

``listed()`` gives fixed cases, ``draw()`` more of the same ranges; ``prepare`` makes what a program holds before the
call; ``run`` makes one pass, through the package where ``own`` is true and in elementary torch operations (fp32,
rounded once at the end) otherwise; ``exact`` computes the same outputs in 64 bits from the definitions.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
LOSS_SCALE = {"f16": 4096.0, "bf16": 1.0}  # keeps gradients of half precision above its smallest numbers
CHUNK = 64  # tokens that the plain form of the attention takes at once


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # serving: the next event of 64 users, eight heads
        {"name": "attention_step_bf16", "op": "attention", "pass": "step", "sequences": 64, "tokens": 64, "heads": 8,
         "d": 128, "type": "bf16", "index32": False, "state": True},
        # training on the mid-size batch's history lengths (2048 bags, Poisson(20)), 512 channels
        {"name": "attention_train_mid_bf16", "op": "attention", "pass": "train", "sequences": 2048, "tokens": 40_960,
         "heads": 8, "d": 64, "type": "bf16", "index32": False, "state": False},
        # reading 257 histories before serving them, states carried in, heads that are no power of two wide
        {"name": "attention_prefill_odd_f16", "op": "attention", "pass": "forward", "sequences": 257, "tokens": 8_191,
         "heads": 5, "d": 100, "type": "f16", "index32": True, "state": True},
        # reading three long histories, 512 channels
        {"name": "attention_prefill_long_bf16", "op": "attention", "pass": "forward", "sequences": 3,
         "tokens": 100_003, "heads": 4, "d": 128, "type": "bf16", "index32": False, "state": False},
        # training on two very long sequences, 1024 channels, states carried in
        {"name": "attention_train_long_f16", "op": "attention", "pass": "train", "sequences": 2, "tokens": 65_537,
         "heads": 16, "d": 64, "type": "f16", "index32": False, "state": True},
        # the loss alone on a handful of rows over a small catalogue
        {"name": "catalogue_eval_small_bf16", "op": "catalogue", "tokens": 8, "V": 1000, "D": 64, "type": "bf16",
         "grad": False, "pad": 0},
        # the loss alone for one step of 64 users over a table of a million rows, an odd number of them
        {"name": "catalogue_eval_million_bf16", "op": "catalogue", "tokens": 64, "V": 1_000_003, "D": 128,
         "type": "bf16", "grad": False, "pad": 0},
        # training on a few sequences over a small catalogue
        {"name": "catalogue_train_small_f16", "op": "catalogue", "tokens": 320, "V": 1000, "D": 128, "type": "f16",
         "grad": True, "pad": 0},
        # training over an odd-sized catalogue with rows of an odd width, hidden rows cut out of wider ones
        {"name": "catalogue_train_odd_f16", "op": "catalogue", "tokens": 4_001, "V": 10_007, "D": 250, "type": "f16",
         "grad": True, "pad": 13},
        # training over the rows of a mid-size table, the largest
        {"name": "catalogue_train_large_bf16", "op": "catalogue", "tokens": 8_192, "V": 100_000, "D": 512,
         "type": "bf16", "grad": True, "pad": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.5:
        what = rng.choice(["step", "forward", "train", "train"])
        heads = rng.randint(1, 16)
        d = rng.choice([32, 64, 64, 128, 128, rng.randint(16, 128)])
        if what == "step":
            sequences = tokens = _spread(rng, 1, 512)
        else:
            tokens = _spread(rng, 1, min(100_000, 64_000_000 // (heads * d)))
            # as many as leave the carried states (a square of d for each sequence and head) within 2 GB
            sequences = _spread(rng, 1, max(1, min(2048, tokens, 500_000_000 // (heads * d * d))))
        return {"op": "attention", "pass": what, "sequences": sequences, "tokens": tokens, "heads": heads, "d": d,
                "type": rng.choice(["bf16", "f16"]), "index32": rng.random() < 0.5,
                "state": what == "step" or rng.random() < 0.5}
    D = _spread(rng, 16, 512)
    if rng.random() < 0.6:
        D = D // 8 * 8
    V = _spread(rng, 50, 150_000)
    tokens = _spread(rng, 1, max(1, min(8192, 800_000_000 // V)))
    return {"op": "catalogue", "tokens": tokens, "V": V, "D": D, "type": rng.choice(["bf16", "f16"]),
            "grad": rng.random() < 0.7, "pad": rng.choice([0, 0, 3, -D % 64])}


def work(case):
    """Bytes and operations a pass cannot do without: each input read once, each output written once; the products of
    the definition (the recurrence's two per state element, the logits and what each gradient takes from them)."""
    if case["op"] == "attention":
        n, s = case["tokens"] * case["heads"] * case["d"], case["sequences"] * case["heads"] * case["d"] ** 2
        if case["pass"] == "step":
            return {"bytes": 8 * n + 8 * s, "flops": 4 * n * case["d"]}
        states = 8 * s if case["state"] else 0
        if case["pass"] == "forward":
            return {"bytes": 8 * n + states, "flops": 4 * n * case["d"]}
        return {"bytes": 16 * n + 2 * states, "flops": 16 * n * case["d"]}
    n, table, hidden = case["tokens"] * case["V"] * case["D"], case["V"] * case["D"], case["tokens"] * case["D"]
    sides = 2 if case["grad"] else 1
    return {"bytes": 2 * sides * (table + hidden) + 16 * case["tokens"], "flops": (6 if case["grad"] else 2) * n}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 32))

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": case}
    N = case["tokens"]
    if case["op"] == "attention":
        S, H, d, dt = case["sequences"], case["heads"], case["d"], DTYPES[case["type"]]
        # queries, keys and values are slices of one projection's output
        s["proj"] = normal(N, 3, H, d).to(dt)
        # heads remember about 2 to 2,000 tokens
        s["decay"] = torch.exp(-torch.rand(H, generator=gen, device="cuda") * math.log(1000.0) - math.log(2.0))
        if case["pass"] == "step":
            s["state"] = normal(S, H, d, d)
            return s
        share = rng.gamma(6.0, size=S)
        lengths = rng.multinomial(N, share / share.sum())  # empty sequences among them
        offsets = torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]))
        s["offsets"] = offsets.to("cuda", torch.int32 if case["index32"] else torch.int64)
        s["longest"] = int(lengths.max())
        s["chunks"] = int((-(-lengths // CHUNK)).sum())
        s["state"] = normal(S, H, d, d) if case["state"] else None
        if case["pass"] == "train":
            s["dout"] = normal(N, H, d).to(dt)
            s["dlast"] = normal(S, H, d, d) if case["state"] else None
        return s

    V, D, dt = case["V"], case["D"], DTYPES[case["type"]]
    s["hidden"] = normal(N, D + case["pad"]).to(dt)[:, :D]
    s["weights"] = normal(V, D, scale=2.0 / math.sqrt(D)).to(dt)
    # popular rows come first and are labels more often
    labels = (V * torch.rand(N, generator=gen, device="cuda", dtype=torch.float64).square()).long().clamp(max=V - 1)
    labels[torch.rand(N, generator=gen, device="cuda") < 0.1] = -1  # tokens that are not to be predicted
    s["labels"] = labels
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    if state["case"]["op"] == "attention":
        return _own_attention(state) if own else _plain_attention(state)
    return _own_catalogue(state) if own else _plain_catalogue(state)


def _scale(case):
    return 1.0 / math.sqrt(case["d"])


def _own_attention(s):
    import table_embedding_bags_gb300 as tbe

    case = s["case"]
    q, k, v = s["proj"].unbind(1)
    if case["pass"] == "step":
        return {"o": tbe.tbe_linear_attention_step(q, k, v, s["decay"], s["state"], scale=_scale(case)),
                "state": s["state"]}
    f = tbe.tbe_linear_attention(q, k, v, s["decay"], s["offsets"], s0=s["state"], scale=_scale(case),
                                 want_last=case["state"])
    out = {"o": f.o, "s_last": f.s_last} if case["state"] else {"o": f.o}
    if case["pass"] == "forward":
        return out
    dproj = torch.empty_like(s["proj"])
    b = tbe.tbe_linear_attention_backward(s["dout"], q, k, v, s["decay"], s["offsets"], s0=s["state"],
                                          ds_last=s["dlast"], scale=_scale(case), out=dproj.unbind(1))
    out["dproj"] = dproj
    return {**out, "ds0": b.ds0} if case["state"] else out


def _own_catalogue(s):
    import table_embedding_bags_gb300 as tbe

    r = tbe.tbe_catalogue_loss(s["hidden"], s["weights"], s["labels"], want_grad=s["case"]["grad"],
                               grad_scale=LOSS_SCALE[s["case"]["type"]])
    out = {"loss": r.loss, "token_loss": r.token_loss}
    return {**out, "dhidden": r.dhidden, "dweights": r.dweights} if s["case"]["grad"] else out


def _chunked(s):
    """Each sequence's tokens in chunks of CHUNK rows: the token of each place (clamped where there is none), whether
    there is one, each chunk's sequence, whether it is the sequence's first and how many tokens it holds."""
    offsets = s["offsets"].long()
    count = (offsets[1:] - offsets[:-1] + CHUNK - 1) // CHUNK
    seq = torch.repeat_interleave(torch.arange(len(count), device="cuda"), count, output_size=s["chunks"])
    number = torch.arange(s["chunks"], device="cuda") - (torch.cumsum(count, 0) - count)[seq]
    token = (offsets[seq] + number * CHUNK)[:, None] + torch.arange(CHUNK, device="cuda")
    there = token < offsets[seq + 1][:, None]
    return token.clamp(max=s["case"]["tokens"] - 1), there, seq, number == 0, there.sum(1)


def _recurrence(s, q, k, v, state, reverse):
    """sum over the sequence's earlier (or, reversed, later) tokens of gamma^distance (q . k) v, in chunks; `state`
    comes before the first (behind the last) token. Returns the rows and the state behind the last token."""
    case, H, d = s["case"], s["case"]["heads"], s["case"]["d"]
    token, there, seq, first, filled = s["plan"]
    decay = s["decay"]

    def power(n):  # [H] by the shape of n
        return torch.exp(-decay.view(H, *[1] * n.dim()) * n.float())

    def rows(x):
        return torch.where(there[:, :, None, None], x[token].float(), 0.0).permute(2, 0, 1, 3)  # [H, chunks, CHUNK, d]

    q, k, v = rows(q), rows(k), rows(v)
    at = torch.arange(CHUNK, device="cuda")
    late = 1 if reverse else 0
    distance = at[None, :] - at[:, None] if reverse else at[:, None] - at[None, :]
    weight = torch.where(distance >= 0, power(distance.clamp(min=0)), 0.0)  # [H, CHUNK, CHUNK]
    out = (q @ k.transpose(-1, -2) * weight[:, None]) @ v
    # how far each place is from its chunk's end (the side that the state leaves by) and from its start
    to_end = at.expand_as(there) + 1 if reverse else filled[:, None] - 1 - at
    from_start = filled[:, None] - 1 - at if reverse else at.expand_as(there) + 1
    local = (k * torch.where(there, power(to_end.clamp(min=0)), 0.0)[..., None]).transpose(-1, -2) @ v
    # the states behind each chunk, over the chunks of its sequence: a doubling of the reach with each pass
    if reverse:
        order = torch.arange(s["chunks"] - 1, -1, -1, device="cuda")
        edge = torch.cat([first[1:], first.new_ones(1)])[order]
    else:
        order, edge = torch.arange(s["chunks"], device="cuda"), first
    carry = power(filled)[:, order]
    total = local[:, order]
    if state is not None:
        total = total + torch.where(edge, carry, 0.0)[..., None, None] * state.transpose(0, 1)[:, seq[order]]
    reach = torch.where(edge, 0.0, carry)
    step = 1
    while step < -(-s["longest"] // CHUNK):
        moved = reach[:, step:, None, None] * total[:, :-step]
        total = torch.cat([total[:, :step], total[:, step:] + moved], 1)
        reach = torch.cat([reach[:, :step], reach[:, step:] * reach[:, :-step]], 1)
        step *= 2
    before = torch.cat([torch.zeros_like(total[:, :1]), total[:, :-1]], 1)
    found = torch.zeros_like(before) if state is None else state.transpose(0, 1)[:, seq[order]]
    before = torch.where(edge[:, None, None], found, before)
    out = out + power(from_start.clamp(min=0))[..., None] * (q @ before[:, order])  # the order is its own inverse
    rows_out = torch.zeros(case["tokens"], H, d, device="cuda")
    rows_out[token[there]] = out.permute(1, 2, 0, 3)[there]
    if state is None:
        return rows_out, None
    last = state.clone()  # an empty sequence hands its state on
    ends = torch.cat([edge[1:], edge.new_ones(1)])
    last[seq[order][ends]] = total[:, ends].transpose(0, 1)
    return rows_out, last


def _plain_attention(s):
    case = s["case"]
    q, k, v = s["proj"].unbind(1)
    dt, scale = s["proj"].dtype, _scale(case)
    if case["pass"] == "step":
        q, k, v = q.float(), k.float(), v.float()
        gamma = torch.exp(-s["decay"])[:, None, None]
        s["state"].copy_(gamma * s["state"] + k[..., :, None] * v[..., None, :])
        return {"o": (scale * (q[..., None, :] @ s["state"]).squeeze(-2)).to(dt), "state": s["state"]}
    s["plan"] = _chunked(s)
    o, last = _recurrence(s, q, k, v, s["state"], False)
    out = {"o": (scale * o).to(dt)}
    if case["state"]:
        out["s_last"] = last
    if case["pass"] == "forward":
        return out
    s0, dlast = s["state"], s["dlast"]
    turned = dlast
    if case["state"]:  # the gradients are scaled as the output is; what comes in from behind is not
        s0, dlast = s0.transpose(-1, -2), dlast / scale
        turned = dlast.transpose(-1, -2)
    dq, _ = _recurrence(s, s["dout"], v, k, s0, False)
    dk, _ = _recurrence(s, v, s["dout"], q, turned, True)
    dv, ds0 = _recurrence(s, k, q, s["dout"], dlast, True)
    out["dproj"] = (scale * torch.stack([dq, dk, dv], 1)).to(dt)
    return {**out, "ds0": scale * ds0} if case["state"] else out


def _plain_catalogue(s):
    h, w = s["hidden"].float(), s["weights"].float()
    taken = s["labels"] >= 0
    label = s["labels"].clamp(min=0)
    logits = h @ w.T
    top = logits.amax(1, keepdim=True)
    mine = logits.gather(1, label[:, None])
    e = torch.exp(logits - top)
    z = e.sum(1, keepdim=True)
    token_loss = torch.where(taken, (top - mine + torch.log(z)).squeeze(1), 0.0)
    count = taken.sum().clamp(min=1)
    out = {"loss": token_loss.sum() / count, "token_loss": token_loss}
    if s["case"]["grad"]:
        share = (taken * LOSS_SCALE[s["case"]["type"]] / count)[:, None]
        g = e.mul_(share / z)
        g.scatter_add_(1, label[:, None], -share)
        out["dhidden"] = (g @ w).to(s["hidden"].dtype)
        out["dweights"] = (g.T @ h).to(s["weights"].dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attention" else _exact_catalogue(s)


def _walk(q, k, v, gamma, state, lengths, behind):
    """The recurrence on [S, L, H, d] tensors of S padded sequences, a block of rows after the other. The state moves on
    before a token reads it (S_t = gamma S_{t-1} + k v^T); `behind` says that gamma comes behind the read instead."""
    S, L, H, d = q.shape
    out = torch.zeros_like(q)
    step = 32
    n = torch.arange(step, device="cuda", dtype=torch.float64)
    apart = n[:, None] - n[None, :]
    mask = torch.where(apart >= 0, gamma[:, None, None] ** apart.clamp(min=0), 0.0)  # [H, step, step]
    for t in range(0, L, step):
        m = min(step, L - t)
        a, b, c = (x[:, t:t + m].transpose(1, 2) for x in (q, k, v))  # [S, H, m, d]
        left = (lengths[:, None] - t).clamp(0, m)  # [S, 1] tokens of this block
        reads = gamma[:, None] ** (n[:m] + (0 if behind else 1))  # [H, m]
        o = (torch.einsum("shid,shjd->shij", a, b) * mask[:, :m, :m]) @ c
        o += reads[..., None] * (a @ state)
        out[:, t:t + m] = o.transpose(1, 2)
        # weight of row j in the state behind the block's last token
        expo = left[:, :, None] - 1 - n[:m] + (1 if behind else 0)  # [S, 1, m]
        w = torch.where(n[:m] < left[:, :, None], gamma[None, :, None] ** expo.clamp(min=0), 0.0)  # [S, H, m]
        state = gamma[None, :, None, None] ** left.double()[:, :, None, None] * state + (b * w[..., None]).transpose(-1, -2) @ c
    return out, state


def _exact_attention(s):
    case = s["case"]
    N, S, H, d = case["tokens"], case["sequences"], case["heads"], case["d"]
    gamma, scale = torch.exp(-s["decay"].double()), _scale(case)
    q, k, v = s["proj"].double().unbind(1)
    if case["pass"] == "step":
        state = s["state"].double() * gamma[:, None, None] + torch.einsum("nhi,nhj->nhij", k, v)
        return {"o": scale * torch.einsum("nhi,nhij->nhj", q, state), "state": state}
    offsets = s["offsets"].long()
    lengths = offsets[1:] - offsets[:-1]
    L = s["longest"]
    if S * L > 40 * N + 4096:
        return None  # too much of the padded form is padding
    place = offsets[:-1, None] + torch.arange(L, device="cuda")
    there = torch.arange(L, device="cuda") < lengths[:, None]
    # turned round, a sequence's last token comes first
    turned = offsets[1:, None] - 1 - torch.arange(L, device="cuda")

    def padded(x, where):
        return torch.where(there[:, :, None, None], x[where.clamp(0, N - 1)], 0.0)

    def flat(x, where):
        y = torch.zeros(N, H, d, dtype=torch.float64, device="cuda")
        y[where[there]] = x[there]
        return y

    none = torch.zeros(S, H, d, d, dtype=torch.float64, device="cuda")
    s0 = none if s["state"] is None else s["state"].double()
    o, last = _walk(padded(q, place), padded(k, place), padded(v, place), gamma, s0, lengths, False)
    out = {"o": scale * flat(o, place)}
    if case["state"]:
        out["s_last"] = last
    if case["pass"] == "forward":
        return out
    # d loss / d o_t, by the chain: g_t = d loss / d S_t = scale q_t do_t^T + gamma g_{t+1}
    do = scale * s["dout"].double()
    dlast = none if s["dlast"] is None else s["dlast"].double()
    dq, _ = _walk(padded(do, place), padded(v, place), padded(k, place), gamma, s0.transpose(-1, -2), lengths, False)
    dv, ds0 = _walk(padded(k, turned), padded(q, turned), padded(do, turned), gamma, dlast, lengths, True)
    dk, _ = _walk(padded(v, turned), padded(do, turned), padded(q, turned), gamma, dlast.transpose(-1, -2), lengths, True)
    out["dproj"] = torch.stack([flat(dq, place), flat(dk, turned), flat(dv, turned)], 1)
    return {**out, "ds0": ds0} if case["state"] else out


def _exact_catalogue(s):
    case = s["case"]
    N, V, D = case["tokens"], case["V"], case["D"]
    rows = torch.nonzero(s["labels"] >= 0).squeeze(1)
    count = max(1, len(rows))
    w = s["weights"].double()
    token_loss = torch.zeros(N, dtype=torch.float64, device="cuda")
    dh = torch.zeros(N, D, dtype=torch.float64, device="cuda")
    dw = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    for part in rows.split(512):
        x, y = s["hidden"][part].double(), s["labels"][part]
        logits = x @ w.T
        token_loss[part] = torch.logsumexp(logits, 1) - logits[torch.arange(len(part), device="cuda"), y]
        if case["grad"]:
            p = torch.softmax(logits, 1)
            p[torch.arange(len(part), device="cuda"), y] -= 1
            p *= LOSS_SCALE[case["type"]] / count
            dh[part] = p @ w
            dw += p.T @ x
    out = {"loss": token_loss.sum() / count, "token_loss": token_loss}
    return {**out, "dhidden": dh, "dweights": dw} if case["grad"] else out
