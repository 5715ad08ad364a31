"""The training operators beside the embedding tables, as cases to be measured and compared.

Three operators make up a training step of a sequence model over jagged user histories, next to the tables' own
forward and backward:

* ``scan``: a gated linear recurrence over jagged sequences (prefill, training pass, single tokens),
* ``preference``: a paired-log-ratio loss over catalogue logits (evaluation, and loss with gradient),
* ``adamw``: one AdamW step over a list of dense tensors (32-bit or 8-bit states).

``listed()`` gives fixed cases, ``draw()`` more of the same ranges; ``prepare`` makes what a program holds before the
call; ``run`` makes one pass, through the package where ``own`` is true and in elementary torch operations (fp32,
rounded once at the end) otherwise; ``exact`` computes the same outputs in 64 bits from the definitions.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
SHARPNESS = 8.0
BLOCK = 256  # elements of a block of optimizer state; every tensor's state starts on a block
ADAM = {"learning_rate": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "weight_decay": 0.01, "step": 1000}
PREF = {"beta": 0.1, "label_smoothing": 0.05}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the top network beside the mid-size tables (8 x 128 columns in): 1024 -> 512 -> 256 -> 1 with its biases
        {"name": "adamw_small_f32", "op": "adamw", "tensors": 6, "total": 656_129, "ptype": "f32", "gtype": "f32",
         "bits": 32, "flat": False},
        # a larger dense network in half precision, states in 8 bits, tensors of ragged sizes
        {"name": "adamw_bf16_8bit", "op": "adamw", "tensors": 56, "total": 64_000_003, "ptype": "bf16",
         "gtype": "bf16", "bits": 8, "flat": False},
        # the largest step: half-precision parameters and gradients, full states
        {"name": "adamw_bf16_32bit", "op": "adamw", "tensors": 40, "total": 200_000_000, "ptype": "bf16",
         "gtype": "bf16", "bits": 32, "flat": False},
        # serving: the next event of 64 users
        {"name": "scan_step_bf16", "op": "scan", "pass": "step", "sequences": 64, "tokens": 64, "C": 256,
         "type": "bf16", "index32": False, "h0": True},
        # training on the mid-size batch's history lengths (2048 bags, Poisson(20)), one table's width
        {"name": "scan_train_mid_bf16", "op": "scan", "pass": "train", "sequences": 2048, "tokens": 40_960, "C": 128,
         "type": "bf16", "index32": False, "h0": False},
        # training in full precision, a width that is no multiple of a vector, state carried in
        {"name": "scan_train_odd_f32", "op": "scan", "pass": "train", "sequences": 257, "tokens": 8_191, "C": 250,
         "type": "f32", "index32": True, "h0": True},
        # reading three long histories before serving them
        {"name": "scan_prefill_long_f16", "op": "scan", "pass": "forward", "sequences": 3, "tokens": 100_003,
         "C": 512, "type": "f16", "index32": False, "h0": False},
        # training on two very long sequences
        {"name": "scan_train_long_bf16", "op": "scan", "pass": "train", "sequences": 2, "tokens": 65_537, "C": 1024,
         "type": "bf16", "index32": False, "h0": True},
        # the loss alone on a handful of pairs over a small catalogue
        {"name": "pref_eval_small_f32", "op": "preference", "pairs": 8, "tokens": 80, "V": 1000, "type": "f32",
         "grad": False, "pad": 0},
        # one pair over a mid-size table's 100,000 rows: few rows, each long
        {"name": "pref_train_one_pair_f32", "op": "preference", "pairs": 1, "tokens": 6, "V": 100_000, "type": "f32",
         "grad": True, "pad": 0},
        # training over an odd-sized catalogue, rows padded to a multiple of 64
        {"name": "pref_train_odd_f16", "op": "preference", "pairs": 48, "tokens": 1_300, "V": 10_007, "type": "f16",
         "grad": True, "pad": 41},
        # training over the rows of a mid-size table, the largest
        {"name": "pref_train_large_bf16", "op": "preference", "pairs": 96, "tokens": 3_840, "V": 100_000,
         "type": "bf16", "grad": True, "pad": 0},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adamw", "scan", "scan", "preference"])
    if op == "adamw":
        tensors = rng.randint(1, 56)
        return {"op": op, "tensors": tensors, "total": _spread(rng, 1000 + 64 * tensors, 100_000_000),
                "ptype": rng.choice(["f32", "bf16", "f16"]), "gtype": rng.choice(["f32", "bf16"]),
                "bits": rng.choice([8, 32]), "flat": rng.random() < 0.3}
    if op == "scan":
        what = rng.choice(["step", "forward", "train", "train"])
        C = _spread(rng, 16, 1024)
        if rng.random() < 0.6:
            C = max(16, C // 8 * 8)
        if what == "step":
            sequences = tokens = _spread(rng, 1, 4096)
        else:
            tokens = _spread(rng, 1, min(100_000, 64_000_000 // C))
            sequences = _spread(rng, 1, max(1, min(4096, tokens)))
        return {"op": op, "pass": what, "sequences": sequences, "tokens": tokens, "C": C,
                "type": rng.choice(["f32", "bf16", "f16"]), "index32": rng.random() < 0.5, "h0": rng.random() < 0.5}
    V = _spread(rng, 50, 120_000)
    tokens = _spread(rng, 2, max(2, min(8000, 250_000_000 // V)))
    return {"op": op, "pairs": _spread(rng, 1, max(1, tokens // 4)), "tokens": tokens, "V": V,
            "type": rng.choice(["f32", "bf16", "f16"]) if V * tokens < 100_000_000 else "bf16",
            "grad": rng.random() < 0.75, "pad": rng.choice([0, 0, 5, -V % 64])}


def work(case):
    """Bytes and operations a pass cannot do without: each input read once, each output written once."""
    if case["op"] == "adamw":
        n, p, g = case["total"], BYTES[case["ptype"]], BYTES[case["gtype"]]
        # 8-bit states: codes read and written, and the values they stand for written for the caller
        state = 16 if case["bits"] == 32 else 4 + 8
        return {"bytes": n * (2 * p + g + state), "flops": 15 * n}
    if case["op"] == "scan":
        n, s, e = case["tokens"] * case["C"], case["sequences"] * case["C"], BYTES[case["type"]]
        carried = (4 if case["h0"] else 0) * s
        if case["pass"] == "step":
            return {"bytes": 4 * n * e + 8 * s, "flops": 20 * n}
        if case["pass"] == "forward":
            return {"bytes": 4 * n * e + carried + 4 * s, "flops": 20 * n}
        # x, r, g and dh read, h and three gradients written; states, their gradients and the decay's
        return {"bytes": 8 * n * e + 2 * carried + 8 * s, "flops": 55 * n}
    n, e = case["tokens"] * case["V"], BYTES[case["type"]]
    return {"bytes": n * e * (2 if case["grad"] else 1), "flops": n * (9 if case["grad"] else 5)}


# ---------------------------------------------------------------------------
# what a program has in hand
# ---------------------------------------------------------------------------

def _sizes(case):
    """Sizes of the list's tensors: spread over two decades, biases among them, odd, adding up to the total."""
    n, total = case["tensors"], case["total"]
    if n == 6 and total == 656_129:
        return [1024 * 512, 512, 512 * 256, 256, 256, 1]
    share = np.exp(np.random.RandomState(n).uniform(-2.3, 2.3, n))
    sizes = 1 + np.floor((total - n) * share / share.sum()).astype(np.int64)
    sizes[0] += total - sizes.sum()
    return [int(v) for v in sizes]


def _lengths(count, tokens, rng):
    """`count` lengths that add up to `tokens`, empty ones among them."""
    share = rng.gamma(6.0, size=count)
    return rng.multinomial(tokens, share / share.sum())


def _offsets(lengths, dtype):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)])).to("cuda", dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    rng = np.random.RandomState(int(seed) % (1 << 32))

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * scale

    s = {"case": case}
    if case["op"] == "adamw":
        sizes = _sizes(case)
        total = sum(sizes)
        padded = sum(-(-n // BLOCK) * BLOCK for n in sizes)

        def split(flat):
            views = flat.split(sizes)
            return list(views) if case["flat"] else [v.clone() for v in views]

        # a tenth of the gradients is exactly zero (units that did not fire)
        g = normal(total, scale=1e-3) * (torch.rand(total, generator=gen, device="cuda") >= 0.1)
        s["params"] = split(normal(total, scale=0.05).to(DTYPES[case["ptype"]]))
        s["grads"] = split(g.to(DTYPES[case["gtype"]]))
        del g
        edge = torch.ones(padded, dtype=torch.bool, device="cuda")  # the padding behind each tensor stays zero
        at = 0
        for n in sizes:
            edge[at + n:at + -(-n // BLOCK) * BLOCK] = False
            at += -(-n // BLOCK) * BLOCK
        m = normal(padded, scale=3e-4) * edge
        v = (normal(padded, scale=1e-3).square() * 0.5 + 2e-8) * edge
        if case["bits"] == 32:
            s["exp_avg"], s["exp_avg_sq"] = m, v
        else:
            blocks = padded // BLOCK
            sm = torch.rand(blocks, generator=gen, device="cuda") * 2e-3 + 1e-4
            sv = torch.rand(blocks, generator=gen, device="cuda") * 1e-5 + 1e-7
            code = (m.view(blocks, BLOCK).abs() / 1.5e-3).clamp(max=1).sqrt().mul(127).round() * m.view(blocks, BLOCK).sign()
            s["exp_avg"] = code.to(torch.int8).view(-1)
            s["exp_avg_sq"] = (v.view(blocks, BLOCK) / 8e-6).clamp(max=1).pow(0.25).mul(255).round().to(torch.uint8).view(-1)
            s["exp_avg_scale"], s["exp_avg_sq_scale"] = sm, sv
        if own:  # the handle that a program makes once for its list of tensors
            import table_embedding_bags_gb300 as tbe

            keep = {k: s[k] for k in ("exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale") if k in s}
            s["plan"] = tbe.AdamWPlan(s["params"], s["grads"], state_bits=case["bits"], state=keep)
        return s

    if case["op"] == "scan":
        N, S, C, dt = case["tokens"], case["sequences"], case["C"], DTYPES[case["type"]]
        # the three inputs are slices of one projection's output
        s["proj"] = normal(N, 3 * C).to(dt)
        # decays of one step between 0.9 and 0.999 where the gate is open
        u = -torch.log(0.9 + 0.099 * torch.rand(C, generator=gen, device="cuda")) / SHARPNESS
        s["decay"] = torch.log(torch.expm1(u))
        if case["pass"] == "step":
            s["state"] = normal(S, C)
            return s
        lengths = _lengths(S, N, rng)
        s["offsets"] = _offsets(lengths, torch.int32 if case["index32"] else torch.int64)
        s["longest"] = int(lengths.max())
        s["h0"] = normal(S, C) if case["h0"] else None
        if case["pass"] == "train":
            s["dh"] = normal(N, C).to(dt)
            s["dh_last"] = normal(S, C)
        return s

    P, N, V = case["pairs"], case["tokens"], case["V"]
    lengths = _lengths(2 * P, N, rng)
    s["logits"] = normal(N, V + case["pad"], scale=2.0).to(DTYPES[case["type"]])[:, :V]
    labels = torch.randint(0, V, (N,), generator=gen, device="cuda")
    labels[torch.rand(N, generator=gen, device="cuda") < 0.1] = -1  # tokens of the prompt
    s["labels"] = labels
    s["offsets"] = _offsets(lengths, torch.int64)
    s["lengths"] = torch.from_numpy(lengths).cuda()
    expected = torch.from_numpy(lengths).to("cuda", torch.float32) * -0.9 * (math.log(V) + 2.0)
    s["ref_logps"] = expected + normal(2 * P, scale=3.0)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if case["op"] == "adamw":
        return _own_adamw(state) if own else _plain_adamw(state)
    if case["op"] == "scan":
        return _own_scan(state) if own else _plain_scan(state)
    return _own_preference(state) if own else _plain_preference(state)


def _own_adamw(s):
    import table_embedding_bags_gb300 as tbe

    tbe.tbe_adamw_step(s["plan"], **ADAM)
    if s["case"]["bits"] == 8:
        m, v = tbe.tbe_adamw_state(s["plan"])
    else:
        m, v = s["plan"].exp_avg, s["plan"].exp_avg_sq
    return {"params": s["params"], "exp_avg": m, "exp_avg_sq": v}


def _own_scan(s):
    import table_embedding_bags_gb300 as tbe

    case, C = s["case"], s["case"]["C"]
    x, recur, gate = s["proj"][:, :C], s["proj"][:, C:2 * C], s["proj"][:, 2 * C:]
    if case["pass"] == "step":
        return {"h": tbe.tbe_gated_scan_step(x, recur, gate, s["decay"], s["state"], sharpness=SHARPNESS),
                "state": s["state"]}
    train = case["pass"] == "train"
    f = tbe.tbe_gated_scan(x, recur, gate, s["decay"], s["offsets"], h0=s["h0"], sharpness=SHARPNESS,
                           want_states=train)
    if not train:
        return {"h": f.h, "h_last": f.h_last}
    dproj = torch.empty_like(s["proj"])
    b = tbe.tbe_gated_scan_backward(s["dh"], x, recur, gate, s["decay"], s["offsets"], f.states, h0=s["h0"],
                                    dh_last=s["dh_last"], sharpness=SHARPNESS,
                                    out=(dproj[:, :C], dproj[:, C:2 * C], dproj[:, 2 * C:]))
    out = {"h": f.h, "h_last": f.h_last, "dproj": dproj, "ddecay": b.ddecay}
    return {**out, "dh0": b.dh0} if case["h0"] else out


def _own_preference(s):
    import table_embedding_bags_gb300 as tbe

    r = tbe.tbe_preference_loss(s["logits"], s["labels"], s["offsets"], s["ref_logps"], want_grad=s["case"]["grad"],
                                **PREF)
    out = {"loss": r.loss, "seq_logps": r.seq_logps}
    return {**out, "dlogits": r.dlogits} if s["case"]["grad"] else out


def _padded(tensors):
    return torch.cat([torch.nn.functional.pad(t.reshape(-1).float(), (0, -t.numel() % BLOCK)) for t in tensors])


def _levels(count, power):
    """Where a code's neighbour begins: half-way between two codes, in the domain where codes are evenly spaced."""
    return torch.tensor([((k - 0.5) / count) ** power for k in range(1, count + 1)], dtype=torch.float32, device="cuda")


def _scaled(x):
    """Each block's largest magnitude, and the block divided by it (zero where there is nothing to divide by)."""
    top = x.view(-1, BLOCK).abs().amax(1)
    top = torch.where(top >= torch.finfo(torch.float32).tiny, top, 0.0)
    inverse = torch.where(top > 0, torch.ones_like(top) / top, 0.0)
    return top, (x.view(-1, BLOCK).abs() * inverse[:, None]).contiguous()


def _plain_adamw(s):
    case, a = s["case"], ADAM
    p, g = _padded(s["params"]), _padded(s["grads"])
    if case["bits"] == 32:
        m, v = s["exp_avg"], s["exp_avg_sq"]
    else:
        q = s["exp_avg"].view(-1, BLOCK).float()
        m = (q * q.abs() * (s["exp_avg_scale"] * (1 / 127**2))[:, None]).view(-1)
        q = s["exp_avg_sq"].view(-1, BLOCK).float()
        q = q * q
        v = (q * q * (s["exp_avg_sq_scale"] * (1 / 255**4))[:, None]).view(-1)
    m = m * a["beta1"] + g * (1 - a["beta1"])
    v = v * a["beta2"] + g * g * (1 - a["beta2"])
    size = a["learning_rate"] / (1 - a["beta1"] ** a["step"])
    root = v.sqrt() * (1 / math.sqrt(1 - a["beta2"] ** a["step"])) + a["eps"]
    p = p * (1 - a["learning_rate"] * a["weight_decay"]) - size * (m / root)
    if case["bits"] == 32:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    else:
        top, y = _scaled(m)
        code = torch.bucketize(y, _levels(127, 2), right=True).float() * m.view(-1, BLOCK).sign()
        s["exp_avg"].copy_(code.view(-1))
        s["exp_avg_scale"].copy_(top)
        m = (code * code.abs() * (top * (1 / 127**2))[:, None]).view(-1)
        top, y = _scaled(v)
        code = torch.bucketize(y, _levels(255, 4), right=True)
        # a second moment that is not zero is never held as zero: it is divided by
        code = torch.maximum(code, (y > 0).long()).float()
        s["exp_avg_sq"].copy_(code.view(-1))
        s["exp_avg_sq_scale"].copy_(top)
        code = code * code
        v = (code * code * (top * (1 / 255**4))[:, None]).view(-1)
    lengths = [t.numel() for t in s["params"]]
    pieces = p.split([-(-n // BLOCK) * BLOCK for n in lengths])
    [t.copy_(x[:n].view(t.shape)) for t, x, n in zip(s["params"], pieces, lengths)]
    return {"params": s["params"], "exp_avg": m, "exp_avg_sq": v}


def _gates(s, proj):
    C = s["case"]["C"]
    x, r, g = (t.float() for t in proj.split(C, dim=1))
    sr, sg = torch.sigmoid(r), torch.sigmoid(g)
    u = SHARPNESS * torch.nn.functional.softplus(s["decay"]) * sr
    a = torch.exp(-u)
    beta = torch.sqrt(-torch.expm1(-2 * u))
    return x, sr, sg, u, a, beta


def _doubling(a, b, longest):
    """h_t = a_t h_{t-1} + b_t down the rows; a is 0 where a sequence starts. log2(longest) passes over the rows."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _plain_scan(s):
    case = s["case"]
    x, sr, sg, u, a, beta = _gates(s, s["proj"])
    dt = s["proj"].dtype
    if case["pass"] == "step":
        s["state"].copy_(a * s["state"] + beta * sg * x)
        return {"h": s["state"].to(dt), "state": s["state"]}
    offsets = s["offsets"].long()
    full = offsets[1:] > offsets[:-1]
    first, last = offsets[:-1][full], offsets[1:][full] - 1
    b = beta * sg * x
    before = torch.zeros_like(b)  # the state that each token finds
    if s["h0"] is not None:
        before[first] = s["h0"][full]
    b = b + a * before
    inner = a.clone()
    inner[first] = 0.0
    h = _doubling(inner, b, s["longest"])
    h_last = torch.zeros_like(s["h0"]) if s["h0"] is not None else torch.zeros(case["sequences"], case["C"], device="cuda")
    if s["h0"] is not None:
        h_last[~full] = s["h0"][~full]
    h_last[full] = h[last]
    if case["pass"] == "forward":
        return {"h": h.to(dt), "h_last": h_last}
    # backward: G_t = dh_t + a_{t+1} G_{t+1}, down the rows turned round
    G = s["dh"].float().index_add(0, last, s["dh_last"][full])
    back = torch.cat([inner[1:], torch.zeros_like(inner[:1])])  # 0 behind each sequence's last token
    G = _doubling(back.flip(0), G.flip(0), s["longest"]).flip(0)
    previous = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    previous[first] = before[first]
    w = G * (torch.where(u > 0, u * a * a / beta, 0.0) * sg * x - u * a * previous)
    ratio = torch.sigmoid(s["decay"]) / torch.nn.functional.softplus(s["decay"])
    dproj = torch.cat([G * beta * sg, w * (1 - sr), G * beta * x * sg * (1 - sg)], dim=1)
    out = {"h": h.to(dt), "h_last": h_last, "dproj": dproj.to(dt), "ddecay": w.sum(0) * ratio}
    if s["h0"] is not None:
        dh0 = s["dh_last"].clone()  # an empty sequence hands its state on
        dh0[full] = (a * G)[first]
        out["dh0"] = dh0
    return out


def _plain_preference(s):
    case, P = s["case"], s["case"]["pairs"]
    x = s["logits"].float()
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(1, keepdim=True)
    lse = (top + torch.log(z)).squeeze(1)
    taken = s["labels"] >= 0
    label = s["labels"].clamp(min=0)
    lp = torch.where(taken, x.gather(1, label[:, None]).squeeze(1) - lse, 0.0)
    which = torch.repeat_interleave(torch.arange(2 * P, device="cuda"), s["lengths"], output_size=case["tokens"])
    logps = torch.zeros(2 * P, device="cuda").index_add_(0, which, lp)
    ratio = logps - s["ref_logps"]
    d = PREF["beta"] * (ratio[:P] - ratio[P:])
    eps = PREF["label_smoothing"]
    up, down = torch.sigmoid(d), torch.sigmoid(-d)
    soft = torch.clamp(-d, min=0) + torch.log1p(torch.exp(-d.abs()))  # log(1 + exp(-d))
    loss = ((1 - eps) * soft + eps * (soft + d)).mean()
    out = {"loss": loss, "seq_logps": logps}
    if case["grad"]:
        c = (eps * up - (1 - eps) * down) * (PREF["beta"] / P)
        c = torch.cat([c, -c])[which] * taken
        grad = e * (-c[:, None] / z)
        grad.scatter_add_(1, label[:, None], c[:, None])
        out["dlogits"] = grad.to(s["logits"].dtype)
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(s)
    if case["op"] == "scan":
        return _exact_scan(s)
    return _exact_preference(s)


def _exact_adamw(s):
    case, a = s["case"], ADAM
    b1, b2, t = a["beta1"], a["beta2"], a["step"]
    params, ms, vs, at = [], [], [], 0
    for p, g in zip(s["params"], s["grads"]):
        n = p.numel()
        end = at + -(-n // BLOCK) * BLOCK
        m, v = s["exp_avg"][at:end].double(), s["exp_avg_sq"][at:end].double()
        if case["bits"] == 8:
            block = slice(at // BLOCK, end // BLOCK)
            scale = s["exp_avg_scale"][block].double().repeat_interleave(BLOCK)
            m = m.sign() * (m / 127) ** 2 * scale
            v = (v / 255) ** 4 * s["exp_avg_sq_scale"][block].double().repeat_interleave(BLOCK)
        g = g.reshape(-1).double()
        m[:n] = b1 * m[:n] + (1 - b1) * g
        v[:n] = b2 * v[:n] + (1 - b2) * g**2
        hat_m, hat_v = m[:n] / (1 - b1**t), v[:n] / (1 - b2**t)
        w = p.reshape(-1).double()
        w = w - a["learning_rate"] * (hat_m / (hat_v.sqrt() + a["eps"]) + a["weight_decay"] * w)
        if case["bits"] == 8:
            top = m.view(-1, BLOCK).abs().amax(1, keepdim=True)
            code = torch.where(top > 0, (m.view(-1, BLOCK).abs() / top).sqrt() * 127, 0.0).round()
            m = (m.view(-1, BLOCK).sign() * (code / 127) ** 2 * top).view(-1)
            top = v.view(-1, BLOCK).amax(1, keepdim=True)
            code = torch.where(top > 0, (v.view(-1, BLOCK) / top) ** 0.25 * 255, 0.0).round()
            code = torch.maximum(code, (v.view(-1, BLOCK) > 0).double())
            v = ((code / 255) ** 4 * top).view(-1)
        params.append(w.view(p.shape))
        ms.append(m)
        vs.append(v)
        at = end
    return {"params": params, "exp_avg": torch.cat(ms), "exp_avg_sq": torch.cat(vs)}


def _exact_scan(s):
    """Token by token: at step t every sequence that is longer than t takes its token (longest sequences first)."""
    case, C = s["case"], s["case"]["C"]
    proj = s["proj"].double()
    x, r, g = proj[:, :C], proj[:, C:2 * C], proj[:, 2 * C:]
    speed = SHARPNESS * torch.log1p(torch.exp(s["decay"].double()))
    open_r, open_g = 1 / (1 + torch.exp(-r)), 1 / (1 + torch.exp(-g))
    a = torch.exp(-speed * open_r)
    beta = torch.sqrt(1 - a * a)
    b = beta * open_g * x
    if case["pass"] == "step":
        h = a * s["state"].double() + b
        return {"h": h, "state": h}
    if s["longest"] > 70_000:  # over 20 seconds, token by token
        return None
    offsets = s["offsets"].long().cpu().numpy()
    lengths = np.diff(offsets)
    order = np.argsort(-lengths, kind="stable")
    start = torch.from_numpy(offsets[:-1][order]).cuda()
    active = [int(v) for v in (lengths[None, :] > np.arange(s["longest"])[:, None]).sum(1)] if s["longest"] * len(lengths) < 5e7 \
        else [int((lengths > t).sum()) for t in range(s["longest"])]
    order = torch.from_numpy(order).cuda()
    S = case["sequences"]
    carry = s["h0"].double()[order] if s["h0"] is not None else torch.zeros(S, C, dtype=torch.float64, device="cuda")
    h, before = torch.zeros_like(b), torch.zeros_like(b)
    for t, k in enumerate(active):
        rows = start[:k] + t
        before[rows] = carry[:k]
        carry[:k] = a[rows] * carry[:k] + b[rows]
        h[rows] = carry[:k]
    h_last = torch.zeros_like(carry)
    h_last[order] = carry
    if case["pass"] == "forward":
        return {"h": h, "h_last": h_last}
    G = torch.zeros_like(h)
    carry = s["dh_last"].double()[order]
    dh = s["dh"].double()
    for t, k in reversed(list(enumerate(active))):
        rows = start[:k] + t
        total = dh[rows] + carry[:k]
        G[rows] = total
        carry[:k] = a[rows] * total
    da = G * before - G * open_g * x * a / beta  # d loss / d a
    dspeed = -a * da * open_r
    dr = -a * da * speed * open_r * (1 - open_r)
    dproj = torch.cat([G * beta * open_g, dr, G * beta * x * open_g * (1 - open_g)], dim=1)
    ddecay = SHARPNESS * dspeed.sum(0) / (1 + torch.exp(-s["decay"].double()))
    out = {"h": h, "h_last": h_last, "dproj": dproj, "ddecay": ddecay}
    if s["h0"] is not None:
        dh0 = torch.zeros_like(carry)
        dh0[order] = carry
        out["dh0"] = dh0
    return out


def _exact_preference(s):
    case, P = s["case"], s["case"]["pairs"]
    lse = torch.cat([torch.logsumexp(c.double(), 1) for c in s["logits"].split(512)])
    labels, offsets = s["labels"].cpu().numpy(), s["offsets"].cpu().numpy()
    rows = np.flatnonzero(labels >= 0)
    lp = np.zeros(case["tokens"])
    at = torch.from_numpy(rows).cuda(), torch.from_numpy(labels[rows]).cuda()
    lp[rows] = (s["logits"][at].double() - lse[at[0]]).cpu().numpy()
    logps = np.array([lp[offsets[k]:offsets[k + 1]].sum() for k in range(2 * P)])
    ratio = logps - s["ref_logps"].double().cpu().numpy()
    d = PREF["beta"] * (ratio[:P] - ratio[P:])
    eps = PREF["label_smoothing"]
    loss = np.mean((1 - eps) * np.logaddexp(0, -d) + eps * np.logaddexp(0, d))
    out = {"loss": torch.tensor(loss, dtype=torch.float64), "seq_logps": logps}
    if case["grad"]:
        slope = PREF["beta"] / P * (eps / (1 + np.exp(-d)) - (1 - eps) / (1 + np.exp(d)))
        c = np.repeat(np.concatenate([slope, -slope]), np.diff(offsets)) * (labels >= 0)
        c = torch.from_numpy(c).cuda()
        grads = []
        for k, chunk in enumerate(s["logits"].split(512)):
            part = c[512 * k:512 * k + chunk.shape[0]]
            y = s["labels"][512 * k:512 * k + chunk.shape[0]].clamp(min=0)
            grad = -part[:, None] * torch.exp(chunk.double() - lse[512 * k:512 * k + chunk.shape[0], None])
            grad[torch.arange(len(y), device="cuda"), y] += part
            grads.append(grad)
        out["dlogits"] = torch.cat(grads)
    return out
