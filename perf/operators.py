"""The operators at the two ends of the model, as measured: token embedding, the
norm in front of the head and the vocabulary loss, each with its gradients.

``listed()`` names the measured cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes the inputs a program has in hand, ``run()`` is one pass: the
plain form in elementary torch operations, or, with ``own`` set, the calls a
user makes of the library.  ``exact()`` is the same result from the definition
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


def listed():
    return [
        # decoding: the embedding row of one new token
        {"name": "embed_one", "op": "embed", "n": 1, "v": 131072, "d": 2048, "dtype": "bf16", "pad": 0.0},
        # a whole long input (128 segments of 1024 tokens) turned into embeddings, some positions padding
        {"name": "embed_long", "op": "embed", "n": 131072, "v": 131072, "d": 2048, "dtype": "bf16", "pad": 0.05},
        # table gradient of a small fp32 model's batch: odd sizes, latency counts
        {"name": "embed_grad_small", "op": "embed_grad", "n": 67, "v": 515, "d": 64, "dtype": "fp32", "pad": 0.1,
         "accumulate": False},
        # table gradient of a long input, a few frequent tokens among many rare ones
        {"name": "embed_grad_long", "op": "embed_grad", "n": 131072, "v": 131072, "d": 2048, "dtype": "bf16",
         "pad": 0.05, "accumulate": False},
        # tied table: the gradient is added to the one the head has left there
        {"name": "embed_grad_tied", "op": "embed_grad", "n": 8192, "v": 50021, "d": 1024, "dtype": "bf16", "pad": 0.0,
         "accumulate": True},
        # norm of one segment in front of the head
        {"name": "norm_segment", "op": "norm", "n": 1024, "d": 2048, "dtype": "bf16"},
        # training through the norm, forward and gradients, many rows
        {"name": "norm_train", "op": "norm_train", "n": 32771, "d": 2048, "dtype": "bf16"},
        # score of one token against the whole vocabulary: the head is read once
        {"name": "loss_one", "op": "loss", "n": 1, "v": 131072, "d": 2048, "dtype": "bf16", "ignored": 0.0},
        # scores of one segment's tokens
        {"name": "loss_segment", "op": "loss", "n": 1024, "v": 131072, "d": 2048, "dtype": "bf16", "ignored": 0.0},
        # training step of an fp32 model, odd sizes
        {"name": "loss_train_fp32", "op": "loss_train", "n": 515, "v": 10007, "d": 256, "dtype": "fp32",
         "ignored": 0.25, "weights": True},
        # training step on few rows: the head's gradient is most of the traffic
        {"name": "loss_train_few", "op": "loss_train", "n": 131, "v": 50021, "d": 2048, "dtype": "bf16",
         "ignored": 0.0, "weights": False},
        # training step of a long input, positions without a target among them
        {"name": "loss_train_long", "op": "loss_train", "n": 8192, "v": 131072, "d": 2048, "dtype": "bf16",
         "ignored": 0.1, "weights": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_train", "loss", "loss_train", "loss_train"])
    dtype = rng.choice(["bf16", "bf16", "fp32"])
    d = 8 * _log(rng, 8, 512)
    c = {"op": op, "d": d, "dtype": dtype}
    if op in ("norm", "norm_train"):
        c["n"] = _log(rng, 1, 32771 * 2048 // d if d > 2048 else 32771)
        return c
    c["v"] = _log(rng, 300, 131072)
    if op == "embed" or op == "embed_grad":
        if c["v"] * d > 131072 * 2048:
            c["v"] = 131072 * 2048 // d
        c["n"] = _log(rng, 1, min(131072, 131072 * 2048 // d))
        c["pad"] = rng.choice([0.0, 0.05, 0.3])
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.4
        return c
    most = 8192 if dtype == "bf16" else 2048
    if c["v"] * d > 131072 * 2048:
        c["v"] = 131072 * 2048 // d
    c["n"] = _log(rng, 1, most)
    c["ignored"] = rng.choice([0.0, 0.1, 0.5])
    if op == "loss_train":
        c["weights"] = rng.random() < 0.5
    return c


def _inputs(case, seed):
    """The tensors of one case, from the seed alone."""
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 2 + 1)
    t = TYPES[case["dtype"]]
    op, n, d = case["op"], case["n"], case["d"]
    rand = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    randn = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x = {}
    if op in ("embed", "embed_grad"):
        v = case["v"]
        ids = (v * rand(n).double() ** 4).long().clamp_(max=v - 1)   # few frequent tokens, many rare ones
        ids[rand(n) < case["pad"]] = -1                              # padding positions
        x["ids"] = ids
        x["scale"] = float(math.sqrt(d))
        if op == "embed":
            x["table"] = (randn(v, d) * 0.02).to(t)
        else:
            x["d_out"] = (randn(n, d) * 1e-2).to(t)
            x["base"] = (randn(v, d) * 1e-2).to(t) if case["accumulate"] else None
    elif op in ("norm", "norm_train"):
        x["x"] = (randn(n, d) * (0.5 + 4 * rand(n, 1))).to(t)
        x["gain"] = (1 + 0.1 * randn(d)).to(t)
        if op == "norm_train":
            x["dy"] = (randn(n, d) * 1e-2).to(t)
    else:
        v = case["v"]
        w = (randn(v, d) / math.sqrt(d)).to(t)
        tg = torch.randint(0, v, (n,), generator=g, device=DEV)
        # hidden states that lean towards their target by up to 14: from a flat to a sure prediction
        x["hidden"] = (randn(n, d) + 14 * rand(n, 1) * w[tg].float()).to(t)
        tg[rand(n) < case["ignored"]] = -100
        x["head"], x["targets"] = w, tg
        if op == "loss_train":
            gl = 0.5 + rand(n) if case["weights"] else torch.ones(n, device=DEV)
            x["d_loss"] = gl / n
    return x


def prepare(case, seed):
    x = _inputs(case, seed)
    x["op"], x["dtype"] = case["op"], TYPES[case["dtype"]]
    if case["op"] == "embed_grad":
        x["v"] = case["v"]
    return x


def _row_scale(x):
    return torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)


def _plain(s):
    op, t = s["op"], s["dtype"]
    if op == "embed":
        ids, table = s["ids"], s["table"]
        ok = (ids >= 0) & (ids < table.shape[0])
        rows = table[ids.clamp(0, table.shape[0] - 1)].float() * s["scale"]
        return {"out": torch.where(ok[:, None], rows, 0.0).to(t)}
    if op == "embed_grad":
        ids, v = s["ids"], s["v"]
        ok = (ids >= 0) & (ids < v)
        rows = torch.where(ok[:, None], s["d_out"].float() * s["scale"], 0.0)
        acc = torch.zeros(v, rows.shape[1], device=DEV)
        acc.index_add_(0, ids.clamp(0, v - 1), rows)
        if s["base"] is not None:
            acc += s["base"].float()
        return {"d_table": acc.to(t)}
    if op in ("norm", "norm_train"):
        x, gain = s["x"].float(), s["gain"].float()
        r = _row_scale(x)
        y = (x * r * gain).to(t)
        if op == "norm":
            return {"y": y}
        dy = s["dy"].float()
        u = dy * gain
        dx = r * (u - x * r * r * (u * x).mean(1, keepdim=True))
        return {"y": y, "dx": dx.to(t), "d_gain": (dy * x * r).sum(0).to(t)}
    hidden, head, tg = s["hidden"].float(), s["head"].float(), s["targets"]
    v = head.shape[0]
    ok = (tg >= 0) & (tg < v)
    at = tg.clamp(0, v - 1)[:, None]
    logits = hidden @ head.t()
    m = logits.max(1, keepdim=True).values
    lse = m + torch.log(torch.exp(logits - m).sum(1, keepdim=True))
    loss = torch.where(ok, (lse - logits.gather(1, at))[:, 0], 0.0)
    out = {"loss": loss, "lse": torch.where(ok, lse[:, 0], 0.0)}
    if op == "loss":
        return out
    gl = torch.where(ok, s["d_loss"], 0.0)[:, None]
    p = torch.exp(logits - lse) * gl
    p.scatter_add_(1, at, -gl)
    return {**out, "d_hidden": (p @ head).to(t), "d_head": (p.t() @ hidden).to(t)}


def _own(s):
    import recurrent_memory_transformer_diag_b200 as armt
    op, t = s["op"], s["dtype"]
    if op == "embed":
        out = torch.empty(s["ids"].shape[0], s["table"].shape[1], dtype=t, device=DEV)
        armt.embed(s["ids"], s["table"], out, scale=s["scale"])
        return {"out": out}
    if op == "embed_grad":
        # the tied gradient is added to in place by a user; the copy keeps the inputs for the next pass
        d_table = torch.empty(s["v"], s["d_out"].shape[1], dtype=t, device=DEV) if s["base"] is None else s["base"].clone()
        armt.embed_grad(s["ids"], s["d_out"], d_table, scale=s["scale"], accumulate=s["base"] is not None)
        return {"d_table": d_table}
    if op in ("norm", "norm_train"):
        x = s["x"]
        y, rstd = torch.empty_like(x), torch.empty(x.shape[0], device=DEV)
        armt.rms_norm(x, s["gain"], y, rstd, EPS)
        if op == "norm":
            return {"y": y}
        dx, d_gain = torch.empty_like(x), torch.empty_like(s["gain"])
        armt.rms_norm_grad(x, s["gain"], rstd, s["dy"], dx, d_gain)
        return {"y": y, "dx": dx, "d_gain": d_gain}
    hidden, head, tg = s["hidden"], s["head"], s["targets"]
    loss = torch.empty(hidden.shape[0], device=DEV)
    lse = torch.empty(hidden.shape[0], device=DEV)
    armt.token_loss(hidden, head, tg, loss, lse)
    if op == "loss":
        return {"loss": loss, "lse": lse}
    d_hidden, d_head = torch.empty_like(hidden), torch.empty_like(head)
    armt.token_loss_grad(hidden, head, tg, lse, s["d_loss"], d_hidden, d_head)
    return {"loss": loss, "lse": lse, "d_hidden": d_hidden, "d_head": d_head}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """Inputs read once, outputs written once, the products of the definition (the
    logits once more for the gradient are not counted); rows without a target need none."""
    s = 2 if case["dtype"] == "bf16" else 4
    op, n, d = case["op"], case["n"], case["d"]
    if op == "embed":
        return {"bytes": n * d * s * (2 - case["pad"]) + 8 * n, "flops": n * d}
    if op == "embed_grad":
        rows = n * (1 - case["pad"])
        table = 3 * min(rows, case["v"]) if case["accumulate"] else case["v"]
        return {"bytes": (rows + table) * d * s + 8 * n, "flops": 2 * n * d}
    if op == "norm":
        return {"bytes": 2 * n * d * s + d * s, "flops": 5 * n * d}
    if op == "norm_train":
        return {"bytes": 4 * n * d * s + 2 * d * s, "flops": 16 * n * d}
    rows = max(1.0, n * (1 - case["ignored"]))
    once = (rows + case["v"]) * d * s + 16 * n
    product = 2.0 * rows * case["v"] * d
    return {"bytes": once, "flops": product} if op == "loss" else {"bytes": 2 * once, "flops": 3 * product}


def exact(case, seed):
    x = _inputs(case, seed)
    op = case["op"]
    if op == "embed":
        t = torch.cat([x["table"].double(), torch.zeros(1, case["d"], device=DEV, dtype=torch.float64)])
        return {"out": t[torch.where(x["ids"] < 0, case["v"], x["ids"])] * x["scale"]}
    if op == "embed_grad":
        order = torch.argsort(x["ids"], stable=True)
        ids = x["ids"][order]
        order, ids = order[ids >= 0], ids[ids >= 0]
        out = torch.zeros(case["v"], case["d"], device=DEV, dtype=torch.float64)
        if x["base"] is not None:
            out += x["base"].double()
        out.index_put_((ids,), x["d_out"][order].double() * x["scale"], accumulate=True)
        return {"d_table": out}
    if op in ("norm", "norm_train"):
        v, g = x["x"].double(), x["gain"].double()
        n = (v.square().sum(1) / case["d"] + EPS).sqrt()[:, None]
        h = v / n
        if op == "norm":
            return {"y": h * g}
        dy = x["dy"].double()
        dh = dy * g
        return {"y": h * g, "dx": (dh - h * ((dh * h).sum(1, keepdim=True) / case["d"])) / n, "d_gain": (dy * h).sum(0)}
    w, keep = x["head"].double(), x["targets"] >= 0
    n, v, d = case["n"], case["v"], case["d"]
    loss = torch.zeros(n, device=DEV, dtype=torch.float64)
    lse = torch.zeros_like(loss)
    train = op == "loss_train"
    dh = torch.zeros(n, d, device=DEV, dtype=torch.float64) if train else None
    dw = torch.zeros(v, d, device=DEV, dtype=torch.float64) if train else None
    rows = keep.nonzero()[:, 0]
    for part in rows.split(2048):
        h, t = x["hidden"][part].double(), x["targets"][part]
        logits = h @ w.t()
        lp = torch.log_softmax(logits, 1)
        loss[part] = -lp[torch.arange(len(part), device=DEV), t]
        lse[part] = torch.logsumexp(logits, 1)
        if train:
            q = lp.exp_()
            q[torch.arange(len(part), device=DEV), t] -= 1.0
            q *= x["d_loss"][part].double()[:, None]
            dh[part] = q @ w
            dw += q.t() @ h
    return {"loss": loss, "lse": lse, "d_hidden": dh, "d_head": dw} if train else {"loss": loss, "lse": lse}
