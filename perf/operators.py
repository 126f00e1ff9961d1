"""Cases of the vocabulary operators: what the two ends of a language model do
with a vocab-parallel [V, K] matrix (TP shards of W rows each).

  embed       out[n] = scale * table[tokens[n]]
  embed_grad  grad_table[v] (+)= scale * sum of grad_out[n] over tokens[n] = v
  loss        softmax cross entropy of logit_scale * hidden @ weight.T against
              the targets, per row, with the row's logsumexp
  loss_grad   its gradient to hidden and weight, from that logsumexp and the
              upstream gradient of each row's loss

A token outside the vocabulary is padding: a row of zeros, and no gradient. A
negative target masks its row: loss, logsumexp and gradient are 0. Columns from
`vocab` on (a vocabulary padded to the shards) are no part of the softmax.

``own`` False computes these in plain 32-bit torch operations; ``own`` True
through tp_vocab_logits_gb300.hg.
"""

import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# The sharded vocabulary of this repository's decode workload and its fused LM
# head: TP8, V = 163840, K = 7168.
FULL = {"tp": 8, "cols": 20480, "vocab": 163840, "hidden": 7168}
# The largest work a case may have (flops of the matrix products).
MOST_FLOPS = 6 * 4096 * 163840 * 7168


def listed():
    return [
        # One drafted token scored against the whole vocabulary: the weights are
        # read once, latency and bandwidth count.
        {"name": "loss, 1 row", "op": "loss", **FULL, "rows": 1, "dtype": "bf16", "masked": 0.0},
        # A small vocabulary and an odd number of rows, short of a tile each way.
        {"name": "loss, 333 rows, odd", "op": "loss", "tp": 1, "cols": 49999, "vocab": 49999,
         "hidden": 1000, "rows": 333, "dtype": "fp16", "masked": 0.1},
        # Fine-tuning: the prompt's tokens, two fifths of the rows, are masked.
        {"name": "loss, 2500 rows, 2/5 masked", "op": "loss", "tp": 4, "cols": 8192,
         "vocab": 32765, "hidden": 2048, "rows": 2500, "dtype": "bf16", "masked": 0.4},
        # A training micro-batch against the whole vocabulary.
        {"name": "loss, 8192 rows", "op": "loss", **FULL, "rows": 8192, "dtype": "bf16",
         "masked": 0.0},
        # The gradient of a few rows (a preference or distillation step on
        # single tokens): reading and writing a [V, K] matrix bounds it.
        {"name": "loss_grad, 16 rows", "op": "loss_grad", **FULL, "rows": 16, "dtype": "bf16",
         "masked": 0.0},
        {"name": "loss_grad, 1000 rows, odd", "op": "loss_grad", "tp": 2, "cols": 25001,
         "vocab": 49999, "hidden": 1544, "rows": 1000, "dtype": "fp16", "masked": 0.4},
        # The gradient of a training micro-batch against the whole vocabulary.
        {"name": "loss_grad, 4096 rows", "op": "loss_grad", **FULL, "rows": 4096,
         "dtype": "bf16", "masked": 0.0},
        # The next decode step's embedding: latency.
        {"name": "embed, 1 row", "op": "embed", **FULL, "rows": 1, "dtype": "bf16",
         "masked": 0.0},
        # A long prefill or a training batch.
        {"name": "embed, 32768 rows", "op": "embed", **FULL, "rows": 32768, "dtype": "bf16",
         "masked": 0.05},
        # A small table kept in 32 bits, odd width, gradient written whole.
        {"name": "embed_grad, 3001 rows, odd", "op": "embed_grad", "tp": 2, "cols": 16001,
         "vocab": 32001, "hidden": 1001, "rows": 3001, "dtype": "fp32", "masked": 0.1,
         "accumulate": False},
        # Tied weights: the embedding's gradient is added to what the loss left
        # in the same matrix.
        {"name": "embed_grad, 8192 rows, tied", "op": "embed_grad", **FULL, "rows": 8192,
         "dtype": "bf16", "masked": 0.0, "accumulate": True},
        # An untied table: every row of the gradient is written.
        {"name": "embed_grad, 16384 rows", "op": "embed_grad", **FULL, "rows": 16384,
         "dtype": "bf16", "masked": 0.05, "accumulate": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case: any operator, any type it takes, rows from one to the
    listed most, widths and vocabularies up to the listed ones."""
    while True:
        op = rng.choice(["loss", "loss_grad", "embed", "embed_grad"])
        c = {"op": op, "tp": rng.choice([1, 2, 3, 4, 8, 16])}
        c["cols"] = _log_int(rng, 500, 20480)
        total = c["tp"] * c["cols"]
        c["vocab"] = total - rng.choice([0, 0, rng.randint(0, c["cols"] // 8)])
        if op.startswith("loss"):
            c["hidden"] = 8 * _log_int(rng, 8, 896)
            c["rows"] = _log_int(rng, 1, 8192)
            c["dtype"] = rng.choice(["bf16", "bf16", "fp16"])
            flops = (2 if op == "loss" else 6) * c["rows"] * total * c["hidden"]
            if flops > MOST_FLOPS:
                continue
        else:
            c["hidden"] = _log_int(rng, 64, 7168)
            c["rows"] = _log_int(rng, 1, 32768)
            c["dtype"] = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        c["masked"] = rng.choice([0.0, 0.05, 0.5])
        if op == "embed_grad":
            c["accumulate"] = rng.random() < 0.5
        if 3072 not in (c["cols"], c["vocab"], c["hidden"], c["rows"], total):
            return c


def _frequencies(vocab):
    """Token frequencies of text, roughly: falling as 1 / (rank + 10)."""
    p = 1.0 / (np.arange(vocab) + 10.0)
    return p / p.sum()


def _expected_rows(c):
    """Rows of the table that the tokens touch, on average."""
    n = c["rows"] * (1.0 - c["masked"])
    return float(np.sum(-np.expm1(n * np.log1p(-_frequencies(c["vocab"])))))


def _tokens(c, gen):
    """Token ids with text's frequencies over an order of its own, the masked
    share of them negative."""
    p = torch.from_numpy(_frequencies(c["vocab"])).to(gen.device, torch.float64)
    u = torch.rand(c["rows"], generator=gen, device=gen.device, dtype=torch.float64)
    rank = torch.searchsorted(torch.cumsum(p, 0), u).clamp_(max=c["vocab"] - 1)
    order = torch.randperm(c["vocab"], generator=gen, device=gen.device)
    ids = order[rank]
    hide = torch.rand(c["rows"], generator=gen, device=gen.device) < c["masked"]
    return torch.where(hide, -100, ids)


def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32) \
        .mul_(std).to(dtype)


def _scale(c):
    """An embedding scaled by sqrt(K), as models with tied weights do; logits
    divided by a temperature of 1.25."""
    return math.sqrt(c["hidden"]) if c["op"].startswith("embed") else 0.8


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = TYPES[c["dtype"]]
    total, K, n = c["tp"] * c["cols"], c["hidden"], c["rows"]
    s = {"case": c, "tokens": _tokens(c, gen)}
    if c["op"] == "embed_grad":
        s["grad_out"] = _normal(gen, (n, K), 1e-3, dtype)
        s["matrix"] = _normal(gen, (total, K), 1e-3, dtype) if c["accumulate"] else \
            torch.empty((total, K), device="cuda", dtype=dtype)
    else:
        s["matrix"] = _normal(gen, (total, K), 0.02, dtype)
    if c["op"] == "embed":
        s["out"] = torch.empty((n, K), device="cuda", dtype=dtype)
    if c["op"].startswith("loss"):
        s["hidden"] = _normal(gen, (n, K), 1.0, dtype)
        s["loss"] = torch.empty(n, device="cuda")
        s["lse"] = torch.empty(n, device="cuda")
    if c["op"] == "loss_grad":
        # In hand from the forward pass: each row's logsumexp, and the upstream
        # gradient of a weighted mean, scaled up where gradients are kept in fp16.
        s["lse"] = _plain_loss(s)[1]
        weight = torch.rand(n, generator=gen, device="cuda") + 0.5
        up = 1024.0 if dtype == torch.float16 else 1.0
        s["grad_loss"] = weight * (up / max(1.0, n * (1.0 - c["masked"])))
        s["grad_hidden"] = torch.empty_like(s["hidden"])
        s["grad_matrix"] = torch.empty_like(s["matrix"])
    s["shards"] = list(s["matrix"].split(c["cols"]))
    if c["op"] == "loss_grad":
        s["grad_shards"] = list(s["grad_matrix"].split(c["cols"]))
    if own:
        from tp_vocab_logits_gb300 import hg
        s["handle"] = hg.hg_vocab_create(c["tp"], c["cols"], K, n, vocab=c["vocab"], dtype=dtype,
                                         ops=(c["op"],))
    return s


def _plain_logits(s):
    c = s["case"]
    logits = s["hidden"].float() @ s["matrix"].float().t()
    logits *= _scale(c)
    logits[:, c["vocab"]:] = -math.inf
    return logits


def _plain_loss(s):
    t = s["tokens"]
    logits = _plain_logits(s)
    at = logits.gather(1, t.clamp(min=0)[:, None])[:, 0]
    top = logits.amax(1)
    lse = top + logits.sub_(top[:, None]).exp_().sum(1).log()
    return torch.where(t < 0, 0.0, lse - at), torch.where(t < 0, 0.0, lse)


def _plain_loss_grad(s):
    c, t = s["case"], s["tokens"]
    d = _plain_logits(s).sub_(s["lse"][:, None]).exp_()
    d.scatter_add_(1, t.clamp(min=0)[:, None], torch.full_like(d[:, :1], -1.0))
    d *= (torch.where(t < 0, 0.0, s["grad_loss"]) * _scale(c))[:, None]
    grad_hidden = d @ s["matrix"].float()
    grad_matrix = d.t() @ s["hidden"].float()
    return grad_hidden.to(s["hidden"].dtype), grad_matrix.to(s["matrix"].dtype)


def _inside(s):
    return (s["tokens"] >= 0)[:, None]


def _plain_embed(s):
    rows = s["matrix"][s["tokens"].clamp(min=0)].float() * _scale(s["case"])
    return torch.where(_inside(s), rows, 0.0).to(s["matrix"].dtype)


def _plain_embed_grad(s):
    m = s["matrix"]
    rows = torch.where(_inside(s), s["grad_out"].float(), 0.0) * _scale(s["case"])
    total = m.float() if s["case"]["accumulate"] else torch.zeros(m.shape, device=m.device)
    if total.data_ptr() == m.data_ptr():
        total = total.clone()
    total.index_add_(0, s["tokens"].clamp(min=0), rows)
    return m.copy_(total)


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "loss":
            loss, lse = _plain_loss(s)
            return {"loss": loss, "lse": lse}
        if op == "loss_grad":
            grad_hidden, grad_weight = _plain_loss_grad(s)
            return {"grad_hidden": grad_hidden, "grad_weight": grad_weight}
        return {"out": _plain_embed(s)} if op == "embed" else {"grad_table": _plain_embed_grad(s)}
    from tp_vocab_logits_gb300 import hg
    h = s["handle"]
    if op == "loss":
        hg.hg_vocab_loss(h, s["hidden"], s["shards"], s["tokens"], s["loss"], s["lse"],
                         logit_scale=_scale(c))
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "loss_grad":
        hg.hg_vocab_loss_grad(h, s["hidden"], s["shards"], s["tokens"], s["lse"], s["grad_loss"],
                              s["grad_hidden"], s["grad_shards"], logit_scale=_scale(c))
        return {"grad_hidden": s["grad_hidden"], "grad_weight": s["grad_matrix"]}
    if op == "embed":
        hg.hg_vocab_embed(h, s["tokens"], s["shards"], s["out"], scale=_scale(c))
        return {"out": s["out"]}
    hg.hg_vocab_embed_grad(h, s["tokens"], s["grad_out"], s["shards"], scale=_scale(c),
                           accumulate=c["accumulate"])
    return {"grad_table": s["matrix"]}


def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    n, K, total = c["rows"], c["hidden"], c["tp"] * c["cols"]
    valid = max(1.0, n * (1.0 - c["masked"]))
    if c["op"] == "loss":
        # The weights and the unmasked rows once; targets, losses, logsumexps.
        return {"bytes": e * K * (c["vocab"] + valid) + 16 * n,
                "flops": 2.0 * valid * c["vocab"] * K}
    if c["op"] == "loss_grad":
        # The weights and the unmasked rows in, both gradients out; the logits
        # again, and a product of their gradient with each side.
        return {"bytes": e * K * (c["vocab"] + total + valid + n) + 16 * n,
                "flops": 6.0 * valid * c["vocab"] * K}
    if c["op"] == "embed":
        return {"bytes": e * K * (_expected_rows(c) + n) + 8 * n, "flops": 1.0 * valid * K}
    out = 2 * _expected_rows(c) if c["accumulate"] else total
    return {"bytes": e * K * (out + valid) + 8 * n, "flops": 2.0 * valid * K}


def exact(case, seed):
    c = case
    e = {"loss": 2.0, "loss_grad": 6.0}.get(c["op"], 0.0)
    if e * c["rows"] * c["tp"] * c["cols"] * c["hidden"] > 1.2e13:
        return None
    s = prepare(case, seed)
    ids, valid, f = s["tokens"], s["tokens"] >= 0, _scale(c)
    M = s["matrix"].double()
    if c["op"] == "embed":
        out = torch.zeros((c["rows"], c["hidden"]), dtype=torch.float64, device="cuda")
        out[valid] = M[ids[valid]] * f
        return {"out": out}
    if c["op"] == "embed_grad":
        add = torch.zeros_like(M)
        add.index_add_(0, ids[valid], s["grad_out"][valid].double())
        return {"grad_table": M + f * add if c["accumulate"] else f * add}
    X = s["hidden"][valid].double()
    real = M[:c["vocab"]]
    z = X @ real.t() * f
    rows = torch.arange(X.shape[0], device="cuda")
    if c["op"] == "loss":
        loss = torch.zeros(c["rows"], dtype=torch.float64, device="cuda")
        lse = torch.zeros_like(loss)
        lse[valid] = torch.logsumexp(z, 1)
        loss[valid] = lse[valid] - z[rows, ids[valid]]
        return {"loss": loss, "lse": lse}
    p = torch.exp(z - s["lse"][valid].double()[:, None])
    p[rows, ids[valid]] -= 1.0
    p *= f * s["grad_loss"][valid].double()[:, None]
    grad_hidden = torch.zeros((c["rows"], c["hidden"]), dtype=torch.float64, device="cuda")
    grad_weight = torch.zeros_like(M)
    grad_hidden[valid] = p @ real
    grad_weight[:c["vocab"]] = p.t() @ X
    return {"grad_hidden": grad_hidden, "grad_weight": grad_weight}
