"""Cases of the operators beside the vocabulary's: the norm in front of the LM
head with its gradient, and a beam search's step behind it.

  norm          s = x + residual, held in the matrix's type; out = s * rstd * gain
                with rstd = 1 / sqrt(mean of s^2 + eps) per row. In 8 bits (e4m3)
                out is divided by scales: the largest magnitude of a row, or of
                each 128 columns of it, over 448
  norm_grad     with d = gain * grad_out: grad_x = rstd * d - s * rstd^3 * mean of
                d * s + grad_sum; grad_gain (+)= sum over rows of grad_out * s * rstd
  beam_select   total = score[beam] + logit - logsumexp of the beam's logits; the
                `picks` largest totals over an item's beams and vocabulary, with
                their beams and tokens. Equal totals: the lower beam, then the
                lower token. A finished beam goes on as it is, with the end token
  beam_reorder  row j of an item's states takes what the row parents[j] holds

A pick that no candidate is left for has token and parent -1 and total -inf; a
parent outside the item's beams leaves its row as it is. `own` False computes
these in plain torch operations, in 32 bits (the totals in 64, where candidates
next to each other are told apart); `own` True through tp_vocab_logits_gb300.hg.
"""

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
E4M3_MOST = 448.0  # largest e4m3 value
BLOCK = 128        # columns that share a scale where a row has several

# The width and the vocabulary of this repository's decode workload and its fused
# LM head.
WIDTH, VOCAB = 7168, 163840


def listed():
    return [
        # The next token of one sequence: latency counts.
        {"name": "norm, 1 row", "op": "norm", "rows": 1, "hidden": WIDTH, "dtype": "bf16",
         "residual": True, "quant": ""},
        # A narrow model of odd width, where rows start at any multiple of two bytes.
        {"name": "norm, 333 rows, odd", "op": "norm", "rows": 333, "hidden": 1001,
         "dtype": "fp16", "residual": False, "quant": ""},
        # A prefill whose next product is in 8 bits, a scale per 128 columns.
        {"name": "norm, 2048 rows, 8 bits", "op": "norm", "rows": 2048, "hidden": WIDTH,
         "dtype": "bf16", "residual": True, "quant": "block"},
        # A training micro-batch in front of the loss.
        {"name": "norm, 8192 rows", "op": "norm", "rows": 8192, "hidden": WIDTH, "dtype": "bf16",
         "residual": True, "quant": ""},
        # The gradient of a few scored tokens.
        {"name": "norm_grad, 16 rows", "op": "norm_grad", "rows": 16, "hidden": WIDTH,
         "dtype": "bf16", "residual": True, "accumulate": False},
        # An odd width kept in 32 bits, added to an earlier micro-batch's gradient.
        {"name": "norm_grad, 1000 rows, odd", "op": "norm_grad", "rows": 1000, "hidden": 1001,
         "dtype": "fp32", "residual": False, "accumulate": True},
        # The gradient of a training micro-batch, with what the residual stream brings.
        {"name": "norm_grad, 4096 rows", "op": "norm_grad", "rows": 4096, "hidden": WIDTH,
         "dtype": "bf16", "residual": True, "accumulate": False},
        # One request with four beams, its logsumexp from the gather's statistics,
        # twice as many picks as beams so that those that end can be set aside.
        {"name": "beam_select, 4 beams", "op": "beam_select", "items": 1, "beams": 4, "picks": 8,
         "vocab": VOCAB, "pad": 0, "dtype": "bf16", "stats": True, "finished": 0.0, "dead": 0.0,
         "banned": 0.0},
        # A small odd vocabulary in 16 bits, beams that have finished, and
        # most tokens ruled out by a grammar.
        {"name": "beam_select, 7 x 5 beams, odd", "op": "beam_select", "items": 7, "beams": 5,
         "picks": 5, "vocab": 49999, "pad": 1, "dtype": "fp16", "stats": False, "finished": 0.2,
         "dead": 0.1, "banned": 0.9},
        # A full batch: the logits of 256 rows.
        {"name": "beam_select, 32 x 8 beams", "op": "beam_select", "items": 32, "beams": 8,
         "picks": 16, "vocab": VOCAB, "pad": 0, "dtype": "bf16", "stats": False, "finished": 0.0,
         "dead": 0.0, "banned": 0.0},
        # One request's token history and small caches, just begun.
        {"name": "beam_reorder, 4 beams", "op": "beam_reorder", "items": 1, "beams": 4,
         "layers": 2, "heads": 2, "held": 64, "used": 17, "width": 64, "dtype": "bf16",
         "rows_first": False, "dead": 0.0},
        # A full batch's caches, nearly filled.
        {"name": "beam_reorder, 32 x 8 beams", "op": "beam_reorder", "items": 32, "beams": 8,
         "layers": 4, "heads": 8, "held": 512, "used": 500, "width": 64, "dtype": "bf16",
         "rows_first": False, "dead": 0.0},
    ]


# The most logits and cache bytes (of keys, or of values) that a drawn case has.
MOST_LOGITS = 32 * 8 * VOCAB
MOST_CACHE = 4 * 256 * 8 * 512 * 64 * 2


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    """One more case: any operator, any type it takes, from one row, beam or
    position to the listed most."""
    while True:
        op = rng.choice(["norm", "norm_grad", "beam_select", "beam_reorder"])
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"])}
        if op.startswith("norm"):
            c["rows"] = _log_int(rng, 1, 8192 if op == "norm" else 4096)
            c["hidden"] = rng.choice([8 * _log_int(rng, 8, WIDTH // 8), _log_int(rng, 50, WIDTH)])
            c["residual"] = rng.random() < 0.7
            if op == "norm":
                c["quant"] = rng.choice(["", "", "row", "block"])
            else:
                c["accumulate"] = rng.random() < 0.5
            return c
        c["items"] = _log_int(rng, 1, 32)
        c["beams"] = _log_int(rng, 1, 32)
        c["dead"] = rng.choice([0.0, 0.0, 0.2])
        if op == "beam_select":
            c["picks"] = c["beams"] * rng.choice([1, 2])
            c["vocab"] = _log_int(rng, 500, VOCAB)
            c["pad"] = rng.choice([0, 0, rng.randint(1, 64)])
            c["stats"] = rng.random() < 0.6
            c["finished"] = rng.choice([0.0, 0.0, 0.3])
            c["banned"] = rng.choice([0.0, 0.0, 0.5, 0.99])
            if c["items"] * c["beams"] * c["vocab"] <= MOST_LOGITS:
                return c
        else:
            c["layers"] = _log_int(rng, 1, 8)
            c["heads"] = _log_int(rng, 1, 8)
            c["held"] = _log_int(rng, 8, 2000)
            c["used"] = rng.randint(1, c["held"])
            c["width"] = rng.choice([32, 64, 128, rng.randint(20, 140)])
            c["rows_first"] = rng.random() < 0.5
            if _cache_bytes(c, c["held"]) <= MOST_CACHE:
                return c


def _cache_bytes(c, length):
    return c["items"] * c["beams"] * c["layers"] * c["heads"] * length * c["width"] \
        * SIZES[c["dtype"]]


def _normal(gen, shape, std, dtype):
    return torch.randn(shape, generator=gen, device=gen.device, dtype=torch.float32) \
        .mul_(std).to(dtype)


def _share(gen, shape, p):
    """True in a share p of the places."""
    return torch.rand(shape, generator=gen, device=gen.device) < p


# ---- inputs ------------------------------------------------------------------------


def _prepare_norm(c, gen):
    dtype, n, K = TYPES[c["dtype"]], c["rows"], c["hidden"]
    s = {"gain": _normal(gen, (K,), 0.1, torch.float32).add_(1.0).to(dtype)}
    x = _normal(gen, (n, K), 1.0, dtype)
    # A few columns far larger than the others, as residual streams have.
    x[:, torch.randint(0, K, (3,), generator=gen, device="cuda")] *= 20.0
    if c["op"] == "norm":
        s["x"] = x
        s["residual"] = _normal(gen, (n, K), 2.0, dtype) if c["residual"] else None
        s["sum"] = torch.empty_like(x) if c["residual"] else None
        s["rstd"] = torch.empty(n, device="cuda")
        s["out"] = torch.empty((n, K), device="cuda",
                               dtype=torch.float8_e4m3fn if c["quant"] else dtype)
        s["scales"] = None
        if c["quant"]:
            blocks = -(-K // BLOCK) if c["quant"] == "block" else 1
            s["scales"] = torch.empty((n, blocks), device="cuda")
        return s
    # In hand from the forward pass: the sum and its reciprocal deviation.
    s["sum"] = x
    s["rstd"] = torch.rsqrt(x.float().square().mean(1) + EPS)
    up = 64.0 if dtype == torch.float16 else 1.0
    s["grad_out"] = _normal(gen, (n, K), 1e-2 * up, dtype)
    s["grad_sum"] = _normal(gen, (n, K), 1e-2 * up, dtype) if c["residual"] else None
    s["grad_x"] = torch.empty_like(x)
    s["grad_gain"] = _normal(gen, (K,), 0.1 * up, dtype)
    return s


def _prepare_select(c, gen):
    rows = c["items"] * c["beams"]
    whole = _normal(gen, (rows, c["vocab"] + c["pad"]), 2.5, TYPES[c["dtype"]])
    s = {"logits": whole[:, :c["vocab"]]}
    if c["banned"]:
        # What a grammar rules out, the same for an item's beams.
        ban = _share(gen, (c["items"], c["vocab"]), c["banned"]).repeat_interleave(c["beams"], 0)
        s["logits"].masked_fill_(ban, -math.inf)
    shape = (c["items"], c["beams"])
    s["scores"] = -20.0 * torch.rand(shape, generator=gen, device="cuda") - 5.0
    s["scores"].masked_fill_(_share(gen, shape, c["dead"]), -math.inf)
    s["finished"] = _share(gen, shape, c["finished"]) if c["finished"] else None
    s["end"] = c["vocab"] // 3
    s["lse"] = None
    if c["stats"]:
        # Rows of four values with the logsumexp last, as the gather leaves them.
        stats = torch.zeros((rows, 4), device="cuda")
        stats[:, 3] = torch.logsumexp(s["logits"].double(), 1)
        s["lse"] = stats[:, 3]
    out = (c["items"], c["picks"])
    s["tokens"] = torch.empty(out, device="cuda", dtype=torch.int64)
    s["parents"] = torch.empty(out, device="cuda", dtype=torch.int64)
    s["picked"] = torch.empty(out, device="cuda")
    s["picked_finished"] = torch.empty(out, device="cuda", dtype=torch.bool)
    return s


def _chances(beams):
    """How often each beam is a parent: the better ones more often."""
    p = 0.75 ** torch.arange(beams, dtype=torch.float64)
    return p / p.sum()


def _prepare_reorder(c, gen):
    items, beams = c["items"], c["beams"]
    rows, dtype = items * beams, TYPES[c["dtype"]]
    front = (rows, c["layers"]) if c["rows_first"] else (c["layers"], rows)
    shape = (*front, c["heads"], c["held"], c["width"])
    s = {"keys": _normal(gen, shape, 1.0, dtype), "values": _normal(gen, shape, 1.0, dtype),
         "history": torch.randint(0, VOCAB, (rows, c["held"]), generator=gen, device="cuda")}
    cut = torch.cumsum(_chances(beams), 0).to("cuda")
    u = torch.rand((items, beams), generator=gen, device="cuda", dtype=torch.float64)
    parents = torch.searchsorted(cut, u).clamp_(max=beams - 1)
    s["parents"] = torch.where(_share(gen, (items, beams), c["dead"]), -1, parents)
    # What is filled of each state, and the dimension of its rows.
    dim = 0 if c["rows_first"] else 1
    s["states"] = [(s["keys"][..., :c["used"], :], dim), (s["values"][..., :c["used"], :], dim),
                   (s["history"][:, :c["used"]], 0)]
    return s


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    make = {"norm": _prepare_norm, "norm_grad": _prepare_norm, "beam_select": _prepare_select,
            "beam_reorder": _prepare_reorder}
    s = make[c["op"]](c, gen)
    s["case"] = c
    if own:
        from tp_vocab_logits_gb300 import hg
        if c["op"].startswith("norm"):
            s["handle"] = hg.hg_norm_create(c["hidden"], c["rows"], dtype=TYPES[c["dtype"]])
        else:
            s["handle"] = hg.hg_beam_create(c["items"], c["beams"], c.get("vocab", VOCAB),
                                            c.get("picks", c["beams"]), dtype=TYPES[c["dtype"]])
    return s


# ---- plain forms -------------------------------------------------------------------


def _plain_norm(s):
    c = s["case"]
    out = {}
    total = s["x"]
    if c["residual"]:
        total = (s["x"].float() + s["residual"].float()).to(total.dtype)
        out["sum"] = total
    total = total.float()
    rstd = torch.rsqrt(total.square().mean(1) + EPS)
    y = total * rstd[:, None] * s["gain"].float()
    out["rstd"] = rstd
    if not c["quant"]:
        return out | {"out": y.to(s["x"].dtype)}
    n, K = y.shape
    width = BLOCK if c["quant"] == "block" else K
    blocks = -(-K // width)
    wide = torch.zeros((n, blocks * width), device="cuda")
    wide[:, :K] = y
    wide = wide.view(n, blocks, width)
    scales = wide.abs().amax(2) / E4M3_MOST
    scales = torch.where(scales > 0.0, scales, 1.0)
    q = (wide / scales[..., None]).view(n, -1)[:, :K]
    return out | {"out": q.to(torch.float8_e4m3fn), "scales": scales}


def _plain_norm_grad(s):
    c = s["case"]
    x, r, g = s["sum"].float(), s["rstd"][:, None], s["grad_out"].float()
    d = g * s["gain"].float()
    grad_x = r * d - x * (r * r * r * (d * x).mean(1, keepdim=True))
    if c["residual"]:
        grad_x = grad_x + s["grad_sum"].float()
    grad_gain = (g * x * r).sum(0)
    if c["accumulate"]:
        grad_gain = grad_gain + s["grad_gain"].float()
    s["grad_gain"].copy_(grad_gain)
    return {"grad_x": grad_x.to(s["sum"].dtype), "grad_gain": s["grad_gain"]}


def _plain_select(s):
    c = s["case"]
    x = s["logits"].double()
    if c["stats"]:
        lse = s["lse"].double()
    else:
        top = x.amax(1)
        top = torch.where(top > -math.inf, top, 0.0)
        lse = top + (x - top[:, None]).exp().sum(1).log()
    score = s["scores"].double().view(-1, 1)
    total = score + (x - lse[:, None])
    if c["finished"]:
        goes_on = torch.full_like(total, -math.inf)
        goes_on[:, s["end"]] = score[:, 0]
        total = torch.where(s["finished"].view(-1, 1), goes_on, total)
    total = torch.where(total.float() > -math.inf, total, -math.inf)
    total = total.view(c["items"], -1)
    best, at = torch.sort(total, dim=1, descending=True, stable=True)
    best, at = best[:, :c["picks"]], at[:, :c["picks"]]
    there = best > -math.inf
    parents = torch.where(there, at // c["vocab"], -1)
    tokens = torch.where(there, at % c["vocab"], -1)
    done = tokens == s["end"]
    if c["finished"]:
        done = done | (s["finished"].gather(1, parents.clamp(min=0)) & there)
    return {"tokens": tokens, "parents": parents, "picked": best.float(), "finished": done}


def _take(state, dim, rows):
    state.copy_(state.index_select(dim, rows))
    return state


def _plain_reorder(s):
    c, parents = s["case"], s["parents"]
    row = torch.arange(c["items"] * c["beams"], device="cuda").view(c["items"], c["beams"])
    source = torch.where(parents >= 0, row[:, :1] + parents, row).view(-1)
    return [_take(state, dim, source) for state, dim in s["states"]]


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "norm_grad":
            return _plain_norm_grad(s)
        if op == "beam_select":
            return _plain_select(s)
        _plain_reorder(s)
        return {"keys": s["keys"], "values": s["values"], "history": s["history"]}
    from tp_vocab_logits_gb300 import hg
    h = s["handle"]
    if op == "norm":
        hg.hg_norm_rows(h, s["x"], s["gain"], s["out"], residual=s["residual"], sum_out=s["sum"],
                        rstd=s["rstd"], scales=s["scales"], eps=EPS)
        return {k: s[k] for k in ("sum", "rstd", "out", "scales") if s[k] is not None}
    if op == "norm_grad":
        hg.hg_norm_rows_grad(h, s["sum"], s["gain"], s["rstd"], s["grad_out"], s["grad_x"],
                             s["grad_gain"], grad_sum=s["grad_sum"],
                             accumulate=s["case"]["accumulate"])
        return {"grad_x": s["grad_x"], "grad_gain": s["grad_gain"]}
    if op == "beam_select":
        hg.hg_beam_select(h, s["logits"], s["scores"], s["tokens"], s["parents"], s["picked"],
                          lse=s["lse"], finished=s["finished"], end=s["end"],
                          picked_finished=s["picked_finished"])
        return {"tokens": s["tokens"], "parents": s["parents"], "picked": s["picked"],
                "finished": s["picked_finished"]}
    hg.hg_beam_reorder(h, s["parents"], s["states"])
    return {"keys": s["keys"], "values": s["values"], "history": s["history"]}


# ---- work --------------------------------------------------------------------------


def work(case):
    c = case
    e = SIZES[c["dtype"]]
    if c["op"] == "norm":
        n, K = c["rows"], c["hidden"]
        # x and the residual in, the sum and out; the gain once.
        blocks = {"": 0, "row": 1, "block": -(-K // BLOCK)}[c["quant"]]
        per = e * (3 if c["residual"] else 1) + (1 if c["quant"] else e)
        return {"bytes": n * K * per + e * K + 4 * n * (1 + blocks), "flops": 6.0 * n * K}
    if c["op"] == "norm_grad":
        n, K = c["rows"], c["hidden"]
        per = 4 if c["residual"] else 3
        return {"bytes": e * (n * K * per + K * (3 if c["accumulate"] else 2)) + 4 * n,
                "flops": 10.0 * n * K}
    if c["op"] == "beam_select":
        # The logits of the beams that are searched, once.
        rows = c["items"] * c["beams"] * (1.0 - c["finished"]) * (1.0 - c["dead"])
        per = 1.0 if c["stats"] else 4.0
        return {"bytes": e * rows * c["vocab"] + 21 * c["items"] * c["picks"]
                + 8 * c["items"] * c["beams"], "flops": per * rows * c["vocab"]}
    # Rows that move are written; each row that some other one takes is read once.
    p = _chances(c["beams"]) * (1.0 - c["dead"])
    moved = float((1.0 - c["dead"] - p).sum())
    read = float((1.0 - (1.0 - p) ** (c["beams"] - 1)).sum())
    row = (2 * _cache_bytes(c, c["used"]) + 8 * c["items"] * c["beams"] * c["used"]) \
        / (c["items"] * c["beams"])
    return {"bytes": c["items"] * (moved + read) * row + 8 * c["items"] * c["beams"], "flops": 0.0}


# ---- exact values ------------------------------------------------------------------


def _exact_norm(s):
    c = s["case"]
    total, out = s["x"], {}
    if c["residual"]:
        total = (total.float() + s["residual"].float()).to(total.dtype)  # held in its type
        out["sum"] = total
    v = total.double()
    rstd = 1.0 / torch.sqrt((v * v).sum(1) / c["hidden"] + EPS)
    y = torch.einsum("nk,n,k->nk", v, rstd, s["gain"].double())
    out["rstd"] = rstd
    if not c["quant"]:
        return out | {"out": y}
    width = BLOCK if c["quant"] == "block" else c["hidden"]
    parts = y.split(width, 1)
    scales = torch.stack([p.abs().max(1).values / E4M3_MOST for p in parts], 1)
    scales[scales == 0] = 1.0
    q = torch.cat([p / scales[:, i:i + 1] for i, p in enumerate(parts)], 1)
    return out | {"out": q, "scales": scales}


def _exact_norm_grad(s):
    c = s["case"]
    v, r, g, gain = (s[k].double() for k in ("sum", "rstd", "grad_out", "gain"))
    inner = torch.einsum("nk,nk,k->n", v, g, gain) / c["hidden"]
    grad_x = torch.einsum("n,nk,k->nk", r, g, gain) - v * (inner * r ** 3)[:, None]
    if c["residual"]:
        grad_x += s["grad_sum"].double()
    grad_gain = torch.einsum("nk,nk,n->k", v, g, r)
    if c["accumulate"]:
        grad_gain += s["grad_gain"].double()
    return {"grad_x": grad_x, "grad_gain": grad_gain}


def _exact_select(s):
    c = s["case"]
    z = s["logits"].double()
    lse = s["lse"].double() if c["stats"] else torch.logsumexp(z, 1)
    shape = (c["items"], c["picks"])
    tokens = torch.full(shape, -1, device="cuda", dtype=torch.int64)
    parents, done = tokens.clone(), torch.zeros(shape, device="cuda", dtype=torch.bool)
    picked = torch.full(shape, -math.inf, device="cuda", dtype=torch.float64)
    for i in range(c["items"]):
        block = z[i * c["beams"]:(i + 1) * c["beams"]] - lse[i * c["beams"]:(i + 1) * c["beams"],
                                                             None]
        block += s["scores"][i].double()[:, None]
        if c["finished"]:
            on = s["finished"][i]
            block[on] = -math.inf
            block[on, s["end"]] = s["scores"][i][on].double()
        block = block.nan_to_num(nan=-math.inf, neginf=-math.inf, posinf=math.inf).view(-1)
        least = block.topk(c["picks"]).values[-1]
        at = ((block >= least) & (block > -math.inf)).nonzero()[:, 0]
        at = at[torch.argsort(block[at], descending=True, stable=True)][:c["picks"]]
        m = at.numel()
        parents[i, :m], tokens[i, :m], picked[i, :m] = at // c["vocab"], at % c["vocab"], block[at]
        done[i, :m] = tokens[i, :m] == s["end"]
        if c["finished"]:
            done[i, :m] |= s["finished"][i][parents[i, :m]]
    return {"tokens": tokens, "parents": parents, "picked": picked, "finished": done}


def _exact_reorder(s):
    c = s["case"]
    held = [(state, dim, state.clone()) for state, dim in s["states"]]
    for i, parents in enumerate(s["parents"].tolist()):
        for j, p in enumerate(parents):
            if 0 <= p < c["beams"]:
                for state, dim, old in held:
                    state.select(dim, i * c["beams"] + j).copy_(old.select(dim, i * c["beams"] + p))
    return {"keys": s["keys"], "values": s["values"], "history": s["history"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "beam_select": _exact_select,
            "beam_reorder": _exact_reorder}[case["op"]](s)
