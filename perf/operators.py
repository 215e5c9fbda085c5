"""The operators of a language model that this library serves around its counting sort, as cases that can be timed and
compared: token embedding and its gradient, a mixture-of-experts router and its gradient, and the experts of a
mixture-of-experts layer for a few tokens.

`run` computes a case either in plain torch operations (`own` false) or through the library (`own` true), from the
inputs that `prepare` makes on the GPU from a seed. `exact` computes the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn,
         "int32": torch.int32, "int64": torch.int64}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "fp8": 1, "int32": 4, "int64": 8}
BLOCK = 128  # rows and columns of an 8-bit weight matrix that share one scale


def listed():
    return [
        # one decoding step of 64 sequences: latency
        dict(name="embed decode", op="embed", tokens=64, dim=2048, rows=50257, dtype="bf16", ids="int64", scale=1.0),
        # the tokens of a training batch, scaled by sqrt(dim) as some models do
        dict(name="embed batch", op="embed", tokens=65536, dim=2048, rows=131072, dtype="bf16", ids="int64",
             scale=45.25483399593904),
        # a short fine-tuning step, odd width, gradient made anew (untouched rows are zero)
        dict(name="embed grad short", op="embed_grad", tokens=1003, dim=1000, rows=32000, dtype="fp16", ids="int64",
             out="fp16", add=False, scale=1.0),
        # the same batch as above in training: a whole new gradient of the table
        dict(name="embed grad batch", op="embed_grad", tokens=65536, dim=2048, rows=131072, dtype="bf16", ids="int64",
             out="bf16", add=False, scale=45.25483399593904),
        # gradient accumulation over micro-batches into a 32-bit gradient
        dict(name="embed grad add", op="embed_grad", tokens=16384, dim=4096, rows=50257, dtype="bf16", ids="int32",
             out="fp32", add=True, scale=1.0),
        # the router of one decoding step
        dict(name="route decode", op="route", tokens=256, experts=256, top_k=8, dtype="fp32", score="softmax",
             bias=False, renorm=True, masked=False, scale=1.0),
        # the router over a long prompt, with sigmoid scores, a selection bias and experts that are switched off
        dict(name="route prompt", op="route", tokens=65536, experts=256, top_k=8, dtype="bf16", score="sigmoid",
             bias=True, renorm=True, masked=True, scale=2.5),
        # training: the gradient of the router's weights, on few tokens and on a batch
        dict(name="route grad short", op="route_grad", tokens=1000, experts=60, top_k=4, dtype="bf16",
             score="softmax", bias=False, renorm=False, masked=False, scale=1.0),
        dict(name="route grad batch", op="route_grad", tokens=65536, experts=256, top_k=8, dtype="fp32",
             score="softmax", bias=False, renorm=True, masked=False, scale=1.0),
        # one sequence decoding: eight experts' weights are read for one token
        dict(name="experts one token", op="experts", tokens=1, experts=128, top_k=8, dim=2048, hidden=768,
             dtype="bf16", weights="bf16", skew=1.0),
        # 64 sequences decoding on weights held in 8 bits
        dict(name="experts 8 bit", op="experts", tokens=64, experts=64, top_k=6, dim=2048, hidden=1408,
             dtype="bf16", weights="fp8", skew=1.0),
        # 256 sequences decoding, top-8 of 256 experts: every expert's weights are read
        dict(name="experts decode", op="experts", tokens=256, experts=256, top_k=8, dim=2048, hidden=768,
             dtype="bf16", weights="bf16", skew=1.0),
    ]


def _log(rng, low, high):
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "route", "route_grad", "experts", "experts"])
    if op in ("embed", "embed_grad"):
        dim = _log(rng, 8, 8192)
        if rng.random() < 0.5:
            dim = max(8, dim // 8 * 8)
        rows = _log(rng, 64, min(262144, (1 << 28) // dim))
        tokens = _log(rng, 1, min(131072, (1 << 27) // dim))
        c = dict(op=op, tokens=tokens, dim=dim, rows=rows, dtype=rng.choice(["bf16", "fp16", "fp32"]),
                 ids=rng.choice(["int32", "int64"]), scale=rng.choice([1.0, math.sqrt(dim)]))
        if op == "embed_grad":
            c["out"] = rng.choice([c["dtype"], "fp32"])
            c["add"] = c["out"] == "fp32" and rng.random() < 0.5
        return c
    if op in ("route", "route_grad"):
        experts = _log(rng, 2, 511)
        return dict(op=op, tokens=_log(rng, 1, 131072), experts=experts, top_k=_log(rng, 1, min(16, experts)),
                    dtype=rng.choice(["bf16", "fp16", "fp32"]), score=rng.choice(["softmax", "sigmoid"]),
                    bias=op == "route" and rng.random() < 0.5, renorm=rng.random() < 0.5, masked=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]))
    dim = _log(rng, 64, 4096)
    hidden = _log(rng, 32, 2048)
    if rng.random() < 0.7:
        dim, hidden = max(64, dim // 64 * 64), max(32, hidden // 32 * 32)
    experts = _log(rng, 4, min(256, max(4, (1 << 30) // (3 * dim * hidden))))
    top_k = _log(rng, 1, min(8, experts))
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    return dict(op=op, tokens=_log(rng, 1, 512), experts=experts, top_k=top_k, dim=dim, hidden=hidden, dtype=dtype,
                weights=rng.choice([dtype, dtype, "fp8"]), skew=rng.choice([0.0, 1.0]))


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------
def _tokens(c, g):
    """Token ids with the skew of text (the r-th most frequent token has a share of 1/r), spread over the table; one in
    a hundred is -1, as packed batches mark padding."""
    n, rows = c["tokens"], c["rows"]
    rank = (torch.rand(n, generator=g, device="cuda", dtype=torch.float64) * math.log(rows + 1)).exp().long() - 1
    ids = (rank.clamp_(0, rows - 1) * 7919 + 13) % rows
    ids[torch.rand(n, generator=g, device="cuda") < 0.01] = -1
    return ids.to(TYPES[c["ids"]])


def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _choices(c, g):
    """Distinct experts per token, in order of choice: expert of popularity rank r is drawn with weight (r + 1)^-skew."""
    t, e, k = c["tokens"], c["experts"], c["top_k"]
    popular = torch.randperm(e, generator=g, device="cuda").float().add_(1).log_().mul_(-c["skew"])
    u = torch.rand((t, e), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    score = popular - torch.log(-torch.log(u))
    return score.topk(k, dim=1).indices.to(torch.int32)


def _eight_bit(g, experts, rows, cols):
    """Weights of a size that keeps activations near 1: 8-bit values and a 32-bit scale for each block of 128 x 128."""
    q = _normal(g, (experts, rows, cols), torch.bfloat16, 64.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
    grid = (experts, -(-rows // BLOCK), -(-cols // BLOCK))
    s = (torch.rand(grid, generator=g, device="cuda") + 0.5) / (64.0 * math.sqrt(cols))
    return q, s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    if c["op"] == "embed":
        s["table"] = _normal(g, (c["rows"], c["dim"]), TYPES[c["dtype"]])
        s["ids"] = _tokens(c, g)
    elif c["op"] == "embed_grad":
        s["dout"] = _normal(g, (c["tokens"], c["dim"]), TYPES[c["dtype"]])
        s["ids"] = _tokens(c, g)
        if c["add"]:  # the gradient of the micro-batches before
            s["grad"] = _normal(g, (c["rows"], c["dim"]), TYPES[c["out"]])
    elif c["op"] in ("route", "route_grad"):
        t, e = c["tokens"], c["experts"]
        logits = _normal(g, (t, e), TYPES[c["dtype"]], 1.5)
        if c["masked"]:  # experts that are switched off for a token, and tokens that have none (padding)
            logits.masked_fill_(torch.rand((t, e), generator=g, device="cuda") < 0.3, float("-inf"))
            logits.masked_fill_(torch.rand((t, 1), generator=g, device="cuda") < 0.01, float("-inf"))
        s["logits"] = logits
        if c["op"] == "route":
            s["bias"] = _normal(g, (e,), torch.float32, 0.3) if c["bias"] else None
        else:
            s["ids"] = _select(logits, None, c["top_k"])[0].to(torch.int32)
            s["dweights"] = _normal(g, (t, c["top_k"]), torch.float32)
    else:
        e, d, f = c["experts"], c["dim"], c["hidden"]
        s["x"] = _normal(g, (c["tokens"], d), TYPES[c["dtype"]])
        s["ids"] = _choices(c, g)
        s["weights"] = torch.rand((c["tokens"], c["top_k"]), generator=g, device="cuda").add_(0.1)
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        s["s_in"] = s["s_out"] = None
        if c["weights"] == "fp8":
            s["w_in"], s["s_in"] = _eight_bit(g, e, 2 * f, d)
            s["w_out"], s["s_out"] = _eight_bit(g, e, d, f)
        else:
            s["w_in"] = _normal(g, (e, 2 * f, d), TYPES[c["weights"]], d ** -0.5)
            s["w_out"] = _normal(g, (e, d, f), TYPES[c["weights"]], f ** -0.5)
    return s


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms, in 32 bits
# ---------------------------------------------------------------------------------------------------------------------
def _embed(s, c):
    ids = s["ids"].long()
    live = (ids >= 0) & (ids < c["rows"])
    y = s["table"][ids.clamp(0, c["rows"] - 1)].float() * c["scale"]
    return torch.where(live[:, None], y, 0.0).to(s["table"].dtype)


def _embed_grad(s, c):
    ids = s["ids"].long()
    ids = torch.where((ids >= 0) & (ids < c["rows"]), ids, c["rows"])  # one row more takes what belongs to none
    grad = torch.zeros((c["rows"] + 1, c["dim"]), device="cuda")
    grad.index_add_(0, ids, s["dout"].float())
    grad = grad[: c["rows"]] * c["scale"]
    return s["grad"].add_(grad) if c["add"] else grad.to(TYPES[c["out"]])


def _select(logits, bias, top_k):
    """The top_k experts of each token by logit + bias (ties to the lowest index), -1 where no expert is left; and
    which experts can be chosen at all (those that are not at -inf or NaN)."""
    sel = logits.float() if bias is None else logits.float() + bias
    can = sel > float("-inf")
    value, order = torch.sort(torch.where(can, sel, float("-inf")), dim=1, descending=True, stable=True)
    value, order = value[:, :top_k], order[:, :top_k]
    return torch.where(value > float("-inf"), order, -1), can


def _scores(logits, can, score):
    """softmax over the experts that can be chosen, or the sigmoid of each; 0 for the others."""
    l = logits.float()
    if score == "sigmoid":
        return torch.where(can, 1 / (1 + torch.exp(-l)), 0.0)
    l = torch.where(can, l, float("-inf"))
    top = l.amax(1, keepdim=True)
    p = torch.where(can, torch.exp(l - torch.where(top > float("-inf"), top, 0.0)), 0.0)
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, 1.0)


def _route(s, c):
    ids, can = _select(s["logits"], s["bias"], c["top_k"])
    p = torch.where(ids >= 0, _scores(s["logits"], can, c["score"]).gather(1, ids.clamp(min=0)), 0.0)
    if c["renorm"]:
        total = p.sum(1, keepdim=True)
        p = p / torch.where(total > 0, total, 1.0)
    return p * c["scale"], ids.to(torch.int32)


def _route_grad(s, c):
    ids = s["ids"].long()
    live, ids = ids >= 0, ids.clamp(min=0)
    l = s["logits"].float()
    p = _scores(s["logits"], l > float("-inf"), c["score"])
    q = torch.where(live, p.gather(1, ids), 0.0)
    dq = torch.where(live, s["dweights"] * c["scale"], 0.0)
    if c["renorm"]:
        total = q.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        q = q / total
        dq = (dq - (dq * q).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(l).scatter_add_(1, ids, torch.where(live, dq, 0.0))
    if c["score"] == "sigmoid":
        dl = dp * p * (1 - p)
    else:
        dl = p * (dp - (dp * p).sum(1, keepdim=True))
    return dl.to(s["logits"].dtype)


def _widen(w, scale):
    if scale is None:
        return w.float()
    rows, cols = w.shape[1:]
    scale = scale.repeat_interleave(BLOCK, 1)[:, :rows].repeat_interleave(BLOCK, 2)[:, :, :cols]
    return w.float() * scale


def _experts(s, c):
    """The assignments, grouped by expert into rows of a padded batch, through each used expert's products."""
    k, f = c["top_k"], c["hidden"]
    used, which, count = s["ids"].long().reshape(-1).unique(return_inverse=True, return_counts=True)
    order = which.argsort(stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device="cuda") - (count.cumsum(0) - count)[which[order]]
    x = torch.zeros((used.numel(), int(count.max()), c["dim"]), device="cuda")
    x[which, place] = s["x"].float().repeat_interleave(k, 0)
    w_in = _widen(s["w_in"][used], None if s["s_in"] is None else s["s_in"][used])
    h = torch.bmm(x, w_in.transpose(1, 2).contiguous())
    h = h[:, :, :f] / (1 + torch.exp(-h[:, :, :f])) * h[:, :, f:]
    w_out = _widen(s["w_out"][used], None if s["s_out"] is None else s["s_out"][used])
    y = torch.bmm(h, w_out.transpose(1, 2).contiguous())[which, place]
    return (y.view(c["tokens"], k, c["dim"]) * s["weights"][:, :, None]).sum(1).to(s["x"].dtype)


# ---------------------------------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------------------------------
def _library(s, c):
    import primitives_device_scan_amd as ds

    if c["op"] == "embed":
        return ds.embedding(s["table"], s["ids"], scale=c["scale"])
    if c["op"] == "embed_grad":
        return ds.embedding_grad(s["dout"], s["ids"], c["rows"], scale=c["scale"], dtype=TYPES[c["out"]],
                                 out=s.get("grad"), accumulate=c["add"])
    if c["op"] == "route":
        return ds.moe_route(s["logits"], c["top_k"], score=c["score"], bias=s["bias"], renormalize=c["renorm"],
                            scale=c["scale"])
    if c["op"] == "route_grad":
        return ds.moe_route_grad(s["logits"], s["ids"], s["dweights"], score=c["score"], renormalize=c["renorm"],
                                 scale=c["scale"])
    return ds.moe_experts(s["x"], s["w_in"], s["w_out"], s["ids"], s["weights"], w_in_scale=s["s_in"],
                          w_out_scale=s["s_out"])


PLAIN = {"embed": _embed, "embed_grad": _embed_grad, "route": _route, "route_grad": _route_grad, "experts": _experts}


def run(state):
    c = state["case"]
    return _library(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def _distinct(share, n):
    """Expected number of different outcomes among n independent draws, outcome i with probability share[i]."""
    return sum(-math.expm1(n * math.log1p(-min(p, 1 - 1e-12))) for p in share)


def _rows_read(c):
    h = math.log(c["rows"] + 1)
    return _distinct([math.log1p(1 / (r + 1)) / h for r in range(c["rows"])], c["tokens"] * 0.99)


def _experts_read(c):
    """Expected number of experts that some token has among its top_k: expert e is in with probability
    1 - exp(-t w_e), where t makes these sum to top_k."""
    w = [(r + 1.0) ** -c["skew"] for r in range(c["experts"])]
    if c["top_k"] == c["experts"]:
        return c["experts"]
    low, high = 0.0, 1e9
    for _ in range(200):
        t = (low + high) / 2
        low, high = (t, high) if sum(-math.expm1(-t * x) for x in w) < c["top_k"] else (low, t)
    return _distinct([-math.expm1(-t * x) for x in w], c["tokens"])


def work(case):
    c = case
    z, n = SIZE[c["dtype"]], c["tokens"]
    if c["op"] == "embed":
        return {"bytes": _rows_read(c) * c["dim"] * z + n * (c["dim"] * z + SIZE[c["ids"]]), "flops": n * c["dim"]}
    if c["op"] == "embed_grad":
        moved = _rows_read(c) * 2 if c["add"] else c["rows"]  # rows of the gradient that are read or written
        return {"bytes": n * (c["dim"] * z + SIZE[c["ids"]]) + moved * c["dim"] * SIZE[c["out"]],
                "flops": 2 * n * c["dim"]}
    if c["op"] == "route":
        return {"bytes": n * (c["experts"] * z + c["top_k"] * 8), "flops": n * c["experts"] * 4}
    if c["op"] == "route_grad":
        return {"bytes": n * (2 * c["experts"] * z + c["top_k"] * 8), "flops": n * c["experts"] * 8}
    d, f, k = c["dim"], c["hidden"], c["top_k"]
    each = 3 * d * f * SIZE[c["weights"]]
    if c["weights"] == "fp8":
        each += 4 * (-(-2 * f // BLOCK) * -(-d // BLOCK) + -(-d // BLOCK) * -(-f // BLOCK))
    return {"bytes": _experts_read(c) * each + 2 * n * d * z + n * k * 8, "flops": n * k * 6 * d * f}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] == "embed":
        table = torch.cat([s["table"].double(), torch.zeros((1, c["dim"]), dtype=torch.float64, device="cuda")])
        ids = s["ids"].long()
        return table[torch.where(ids < 0, c["rows"], ids)] * c["scale"]
    if c["op"] == "embed_grad":
        # rows in order of their token; a token's sum is the difference of two running sums
        ids, order = s["ids"].long().sort(stable=True)
        total = torch.zeros((c["tokens"] + 1, c["dim"]), dtype=torch.float64, device="cuda")
        torch.cumsum(s["dout"][order].double(), 0, out=total[1:])
        at = torch.searchsorted(ids, torch.arange(c["rows"] + 1, device="cuda"))
        grad = (total[at[1:]] - total[at[:-1]]) * c["scale"]
        return grad + s["grad"].double() if c["add"] else grad
    if c["op"] == "route":
        sel = s["logits"].float()
        sel = torch.nan_to_num(sel if s["bias"] is None else sel + s["bias"], nan=-math.inf, neginf=-math.inf)
        odds = _odds(s["logits"], sel != -math.inf, c["score"])
        got = []
        for _ in range(c["top_k"]):
            best = sel.argmax(1, keepdim=True)
            got.append(odds.gather(1, best) * (sel.gather(1, best) != -math.inf))
            sel = sel.scatter(1, best, -math.inf)
        got = torch.cat(got, 1)
        # an odds row is a score up to a factor of its own, which a share of the chosen ones does not see
        whole = got if c["renorm"] else odds if c["score"] == "softmax" else None
        if whole is not None:
            got = got / whole.sum(1, keepdim=True).clamp(min=1e-300)
        return got * c["scale"], None
    if c["op"] == "route_grad":
        # d w_j / d l_e from the definition of the weights, token by token: t x top_k x experts values, in pieces
        size = max(1, (1 << 26) // (c["top_k"] * c["experts"]))
        return torch.cat([_route_vjp(s, c, slice(t, t + size)) for t in range(0, c["tokens"], size)])
    x, w, y = s["x"].double(), s["weights"].double(), torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        token, slot = (s["ids"] == e).nonzero(as_tuple=True)
        if token.numel():
            w_in, w_out = (_dense(s, name, e) for name in ("in", "out"))
            gate, up = (x[token] @ w_in.T.contiguous()).split(c["hidden"], 1)
            h = gate * torch.sigmoid(gate) * up
            y.index_add_(0, token, (h @ w_out.T.contiguous()) * w[token, slot, None])
    return y


def _dense(s, name, e):
    w, scale = s["w_" + name][e].double(), s["s_" + name]
    if scale is not None:
        i, j = (torch.arange(n, device="cuda") // BLOCK for n in w.shape)
        w = w * scale[e].double()[i][:, j]
    return w


def _odds(logits, can, score):
    l = torch.where(can, logits.double(), -math.inf)
    if score == "sigmoid":
        return torch.sigmoid(l)
    top = l.max(1, keepdim=True).values
    return torch.where(can, (l - top.clamp(min=-1e300)).exp(), 0.0)


def _route_vjp(s, c, part):
    l, ids, dw = s["logits"][part].double(), s["ids"][part].long(), s["dweights"][part].double() * c["scale"]
    chosen = torch.nn.functional.one_hot(ids + 1, c["experts"] + 1)[:, :, 1:].double()  # t x k x e; -1: no expert
    odds = _odds(s["logits"][part], l > -math.inf, c["score"])
    mine = (chosen * odds[:, None]).sum(2)  # t x k
    slope = odds * (1 - odds) if c["score"] == "sigmoid" else odds  # d odds / d logit
    if c["renorm"]:
        whole, spread = mine.sum(1), chosen.sum(1) * slope
    elif c["score"] == "softmax":
        whole, spread = odds.sum(1), slope
    else:
        return (chosen * dw[:, :, None]).sum(1) * slope
    whole = whole.clamp(min=1e-300)[:, None]
    direct = (chosen * dw[:, :, None]).sum(1) * slope / whole
    return direct - spread * (dw * mine).sum(1, keepdim=True) / whole ** 2
