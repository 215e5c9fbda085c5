"""The operators of a language model that work on ragged batches, as cases that can be timed and compared: a gated linear
recurrence over packed sequences, its gradient and its step for single tokens; matrix products grouped by expert and the
gradient of their weights; page tables and slot maps of requests.

`run` computes a case either in plain torch operations (`own` false) or through the library (`own` true), from the
inputs that `prepare` makes on the GPU from a seed. `exact` computes the same outputs in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
MOST = 1 << 27  # elements of a recurrence's inputs


def listed():
    return [
        # one request's prompt of odd length and width through a recurrent layer
        dict(name="scan prompt", op="scan", tokens=777, dim=1000, sequences=1, dtype="fp16", form="log", mix=False,
             initial=False),
        # a training or prefill batch of 32 packed sequences, gates as logits and inputs weighted by 1 - gate
        dict(name="scan batch", op="scan", tokens=65536, dim=2048, sequences=32, dtype="bf16", form="sigmoid", mix=True,
             initial=True),
        # a short fine-tuning step in 32 bits, five sequences, gates given as they are
        dict(name="scan grad short", op="scan_grad", tokens=1003, dim=1000, sequences=5, dtype="fp32", form="decay",
             mix=False, initial=True),
        # one long sequence in training
        dict(name="scan grad long", op="scan_grad", tokens=32768, dim=4096, sequences=1, dtype="bf16", form="sigmoid",
             mix=True, initial=False),
        # a decoding step of 64 sequences: latency
        dict(name="step decode", op="step", tokens=64, dim=2048, slots=64, dtype="bf16", form="sigmoid", mix=True),
        # a decoding step of a full server, states in a pool
        dict(name="step pool", op="step", tokens=1024, dim=4096, slots=4096, dtype="bf16", form="log", mix=False),
        # the gate and up products of a prompt's tokens in a mixture-of-experts layer, rows taken from the tokens
        dict(name="grouped prompt", op="grouped", tokens=8192, top_k=8, experts=64, rows=1536, cols=2048, dtype="bf16",
             block=16, gather=True, transposed=False, skew=0.5),
        # the gradient of the inputs of a short fine-tuning step, odd sizes
        dict(name="grouped short", op="grouped", tokens=1003, top_k=2, experts=20, rows=777, cols=1000, dtype="fp16",
             block=1, gather=False, transposed=True, skew=1.0),
        # the gradient of the weights of those gate and up products, as a batch in training
        dict(name="grouped grad batch", op="grouped_grad", tokens=8192, top_k=8, experts=64, rows=1536, cols=2048,
             dtype="bf16", block=16, gather=True, out="bf16", add=False, skew=0.5),
        # gradient accumulation over micro-batches into 32-bit gradients, few experts
        dict(name="grouped grad add", op="grouped_grad", tokens=1000, top_k=2, experts=8, rows=1024, cols=1024,
             dtype="bf16", block=1, gather=False, out="fp32", add=True, skew=1.0),
        # a decoding step of 256 requests: one token each, a page now and then
        dict(name="pages decode", op="pages", requests=256, longest=1, context=8192, page=16, spare=0),
        # prompts of 512 requests, packed into a batch with room to spare
        dict(name="pages prompts", op="pages", requests=512, longest=512, context=4096, page=64, spare=1000),
    ]


def _log(rng, low, high):
    return min(high, int(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))


def draw(rng):
    op = rng.choice(["scan", "scan_grad", "step", "grouped", "grouped", "grouped_grad", "pages"])
    if op in ("scan", "scan_grad", "step"):
        dim = _log(rng, 16, 8192)
        if rng.random() < 0.5:
            dim = max(16, dim // 64 * 64)
        c = dict(op=op, tokens=_log(rng, 1, min(65536, MOST // dim)), dim=dim,
                 dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), form=rng.choice(["decay", "log", "sigmoid"]),
                 mix=rng.random() < 0.5)
        if c["dtype"] == "fp32":
            c["tokens"] = (c["tokens"] + 1) // 2
        if op == "step":
            c["tokens"] = min(c["tokens"], 4096)
            c["slots"] = rng.choice([c["tokens"], 2 * c["tokens"] + 5])
        else:
            c["sequences"] = _log(rng, 1, min(1024, c["tokens"]))
            c["initial"] = rng.random() < 0.5
        return c
    if op == "pages":
        return dict(op=op, requests=_log(rng, 1, 4096), longest=_log(rng, 1, 64), context=_log(rng, 16, 32768),
                    page=rng.choice([1, 16, 24, 64, 128]), spare=rng.choice([0, 0, 777]))
    rows, cols = _log(rng, 64, 4096), _log(rng, 64, 4096)
    if rng.random() < 0.7:
        rows, cols = max(64, rows // 64 * 64), max(64, cols // 64 * 64)
    experts = _log(rng, 1, min(256, max(1, (1 << 28) // (rows * cols))))
    top_k = _log(rng, 1, min(8, experts))
    tokens = _log(rng, 1, max(1, min(16384, 65536 // top_k, (3 << 36) // (2 * rows * cols * top_k))))
    c = dict(op=op, tokens=tokens, top_k=top_k, experts=experts, rows=rows, cols=cols,
             dtype=rng.choice(["bf16", "bf16", "fp16"]), block=rng.choice([1, 16, 64]), gather=rng.random() < 0.5,
             skew=rng.choice([0.0, 0.5, 1.0]))
    if op == "grouped":
        c["transposed"] = rng.random() < 0.4
    else:
        c["out"] = rng.choice([c["dtype"], "fp32"])
        c["add"] = c["out"] == "fp32" and rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------
def _normal(g, shape, dtype, std=1.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=dtype).mul_(std)


def _gates(c, g):
    """Gates as a trained layer has them: most keep their state for some tens of steps, some for thousands."""
    shape = (c["tokens"], c["dim"])
    keep = _normal(g, (c["dim"],), torch.float32, 2.0) + 3.0  # logit of a channel's usual gate
    logit = _normal(g, shape, torch.float32).add_(keep)
    if c["form"] == "sigmoid":
        return logit.to(TYPES[c["dtype"]])
    if c["form"] == "log":
        return torch.log1p(torch.exp(logit.neg_())).neg_().to(TYPES[c["dtype"]])
    return torch.sigmoid(logit).to(TYPES[c["dtype"]])


def _offsets(c, seed):
    """Offsets of the packed sequences: lengths that differ, and among many sequences one in sixteen is empty."""
    rng = random.Random(seed)
    n, s = c["tokens"], c["sequences"]
    share = [0.0 if s >= 4 and rng.random() < 1 / 16 else rng.expovariate(1.0) + 0.1 for _ in range(s)]
    share[0] = share[0] or 1.0
    at, total, offsets = 0.0, sum(share), [0]
    for v in share:
        at += v
        offsets.append(min(n, int(n * at / total + 0.5)))
    offsets[-1] = n
    return torch.tensor(offsets, dtype=torch.int32, device="cuda")


def _choices(c, g):
    """Distinct experts per token; the expert of popularity rank r is drawn with weight (r + 1)^-skew."""
    popular = torch.randperm(c["experts"], generator=g, device="cuda").float().add_(1).log_().mul_(-c["skew"])
    u = torch.rand((c["tokens"], c["experts"]), generator=g, device="cuda").clamp_(1e-7, 1 - 1e-7)
    return (popular - torch.log(-torch.log(u))).topk(c["top_k"], dim=1).indices.reshape(-1)


def _grouping(c, g):
    """Assignments by expert, each expert's part padded to a multiple of block with the mark n, as the MoE alignment
    writes them: (offsets [experts + 1], index [n + experts * (block - 1)])."""
    ids, n, e, block = _choices(c, g), c["tokens"] * c["top_k"], c["experts"], c["block"]
    count = torch.bincount(ids, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    torch.cumsum((count + block - 1) // block * block, 0, out=offsets[1:])
    order = torch.argsort(ids, stable=True)
    place = torch.arange(n, device="cuda") - (count.cumsum(0) - count)[ids[order]] + offsets[ids[order]]
    index = torch.full((n + e * (block - 1),), n, dtype=torch.int32, device="cuda")
    index[place] = order.to(torch.int32)
    return offsets.to(torch.int32), index


def _new_tokens(c):
    return c["requests"] // 2 * (c["longest"] + 1) + c["requests"] % 2 * ((c["longest"] + 1) // 2)


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": c}
    op = c["op"]
    if op == "pages":
        n, page = c["requests"], c["page"]

        def whole(low, high, shape):
            return torch.randint(low, high + 1, shape, generator=g, device="cuda", dtype=torch.int32)

        s["context"], s["new"] = whole(0, c["context"], (n,)), whole(1, c["longest"], (n,))
        pairs = s["new"][: n // 2]
        s["new"][n - n // 2:] = c["longest"] + 1 - pairs.flip(0)  # as many tokens whatever the seed
        if n % 2:
            s["new"][n // 2] = (c["longest"] + 1) // 2
        width = -(-(c["context"] + c["longest"]) // page)
        total = n * width
        pages = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
        s["tables"] = pages.view(n, width).clone()  # a request's later entries are left over from earlier ones
        held = (s["context"] + page - 1) // page
        s["free"] = torch.cat([r[h:] for r, h in zip(s["tables"], held.tolist())])
        s["count"] = torch.tensor([s["free"].numel()], dtype=torch.int32, device="cuda")
        s["tokens"] = _new_tokens(c) + c["spare"]
        return s
    dtype = TYPES[c["dtype"]]
    if op in ("scan", "scan_grad", "step"):
        shape = (c["tokens"], c["dim"])
        s["gate"], s["x"] = _gates(c, g), _normal(g, shape, dtype)
        if op == "step":
            s["state"] = _normal(g, (c["slots"], c["dim"]), torch.float32)
            s["slots"] = None
            if c["slots"] != c["tokens"]:  # one in 64 is a row that only fills the batch
                s["slots"] = torch.randperm(c["slots"], generator=g, device="cuda")[: c["tokens"]].to(torch.int32)
                s["slots"][torch.rand(c["tokens"], generator=g, device="cuda") < 1 / 64] = -1
            return s
        s["offsets"] = _offsets(c, seed)
        states = (c["sequences"], c["dim"])
        s["initial"] = _normal(g, states, torch.float32) if c["initial"] else None
        if op == "scan_grad":
            s["h"] = _scan(s, c)[0]
            s["dh"], s["dfinal"] = _normal(g, shape, dtype), _normal(g, states, torch.float32)
            if not c["mix"]:
                s["x"] = None  # the gradient does not need it
        return s
    s["offsets"], s["index"] = _grouping(c, g)
    rows, cols, m = c["rows"], c["cols"], s["index"].numel()
    if not c["gather"]:
        s["index"] = None
    width = rows if op == "grouped" and c["transposed"] else cols
    if c["gather"]:
        s["x"] = _normal(g, (c["tokens"], width), dtype)
    else:
        s["x"] = _normal(g, (m, width), dtype)
    if op == "grouped":
        s["w"] = _normal(g, (c["experts"], rows, cols), dtype, width ** -0.5)
        s["y"] = torch.zeros((m, rows + cols - width), dtype=dtype, device="cuda")  # rows behind the last stay as they are
    else:
        s["dy"] = _normal(g, (m, rows), dtype)
        s["dw"] = _normal(g, (c["experts"], rows, cols), torch.float32) if c["add"] else None
    return s


# ---------------------------------------------------------------------------------------------------------------------
# Plain forms, in 32 bits; the recurrences in 64, since a gate near 1 to 32 bits is some steps off over thousands
# ---------------------------------------------------------------------------------------------------------------------
def _decay(g, form):
    """(a, 1 - a, d a / d gate)"""
    if form == "sigmoid":
        up, down = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
        return up, down, up * down
    if form == "log":
        a = torch.exp(g)
        return a, -torch.expm1(g), a
    return g, 1 - g, torch.ones_like(g)


def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t by doubling: after the step of distance d each pair (a, b) covers 2 d steps."""
    d = 1
    while d < a.shape[0]:
        b = torch.cat([b[:d], a[d:] * b[:-d] + b[d:]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _ends(offsets):
    """Sequences that are not empty, their first and their last tokens."""
    o = offsets.long()
    live = (o[1:] > o[:-1]).nonzero().squeeze(1)
    return live, o[live], o[live + 1] - 1


def _scan(s, c):
    a, rest, _ = _decay(s["gate"].double(), c["form"])
    b = rest * s["x"] if c["mix"] else s["x"].double()
    live, first, last = _ends(s["offsets"])
    if s["initial"] is not None:
        b = b.index_put((first,), b[first] + a[first] * s["initial"][live])
    h = _recur(a.index_fill(0, first, 0.0), b)
    final = torch.zeros((c["sequences"], c["dim"]), device="cuda") if s["initial"] is None else s["initial"].clone()
    final[live] = h[last].float()
    return h.to(s["gate"].dtype), final


def _scan_grad(s, c):
    a, rest, slope = _decay(s["gate"].double(), c["form"])
    live, first, last = _ends(s["offsets"])
    dh = s["dh"].double()
    dh[last] += s["dfinal"][live]
    onward = torch.cat([a[1:], a[:1]]).index_fill(0, last, 0.0)
    total = _recur(onward.flip(0), dh.flip(0)).flip(0)
    before = torch.cat([s["h"][:1], s["h"][:-1]]).double()
    before[first] = 0.0 if s["initial"] is None else s["initial"][live].double()
    dinitial = s["dfinal"].clone()
    dinitial[live] = (a[first] * total[first]).float()
    if c["mix"]:
        dgate, dx = total * (before - s["x"]) * slope, total * rest
    else:
        dgate, dx = total * before * slope, total
    return dgate.to(s["gate"].dtype), dx.to(s["gate"].dtype), dinitial


def _step(s, c):
    a, rest, _ = _decay(s["gate"].float(), c["form"])
    b = rest * s["x"].float() if c["mix"] else s["x"].float()
    if s["slots"] is None:
        s["state"].mul_(a).add_(b)
        return s["state"].to(s["x"].dtype), s["state"]
    at = s["slots"].long()
    live = at >= 0
    h = torch.where(live[:, None], a * s["state"][at.clamp(min=0)] + b, 0.0)
    s["state"][at[live]] = h[live]
    return h.to(s["x"].dtype), s["state"]


def _rows_of(s, c):
    """The rows of the grouped batch in 32 bits: those of x, or the tokens that the index names."""
    x = s["x"].float()
    if s["index"] is None:
        return x
    x = torch.cat([x, torch.zeros((1, x.shape[1]), device="cuda")])
    return x[torch.div(s["index"].long(), c["top_k"], rounding_mode="floor").clamp(max=c["tokens"])]


def _grouped(s, c):
    x, at = _rows_of(s, c), s["offsets"].tolist()
    for e in range(c["experts"]):
        if at[e + 1] > at[e]:
            w = s["w"][e].float()
            s["y"][at[e]:at[e + 1]] = x[at[e]:at[e + 1]] @ (w if c["transposed"] else w.T)
    return s["y"]


def _grouped_grad(s, c):
    x, at = _rows_of(s, c), s["offsets"].tolist()
    dw = s["dw"] if c["add"] else torch.zeros((c["experts"], c["rows"], c["cols"]), dtype=TYPES[c["out"]], device="cuda")
    for e in range(c["experts"]):
        if at[e + 1] > at[e]:
            dw[e] += s["dy"][at[e]:at[e + 1]].float().T @ x[at[e]:at[e + 1]]
    return dw


def _pages(s, c):
    page, tables, context, new = c["page"], s["tables"], s["context"].long(), s["new"].long()
    n, width = tables.shape
    offsets = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = new.cumsum(0)
    held = (context + page - 1) // page
    need = (context + new + page - 1) // page - held
    from_free = torch.arange(width, device="cuda") - held[:, None]
    take = (from_free >= 0) & (from_free < need[:, None])
    rank = (need.cumsum(0) - need)[:, None] + from_free
    top = s["count"].long() - 1
    tables[take] = s["free"][(top - rank[take]).clamp(min=0)]
    request = torch.repeat_interleave(torch.arange(n, device="cuda"), new)
    position = context[request] + torch.arange(request.numel(), device="cuda") - offsets.long()[request]
    slots = torch.full((s["tokens"],), -1, dtype=torch.int64, device="cuda")
    positions = torch.zeros(s["tokens"], dtype=torch.int32, device="cuda")
    slots[: request.numel()] = tables[request, position // page].long() * page + position % page
    positions[: request.numel()] = position.to(torch.int32)
    return offsets, slots, positions, (s["count"] - need.sum()).to(torch.int32), tables


# ---------------------------------------------------------------------------------------------------------------------
# The library's calls
# ---------------------------------------------------------------------------------------------------------------------
def _library(s, c):
    import primitives_device_scan_amd as ds

    op = c["op"]
    if op == "scan":
        return ds.gated_scan(s["gate"], s["x"], s["offsets"], form=c["form"], mix=c["mix"], initial=s["initial"])
    if op == "scan_grad":
        return ds.gated_scan_grad(s["gate"], s["h"], s["dh"], s["offsets"], x=s["x"], form=c["form"], mix=c["mix"],
                                  initial=s["initial"], dfinal=s["dfinal"])
    if op == "step":
        return ds.gated_step(s["gate"], s["x"], s["state"], s["slots"], form=c["form"], mix=c["mix"]), s["state"]
    if op == "grouped":
        return ds.grouped_matmul(s["x"], s["w"], s["offsets"], index=s["index"], top_k=c["top_k"],
                                 transposed=c["transposed"], out=s["y"])
    if op == "grouped_grad":
        return ds.grouped_matmul_grad(s["dy"], s["x"], s["offsets"], index=s["index"], top_k=c["top_k"],
                                      dtype=TYPES[c["out"]], out=s["dw"], accumulate=c["add"])
    return *ds.page_slots(s["context"], s["new"], s["tables"], s["free"], s["count"], c["page"], s["tokens"]), s["tables"]


PLAIN = {"scan": _scan, "scan_grad": _scan_grad, "step": _step, "grouped": _grouped, "grouped_grad": _grouped_grad,
         "pages": _pages}


def run(state):
    c = state["case"]
    return _library(state, c) if own else PLAIN[c["op"]](state, c)


# ---------------------------------------------------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------------------------------------------------
def _experts_read(c):
    """Expected number of experts that some token has among its top_k: expert e is in with probability
    1 - exp(-t w_e), where t makes these sum to top_k."""
    if c["top_k"] == c["experts"]:
        return c["experts"]
    w = [(r + 1.0) ** -c["skew"] for r in range(c["experts"])]
    low, high = 0.0, 1e9
    for _ in range(200):
        t = (low + high) / 2
        low, high = (t, high) if sum(-math.expm1(-t * x) for x in w) < c["top_k"] else (low, t)
    return sum(-math.expm1(-c["tokens"] * t * x) for x in w)


def work(case):
    c = case
    op = c["op"]
    if op == "pages":
        tokens = _new_tokens(c)
        taken = tokens / c["page"]
        return {"bytes": c["requests"] * 12 + 8 * taken + 12 * (tokens + c["spare"]), "flops": 4 * tokens}
    z = SIZE[c["dtype"]]
    if op in ("scan", "scan_grad", "step"):
        n = c["tokens"] * c["dim"]
        if op == "step":
            return {"bytes": n * (3 * z + 8), "flops": n * 8}
        states = c["sequences"] * c["dim"] * 4
        if op == "scan":
            return {"bytes": n * 3 * z + states * (1 + c["initial"]), "flops": n * 8}
        return {"bytes": n * (5 + c["mix"]) * z + states * (2 + c["initial"]), "flops": n * 12}
    n = c["tokens"] * c["top_k"]
    wide = c["rows"] if op == "grouped" and c["transposed"] else c["cols"]
    each, flops = c["rows"] * c["cols"], 2 * n * c["rows"] * c["cols"]
    into = (c["tokens"] if c["gather"] else n) * wide * z + n * 4 * c["gather"]
    if op == "grouped":
        return {"bytes": into + n * (c["rows"] + c["cols"] - wide) * z + _experts_read(c) * each * z, "flops": flops}
    moved = _experts_read(c) * 2 if c["add"] else c["experts"]  # matrices of the gradient that are read or written
    return {"bytes": into + n * c["rows"] * z + moved * each * SIZE[c["out"]], "flops": flops}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions, in 64 bits
# ---------------------------------------------------------------------------------------------------------------------
def _gate_exact(g, form):
    """(a, 1 - a, log of d a / d g): the slope is taken through its logarithm."""
    g = g.double()
    if form == "decay":
        return g, 1.0 - g, torch.zeros_like(g)
    if form == "log":
        return g.exp(), -g.expm1(), g
    log_up, log_down = torch.nn.functional.logsigmoid(g), torch.nn.functional.logsigmoid(-g)
    return log_up.exp(), log_down.exp(), log_up + log_down


def exact(case, seed):
    if case["op"] == "pages":
        return None  # whole numbers
    s = prepare(case, seed)
    c = s["case"]
    if c["op"] in ("grouped", "grouped_grad"):
        return _grouped_exact(s, c)
    a, rest, log_slope = _gate_exact(s["gate"], c["form"])
    if c["op"] != "scan_grad":
        b = s["x"].double() * rest if c["mix"] else s["x"].double()
    del rest
    if c["op"] == "step":
        state, y = s["state"].double(), torch.zeros_like(b)
        for t, slot in enumerate(range(c["tokens"]) if s["slots"] is None else s["slots"].tolist()):
            if slot >= 0:
                torch.addcmul(b[t], a[t], state[slot], out=state[slot])
                y[t] = state[slot]
        return y, state
    at = s["offsets"].tolist()
    zero = torch.zeros((c["sequences"], c["dim"]), dtype=torch.float64, device="cuda")
    initial = zero if s["initial"] is None else s["initial"].double()
    if c["op"] == "scan":
        final = initial.clone()
        for i in range(c["sequences"]):
            h = initial[i]
            for t in range(at[i], at[i + 1]):
                h = torch.addcmul(b[t], a[t], h, out=b[t])
            final[i] = h
        return b, final
    total, dinitial = s["dh"].double(), s["dfinal"].double()
    before = torch.zeros_like(total)
    for i in range(c["sequences"]):
        if at[i + 1] > at[i]:
            before[at[i]] = initial[i]
            before[at[i] + 1:at[i + 1]] = s["h"][at[i]:at[i + 1] - 1].double()
            total[at[i + 1] - 1] += dinitial[i]
            for t in range(at[i + 1] - 2, at[i] - 1, -1):
                total[t].addcmul_(a[t + 1], total[t + 1])
            dinitial[i] = total[at[i]] * a[at[i]]
    del a
    if c["mix"]:
        before -= s["x"].double()
    dgate = before.mul_(total).mul_(log_slope.exp_())
    return dgate, total * _gate_exact(s["gate"], c["form"])[1] if c["mix"] else total, dinitial


def _grouped_exact(s, c):
    offsets, n = s["offsets"].long(), s["offsets"][-1].item()
    row = torch.arange(n, device="cuda")
    expert = torch.searchsorted(offsets[1:], row, right=True)
    token = row if s["index"] is None else s["index"][:n].long() // c["top_k"]
    there = token < s["x"].shape[0]
    if c["op"] == "grouped":
        y = s["y"].double()
    else:
        y = torch.zeros((c["experts"], c["rows"], c["cols"]), dtype=torch.float64, device="cuda")
        if c["add"]:
            y += s["dw"]
    for e in range(c["experts"]):
        mine = row[(expert == e) & there]
        if mine.numel() == 0:
            continue
        x = s["x"][token[mine]].double()
        if c["op"] == "grouped_grad":
            y[e].addmm_(s["dy"][mine].double().T.contiguous(), x)
        else:
            w = s["w"][e].double()
            y[mine] = torch.mm(x, w if c["transposed"] else w.T.contiguous())
    return y
