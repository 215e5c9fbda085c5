"""The operators on ragged batches in 64 bits, on the CPU, with bounds on what 32-bit sums may be off.

u = 2^-24 is the largest relative error of one rounding to 32 bits. Each bound is to first order, doubled where a split
into chunks adds a composition for every step (a chunk's product of gates, and the state joined to it)."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step of rounding
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}  # of subnormal results


def rounded(err, ref, dtype):
    """The bound err of a 32-bit value, with its rounding to dtype on the way out."""
    return err + STEP[dtype] * (ref.abs() + err) + TINY[dtype]


def gates(g, form):
    """(a, 1 - a, d a / d g, relative error of the smaller of a and 1 - a in 32 bits). The exponential is taken of
    |g| log2(e), whose rounding and constant's are |g| u each, at 1 ulp, and a sum, a reciprocal (1 ulp) and a product
    follow; the logarithmic form's series has ten terms of decreasing size, 4 u in all, and its product. An exponential
    below 2^-126, the smallest normal number of 32 bits, may come out as 0: all of it is off then (a state moves by at
    most 2^-126 of itself for that)."""
    g = g.double()
    if form == "decay":
        return g, 1 - g, torch.ones_like(g), torch.zeros_like(g)
    off = (2 * torch.nan_to_num(g.abs(), posinf=0.0) + 8) * U
    small = torch.exp(g if form == "log" else -g.abs())
    off = torch.where((small > 0) & (small < 2.0 ** -125.9), 1.0, off)
    if form == "log":
        return g.exp(), -torch.expm1(g), g.exp(), off
    up, down = 1 / (1 + torch.exp(-g)), 1 / (1 + torch.exp(g))
    return up, down, up * down, off


def ranges(offsets, tokens):
    return [(0, tokens)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))


def scan(gate, x, offsets, form, mix, initial):
    """(h, final, bound of h, bound of final): a step's error is the gate's, on the part of the state that it moves, and
    its two roundings, each at most u times E, the recurrence of the terms' magnitudes."""
    a, rest, _, off = gates(gate, form)
    x = x.double()
    b = rest * x if mix else x
    h, err = torch.full_like(b, float("nan")), torch.zeros_like(b)
    spans = ranges(offsets, len(x))
    final = torch.zeros((len(spans), x.shape[1]), dtype=torch.float64) if initial is None else initial.double().clone()
    ferr = torch.zeros_like(final)
    for s, (lo, hi) in enumerate(spans):
        state, size, e = final[s].clone(), final[s].abs(), torch.zeros(x.shape[1], dtype=torch.float64)
        for t in range(lo, hi):
            size = a[t].abs() * size + b[t].abs()
            e = a[t].abs() * e + 2 * (off[t] + 4 * U) * size
            state = a[t] * state + b[t]
            h[t], err[t] = state, e
        final[s], ferr[s] = state, e
    return h, final, err, ferr


def scan_grad(gate, h, dh, x, offsets, form, mix, initial, dfinal):
    """((dgate, dx, dinitial), their bounds): the reverse recurrence's as above, then the products' relative errors."""
    a, rest, slope, off = gates(gate, form)
    h, dh = h.double(), dh.double()
    spans = ranges(offsets, len(h))
    n, d = h.shape
    zero = torch.zeros((len(spans), d), dtype=torch.float64)
    initial = zero if initial is None else initial.double()
    dinitial = zero.clone() if dfinal is None else dfinal.double().clone()
    out = [torch.full_like(h, float("nan")) for _ in range(2)]
    err = [torch.zeros_like(h) for _ in range(2)] + [zero.clone()]
    for s, (lo, hi) in enumerate(spans):
        total, size, e = dinitial[s].clone(), dinitial[s].abs(), torch.zeros(d, dtype=torch.float64)
        for t in range(hi - 1, lo - 1, -1):
            total, size = total + dh[t], size + dh[t].abs()
            e = e + 2 * U * size
            before = h[t - 1] if t > lo else initial[s]
            if mix:
                before = before - x[t].double()
            r = rest[t] if mix else torch.ones(d, dtype=torch.float64)
            out[0][t], out[1][t] = total * before * slope[t], total * r
            err[0][t] = e * (before * slope[t]).abs() + (2 * off[t] + 8 * U) * out[0][t].abs()
            err[1][t] = e * r.abs() + (off[t] + 3 * U) * out[1][t].abs()
            e = a[t].abs() * e + 2 * (off[t] + 4 * U) * a[t].abs() * size
            total, size = a[t] * total, a[t].abs() * size
        dinitial[s], err[2][s] = total, e
    return (*out, dinitial), err


def step(gate, x, state, slots, form, mix):
    """(h, state, bounds) of one token a row, rows of one slot in order."""
    state = state.double().clone()
    h, he, se = torch.zeros(x.shape, dtype=torch.float64), torch.zeros(x.shape, dtype=torch.float64), torch.zeros_like(state)
    a, rest, _, off = gates(gate, form)
    b = rest * x.double() if mix else x.double()
    for i in range(len(x)):
        k = i if slots is None else int(slots[i])
        if 0 <= k < len(state):
            size = a[i].abs() * state[k].abs() + b[i].abs()
            state[k] = a[i] * state[k] + b[i]
            se[k] = a[i].abs() * se[k] + (off[i] + 4 * U) * size
            h[i], he[i] = state[k], se[k]
    return h, state, he, se


def batch(x, index, top_k):
    if index is None:
        return x.double()
    rows = torch.zeros((len(index), x.shape[1]), dtype=torch.float64)
    for r, i in enumerate(index.tolist()):
        if i >= 0 and i // top_k < len(x):
            rows[r] = x[i // top_k].double()
    return rows


def grouped(x, w, offsets, index, top_k, transposed):
    """(y, bound; NaN in rows outside the groups): a sum of n products in 32 bits, each addition at most 2 u off."""
    rows, w = batch(x, index, top_k), w.double()
    if not transposed:
        w = w.transpose(1, 2)
    y = torch.full((len(rows), w.shape[2]), float("nan"), dtype=torch.float64)
    size = torch.zeros_like(y)
    for e in range(len(w)):
        lo, hi = offsets[e], offsets[e + 1]
        y[lo:hi], size[lo:hi] = rows[lo:hi] @ w[e], rows[lo:hi].abs() @ w[e].abs()
    return y, 2 * U * (w.shape[1] + 2) * size


def grouped_grad(dy, x, offsets, index, top_k, old):
    rows, dy = batch(x, index, top_k), dy.double()
    n = len(offsets) - 1
    dw = torch.zeros((n, dy.shape[1], x.shape[1]), dtype=torch.float64)
    size = torch.zeros_like(dw)
    for e in range(n):
        lo, hi = offsets[e], offsets[e + 1]
        dw[e], size[e] = dy[lo:hi].T @ rows[lo:hi], dy[lo:hi].T.abs() @ rows[lo:hi].abs() * (hi - lo + 2)
    if old is not None:
        dw, size = dw + old.double(), size + old.double().abs()
    return dw, 2 * U * size


def pages(context, new, tables, free, count, page, tokens):
    """(offsets, slots, positions, left, tables), request by request and token by token."""
    tables = tables.copy()
    count = min(max(int(count), 0), len(free))
    offsets, slots, positions, taken = [0], [], [], 0
    for r, (c, n) in enumerate(zip(np.maximum(context, 0).tolist(), np.maximum(new, 0).tolist())):
        held = -(-c // page)
        for col in range(held, -(-(c + n) // page)):
            if col < tables.shape[1]:
                tables[r, col] = free[count - 1 - taken] if taken < count else -1
            taken += 1
        for p in range(c, c + n):
            at = tables[r, p // page] if p // page < tables.shape[1] else -1
            slots.append(int(at) * page + p % page if at >= 0 else -1)
            positions.append(p)
        offsets.append(offsets[-1] + n)
    slots, positions = slots[:tokens], positions[:tokens]
    slots += [-1] * (tokens - len(slots))
    positions += [0] * (tokens - len(positions))
    return np.array(offsets), np.array(slots, dtype=np.int64), np.array(positions), count - taken, tables
