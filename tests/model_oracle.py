"""The language-model operators in 64 bits on the host (numpy), from their definitions, and bounds on how far 32-bit
sums and one rounding of the output may be from them.

U = 2^-24 is half a step of a 32-bit float. A sum of c terms in 32 bits, in any
order, is within c * U * sum |terms| of the exact one to first order; twice that is allowed, which covers the second
order and the matrix cores' own order of additions."""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -24}


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def rounding(ref: np.ndarray, dtype) -> np.ndarray:
    """Half a step of dtype at ref, and half its smallest step near 0."""
    return torch.finfo(dtype).eps / 2 * np.abs(ref) + TINY[dtype]


def embedding_grad(dout: np.ndarray, ids: np.ndarray, rows: int, scale: float, old=None):
    """(gradient, count of terms per row, sum of |terms| per element)."""
    g = np.zeros((rows, dout.shape[1]))
    s = np.zeros_like(g)
    c = np.zeros(rows)
    for i, v in enumerate(ids):
        if 0 <= v < rows:
            g[v] += dout[i]
            s[v] += np.abs(dout[i])
            c[v] += 1
    g, s = g * scale, s * abs(scale)
    if old is not None:
        g, s = g + old, s + np.abs(old)
    return g, c, s


def embedding_grad_bound(g, c, s, dtype):
    # c additions, the scaling and the addition to the old value
    return 2 * (c[:, None] + 2) * U * s + rounding(g, dtype)


def scores(logits: np.ndarray, can: np.ndarray, score: str) -> np.ndarray:
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(can, 1 / (1 + np.exp(-np.where(can, logits, 0.0))), 0.0)
    l = np.where(can, logits, -np.inf)
    top = l.max(1, keepdims=True)
    e = np.where(can, np.exp(np.where(can, l, 0.0) - np.where(np.isfinite(top), top, 0.0)), 0.0)
    return e / np.maximum(e.sum(1, keepdims=True), 1e-300)


def route(logits: torch.Tensor, bias, top_k: int, score: str, renorm: bool, scale: float):
    l32 = logits.detach().cpu().float().numpy()
    sel = l32 if bias is None else (l32 + bias.detach().cpu().numpy()).astype(np.float32)
    can = sel > -np.inf  # False for NaN
    key = np.where(can, sel, -np.inf)
    order = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    ids = np.where(np.take_along_axis(can, order, 1), order, -1)
    p = scores(l32.astype(np.float64), can, score)
    w = np.where(ids >= 0, np.take_along_axis(p, np.maximum(ids, 0), 1), 0.0)
    if renorm:
        t = w.sum(1, keepdims=True)
        w = w / np.where(t > 0, t, 1.0)
    return w * scale, ids.astype(np.int32)


def logit_range(logits: torch.Tensor) -> float:
    l = f64(logits)
    l = l[np.isfinite(l)]
    return float(np.abs(l).max()) if l.size else 0.0


def route_terms(logits: torch.Tensor) -> float:
    """Steps U that a score may be off by, relative: the exponent's argument is off by U times its size (at most twice
    the largest logit), the sum has one addition per expert; 16 for the exponentials, divisions and the scale."""
    return 2 * (logits.shape[1] + 2 * logit_range(logits) + 16)


def route_grad(logits: np.ndarray, ids: np.ndarray, dw: np.ndarray, score: str, renorm: bool, scale: float):
    """(gradient, scale of the terms it is made of) token by token, from the Jacobian of the weights."""
    T, E = logits.shape
    can = logits > -np.inf
    p = scores(logits, can, score)
    out, size = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        if score == "softmax":
            dp = np.diag(p[t]) - np.outer(p[t], p[t])  # d p_a / d l_b
        else:
            dp = np.diag(p[t] * (1 - p[t]))
        live = [(j, int(e)) for j, e in enumerate(ids[t]) if 0 <= e < E]
        total = sum(p[t, e] for _, e in live) if renorm else 1.0
        total = total if total > 0 else 1.0
        most = max([abs(dw[t, j]) for j, _ in live], default=0.0) * abs(scale)
        for j, e in live:
            g = dp[e].copy()
            if renorm:
                g = g / total - p[t, e] / total ** 2 * sum(dp[f] for _, f in live)
            out[t] += g * dw[t, j] * scale
        size[t] = p[t] * most * (2 + 2 * len(live)) / (total if renorm else 1.0)
    return out, size


def silu(g):
    return g / (1 + np.exp(-g))


def widen(w: torch.Tensor, scale) -> np.ndarray:
    w = f64(w.float())
    if scale is None:
        return w
    s = f64(scale)
    return w * np.repeat(np.repeat(s, 128, 1)[:, :w.shape[1]], 128, 2)[:, :, :w.shape[2]]


def experts(x: torch.Tensor, w_in, w_out, ids, weights, s_in=None, s_out=None):
    """(y, bound on its error). The bound follows the errors through: gate and up are 32-bit sums, h is rounded to x's
    type, the down products are 32-bit sums, as is the sum over the choices, and y is rounded once."""
    dtype = x.dtype
    half = torch.finfo(dtype).eps / 2
    X, WI, WO = f64(x), widen(w_in, s_in), widen(w_out, s_out)
    ids, wt = ids.cpu().numpy(), f64(weights)
    T, D = X.shape
    F = WI.shape[1] // 2
    y, err = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if not 0 <= e < WI.shape[0]:
                continue
            v, ev = WI[e] @ X[t], 2 * (D + 4) * U * (np.abs(WI[e]) @ np.abs(X[t]))
            g, u, eg, eu = v[:F], v[F:], ev[:F], ev[F:]
            h = silu(g) * u
            eh = 1.1 * eg * np.abs(u) + np.abs(silu(g)) * eu + 1.1 * eg * eu + (half + (8 + np.abs(g)) * U) * np.abs(h) + TINY[dtype]
            z, ez = WO[e] @ h, np.abs(WO[e]) @ eh
            ez = ez + 2 * (F + 4) * U * (np.abs(WO[e]) @ (np.abs(h) + eh))
            y[t] += wt[t, j] * z
            err[t] += np.abs(wt[t, j]) * (ez + 2 * (ids.shape[1] + 2) * U * np.abs(z))
    return y, err + half * (np.abs(y) + err) + TINY[dtype]


def within(got: torch.Tensor, ref: np.ndarray, bound: np.ndarray, what: str):
    g = f64(got)
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    off = np.abs(g - ref)
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: got {g[i]} "
                             f"want {ref[i]} off {off[i]:.3e} allowed {bound[i]:.3e}")
    return float((off / np.maximum(bound, 1e-300)).max()) if off.size else 0.0


