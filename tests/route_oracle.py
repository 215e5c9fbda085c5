"""The router's weights for given choices, and their gradient, in 64 bits on the host (numpy): relative to the largest
chosen logit, so that no distance between logits loses them, and over the experts that can be chosen with the bias.

The gradient comes from the derivatives of the logarithms of the scores: with D[j, b] = d log p_j / d l_b, a weight that
is a score has d w_j / d l_b = w_j D[j, b], one that is a share of the chosen scores w_j (D[j, b] - sum_i w_i D[i, b])."""
from __future__ import annotations

import numpy as np

from model_oracle import U, rounding


def can_choose(logits32: np.ndarray, bias32) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        s = logits32 if bias32 is None else (logits32 + bias32).astype(np.float32)
    return s > -np.inf  # False for NaN


def log_scores(logits: np.ndarray, can: np.ndarray, score: str) -> np.ndarray:
    """Logarithm of every expert's score, -inf where it cannot be chosen."""
    l = np.where(can, logits, 0.0)
    if score == "sigmoid":
        return np.where(can, -np.logaddexp(0.0, -l), -np.inf)
    top = np.where(can, l, -np.inf).max(1, keepdims=True)
    top = np.where(np.isfinite(top), top, 0.0)
    total = np.where(can, np.exp(l - top), 0.0).sum(1, keepdims=True)
    return np.where(can, l - top - np.log(np.maximum(total, 1e-300)), -np.inf)


# The logarithm below which a score is 0 in 32 bits: half the smallest number, 2^-150.
LOG_NONE = -150 * np.log(2.0)


def weights_and_grad(logits32: np.ndarray, bias32, ids: np.ndarray, dw: np.ndarray, score: str, renorm: bool,
                     scale: float):
    """(weights, gradient, size of the terms that the gradient is made of, spread of the chosen logits per token)."""
    T, E = logits32.shape
    logits, can = logits32.astype(np.float64), can_choose(logits32, bias32)
    lp = log_scores(logits, can, score)
    w, grad, size, spread = np.zeros(ids.shape), np.zeros((T, E)), np.zeros((T, E)), np.zeros(T)
    for t in range(T):
        live = [j for j, e in enumerate(ids[t]) if 0 <= e < E and can[t, e]]
        if not live:
            continue
        at = ids[t, live]
        most = logits[t, at].max()
        spread[t] = (most - logits[t, at]).max()
        if renorm:
            if score == "sigmoid" and lp[t, at].max() < LOG_NONE:
                continue
            # softmax scores share a factor, and a share does not see it: the logits stand for them
            p = np.exp((logits if score == "softmax" else lp)[t, at] - (most if score == "softmax" else lp[t, at].max()))
            p = p / p.sum()
        else:
            p = np.exp(lp[t, at])
        w[t, live] = p * scale
        D = np.zeros((len(live), E))
        D[np.arange(len(live)), at] = 1.0
        if score == "sigmoid":
            D *= np.exp(-np.logaddexp(0.0, np.where(can[t], logits[t], 0.0)))  # 1 - sigmoid
        elif not renorm:
            D -= np.exp(lp[t])
        if renorm:
            D = D - p @ D
        grad[t] = (dw[t, live] * p * scale) @ D
        largest = np.abs(dw[t, live]).max() * abs(scale)
        if renorm or score == "sigmoid":
            np.add.at(size[t], at, p * largest)
        else:
            size[t] = np.exp(lp[t]) * largest * len(live)
    return w, grad, size, spread


def grad_bound(grad, size, spread, ids, dtype, renorm: bool, score: str):
    """With k choices and a spread R of the chosen logits, in units of U: a chosen score is off by R (its difference
    from the largest) + 4 (the exponential), the sum of scores by that and k, a share by 2 R + k + 10; the products with
    dw, their sum and the difference from it by as much again, twice; 26 more for the sigmoid's factor. Without
    renormalising, a softmax score is off by the experts' sum too, and its element's own distance from the largest."""
    k, e = ids.shape[1], grad.shape[1]
    steps = 6 * spread[:, None] + 4 * k + 64
    if not renorm and score == "softmax":
        steps = steps + 2 * e + 4 * 128  # distances up to 128: below that a score is no normal number
    return steps * U * size + rounding(grad, dtype)
