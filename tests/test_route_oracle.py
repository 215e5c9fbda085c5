"""The 64-bit definition of the router's weights and their gradient (tests/route_oracle.py), held to differences, to a
hand-worked token and to the other definition (tests/model_oracle.py) where logits lie near each other (CPU only)."""
import numpy as np
import pytest
import torch

import model_oracle as mo
import route_oracle as ro


def case(seed, tokens=5, experts=11, top_k=4):
    rng = np.random.default_rng(seed)
    l = rng.normal(size=(tokens, experts)).astype(np.float32)
    l[1, 3] = -np.inf
    ids = np.argsort(-l, axis=1)[:, :top_k]
    ids[2, 1], ids[3, 2] = -1, ids[3, 0]
    return l, ids, rng.normal(size=(tokens, top_k))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_equals_the_other_definition(score, renorm):
    l, ids, dw = case(1)
    w, grad, _, _ = ro.weights_and_grad(l, None, ids, dw, score, renorm, 2.5)
    ref, _ = mo.route_grad(l.astype(np.float64), ids, dw, score, renorm, 2.5)
    assert np.abs(grad - ref).max() < 1e-14
    rw, rids = mo.route(torch.from_numpy(l), None, 4, score, renorm, 2.5)
    w, _, _, _ = ro.weights_and_grad(l, None, rids, dw, score, renorm, 2.5)
    assert np.abs(w - rw).max() < 1e-14


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("distance", [0.0, 300.0])
def test_against_differences(score, renorm, distance):
    # weights by themselves, in steps that 32-bit logits hold; experts 2, 5, 8 switched off by the bias
    l, ids, dw = case(2)
    ids[0] = [0, 1, 3, 4]
    l[:, 6:] += np.float32(distance)
    l = np.round(l * 64) / np.float32(64)
    bias = np.zeros(11, np.float32)
    bias[2::3] = [-np.inf, np.nan, -np.inf]
    _, grad, size, _ = ro.weights_and_grad(l, bias, ids, dw, score, renorm, 1.5)
    step = np.float32(2.0 ** -12)
    for e in range(11):
        up, down = l.copy(), l.copy()
        up[:, e] += step
        down[:, e] -= step
        loss = [(ro.weights_and_grad(x, bias, ids, dw, score, renorm, 1.5)[0] * dw).sum(1) for x in (up, down)]
        assert np.abs((loss[0] - loss[1]) / (2 * step) - grad[:, e]).max() < 1e-6
        assert np.isfinite(bias[e]) or not grad[:, e].any()


def test_far_logits_by_hand():
    l = np.array([[90.0, 0.0, 0.5]], np.float32)
    for d in (0.0, 2000.0):
        l[0, 0] = 90 + d
        w, grad, _, _ = ro.weights_and_grad(l, None, np.array([[1, 2]]), np.array([[1.0, -1.0]]), "softmax", True, 1.0)
        p = 1 / (1 + np.exp(0.5))
        assert np.abs(w - [[p, 1 - p]]).max() < 1e-15
        assert np.abs(grad - [[0, 2 * p * (1 - p), -2 * p * (1 - p)]]).max() < 1e-15
