"""The router's gradient against the weights that the router itself returned: logits that lie far apart, and experts that
the bias switches off. Definitions and bounds: tests/route_oracle.py."""
import numpy as np
import pytest
import torch

import model_oracle as mo
import route_oracle as ro
import primitives_device_scan_amd as ds
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def normal(seed, shape, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def f32(t):
    return None if t is None else t.detach().cpu().float().numpy()


def check(l, ids, score, renorm, scale, bias=None, what=""):
    """Weights (where ids are the router's own) and gradient for the ids given."""
    dw = normal(l.shape[0] + ids.shape[1], tuple(ids.shape))
    more = {} if bias is None else {"bias": bias.cuda()}
    got = ds.moe_route_grad(l.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, scale=scale, **more)
    n = ids.cpu().numpy()
    w, ref, size, spread = ro.weights_and_grad(f32(l), f32(bias), n, mo.f64(dw), score, renorm, float(np.float32(scale)))
    worst = mo.within(got, ref, ro.grad_bound(ref, size, spread, n, l.dtype, renorm, score), what)
    say(what, l.dtype, score, renorm, "worst share of the bound %.2f" % worst)
    return got, w


def test_renormalised_gradient_of_a_hand_worked_token():
    # weights 1 / (1 + e^0.5) and its rest, 0.378 and 0.622; their product is 0.235
    l = torch.tensor([[90.0, 0.0, 0.5]])
    got = ds.moe_route_grad(l.cuda(), torch.tensor([[1, 2]], dtype=torch.int32).cuda(), torch.tensor([[1.0, -1.0]]).cuda())
    p = 1 / (1 + np.exp(0.5))
    assert np.abs(mo.f64(got) - [[0.0, 2 * p * (1 - p), -2 * p * (1 - p)]]).max() <= 16 * mo.U


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("distance", [0.0, 50.0, 100.0, 1000.0])
@pytest.mark.parametrize("tokens,experts,top_k", [(3, 5, 2), (9, 64, 6), (5, 100, 64), (40, 256, 8), (3, 511, 5)])
def test_renormalised_gradient_far_below_the_largest_logit(dtype, distance, tokens, experts, top_k):
    # the choice is the caller's (a bias makes it): the last experts, `distance` below the others
    l = normal(tokens + experts, (tokens, experts))
    l[:, :experts - top_k] += distance
    l = l.to(dtype)
    ids = torch.stack([torch.randperm(top_k, generator=torch.Generator().manual_seed(t)) for t in range(tokens)])
    ids = (ids + experts - top_k).to(torch.int32)
    got, _ = check(l, ids, "softmax", True, 2.5, what=f"{distance} below, {top_k} of {experts}")
    assert not bool(got[:, :experts - top_k].any())   # an expert that was not chosen has no part in the weights


def switched_off(experts, seed=2):
    """A selection bias that takes experts out of the choice."""
    bias = normal(seed, (experts,), std=0.5)
    bias[1::5] = float("-inf")
    bias[3::11] = float("nan")
    return bias


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 2, 1), (33, 60, 4), (9, 64, 6), (40, 128, 8), (21, 256, 8),
                                                  (6, 300, 16), (5, 511, 5)])
def test_weights_and_gradient_agree_with_a_bias(dtype, score, renorm, tokens, experts, top_k):
    # experts that the bias switches off have large logits: they must not be in any sum
    l, bias = normal(tokens + experts, (tokens, experts), std=1.5), switched_off(experts)
    l[:, 1::5] += 20.0
    l[0] = float("-inf")
    l = l.to(dtype)
    w, ids = ds.moe_route(l.cuda(), top_k, score=score, renormalize=renorm, scale=2.5, bias=bias.cuda())
    got, want = check(l, ids.cpu(), score, renorm, 2.5, bias, f"{top_k} of {experts}")
    mo.within(w, want, mo.route_terms(l) * mo.U * np.abs(want) + 2.0 ** -120, "weights")
    off = ~np.isfinite(f32(bias))
    assert not bool(got[:, torch.from_numpy(off)].any()) and not bool(got[0].any())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_choices_that_cannot_be_made_have_no_part(score, renorm):
    # ids that the caller gives: switched off by the bias or by the logit, outside the experts, twice the same
    l, bias = normal(3, (12, 40), std=1.5), switched_off(40)
    l[:, 7] = float("-inf")
    l[:, 8] = float("nan")
    ids = torch.randint(0, 40, (12, 6), generator=torch.Generator().manual_seed(4)).to(torch.int32)
    ids[0], ids[1, :3], ids[2, 2], ids[3, 0] = 1, 7, 8, 40
    ids[4, 1] = ids[4, 0] = 10
    check(l, ids, score, renorm, 1.5, bias, "given ids")
    dw = torch.ones(12, 6)
    dw[(ids == 1) | (ids == 7) | (ids == 8) | (ids == 40)] = float("nan")   # what no weight came from is not looked at
    got = ds.moe_route_grad(l.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, bias=bias.cuda())
    assert not bool(got.isnan().any()) and not bool(got[0].any())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("biased", [False, True])
def test_gradient_against_differences_of_the_router(score, renorm, biased):
    # A symmetric difference of the router's own weights along one direction, at logits far enough apart that the choice
    # stays. Its error: the step's square times a third of the third derivative along the direction (under 20 |d|^3 for
    # these sums of products of scores, |d| the largest part), and the weights' error of route_terms over the step.
    tokens, experts, top_k, step = 16, 40, 5, 2.0 ** -6
    l = torch.stack([torch.randperm(experts, generator=torch.Generator().manual_seed(t)) for t in range(tokens)]) / 8.0
    d = normal(9, (tokens, experts)).clamp(-3, 3)
    bias = None
    if biased:
        bias = torch.zeros(experts)
        bias[2::3] = float("-inf")
    more = {} if bias is None else {"bias": bias.cuda()}
    up, ids = ds.moe_route((l + step * d).cuda(), top_k, score=score, renormalize=renorm, **more)
    down, ids2 = ds.moe_route((l - step * d).cuda(), top_k, score=score, renormalize=renorm, **more)
    at, ids3 = ds.moe_route(l.cuda(), top_k, score=score, renormalize=renorm, **more)
    assert torch.equal(ids, ids2) and torch.equal(ids, ids3)
    dw = normal(10, (tokens, top_k))
    grad = mo.f64(ds.moe_route_grad(l.cuda(), ids, dw.cuda(), score=score, renormalize=renorm, **more))
    moved = mo.f64(l + step * d) - mo.f64(l - step * d)
    slope = ((mo.f64(up) - mo.f64(down)) * mo.f64(dw)).sum(1) / (2 * step)
    most = np.abs(mo.f64(dw)).sum(1)
    bound = 20 * step ** 2 * most * np.abs(mo.f64(d)).max(1) ** 3 + mo.route_terms(l) * mo.U * most / step
    assert bool((np.abs(slope - (grad * moved).sum(1) / (2 * step)) <= bound).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [-80.0, -87.0, -89.0, -95.0, -102.0])
def test_renormalised_sigmoid_scores_of_very_negative_logits(dtype, low):
    # scores down to 2^-149 are numbers of 32 bits, and their shares are held relative to the largest
    l = (low + normal(7, (20, 48)).clamp(-1, 1)).to(dtype)
    w, ids = ds.moe_route(l.cuda(), 6, score="sigmoid", renormalize=True, scale=2.5)
    _, want = check(l, ids.cpu(), "sigmoid", True, 2.5, what=f"sigmoid around {low}")
    mo.within(w, want, mo.route_terms(l) * mo.U * np.abs(want), "weights")
    # below half of that they are 0, and so are the weights and their gradient
    l = torch.full((3, 9), -104.5, dtype=dtype)
    w, ids = ds.moe_route(l.cuda(), 4, score="sigmoid", renormalize=True)
    got = ds.moe_route_grad(l.cuda(), ids, torch.ones_like(w), score="sigmoid", renormalize=True)
    assert ids.tolist() == [[0, 1, 2, 3]] * 3 and not bool(w.any()) and not bool(got.any())


def test_gradient_of_small_scores_keeps_32_bits():
    # Multiples of 1/16: every difference from the largest logit is exact, so only the exponentials (4 steps each way),
    # the sum of 8 scores and 16 products, quotients and differences count: 8 + 2 * 4 + 16 steps, relative. Few choices,
    # the largest expert's: its weight's gradient is p_e (0 - p_0), with p_0 next to 1.
    l = torch.randint(-80 * 16, -20 * 16, (4000, 8), generator=torch.Generator().manual_seed(6)) / 16.0
    l[:, 0] = 0.0
    ids = torch.zeros(4000, 1, dtype=torch.int32)
    got = mo.f64(ds.moe_route_grad(l.cuda(), ids.cuda(), torch.ones(4000, 1).cuda(), renormalize=False))[:, 1:]
    _, ref, _, _ = ro.weights_and_grad(f32(l), None, ids.numpy(), np.ones((4000, 1)), "softmax", False, 1.0)
    worst = (np.abs(got - ref[:, 1:]) / np.abs(ref[:, 1:])).max() / mo.U
    say("small scores: off by %.1f steps" % worst)
    assert worst <= 32


@pytest.mark.parametrize("low", [-20.0, -60.0, -79.0])
def test_large_weight_gradients_of_small_sigmoid_scores(low):
    # the scores' sum is as small as 2^-115: a share, not dw, is divided by it
    l = low + normal(11, (20, 48)).clamp(-1, 1)
    _, ids = ds.moe_route(l.cuda(), 6, score="sigmoid")
    dw = normal(12, (20, 6)) * 2.0 ** 20
    got = ds.moe_route_grad(l.cuda(), ids, dw.cuda(), score="sigmoid")
    n = ids.cpu().numpy()
    _, ref, size, spread = ro.weights_and_grad(f32(l), None, n, mo.f64(dw), "sigmoid", True, 1.0)
    mo.within(got, ref, ro.grad_bound(ref, size, spread, n, l.dtype, True, "sigmoid"), f"around {low}")
