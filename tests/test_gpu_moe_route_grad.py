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
