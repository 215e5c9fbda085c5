"""The example's decoding and training step: the operators together, against the definitions in 64 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import model_oracle as mo
import primitives_device_scan_amd as ds

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "moe_block.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_decode_step(example):
    block = example.Block(rows=500, dim=192, hidden=96, experts=12, top_k=3, seed=5)
    ids = torch.from_numpy(np.random.default_rng(5).integers(-1, 500, 37)).cuda()
    x, logits, weights, chosen, y = example.decode_step(block, ids)
    # each operator against its definition on the inputs it had
    live = (ids >= 0)[:, None]
    want = torch.where(live, block.table[ids.clamp(min=0)].float() * block.scale, 0.0).to(x.dtype)
    assert torch.equal(x, want)
    rw, rids = mo.route(logits, None, 3, "softmax", True, 1.0)
    assert np.array_equal(chosen.cpu().numpy(), rids)
    mo.within(weights, rw, mo.route_terms(logits) * mo.U * np.abs(rw) + 2.0 ** -120, "weights")
    ref, bound = mo.experts(x, block.w_in, block.w_out, chosen, weights)
    mo.within(y, ref, bound, "experts")


def test_train_steps_accumulate(example):
    block = example.Block(rows=300, dim=64, hidden=32, experts=10, top_k=3, dtype=torch.float32, seed=6)
    rng = np.random.default_rng(6)
    want_t, want_r = np.zeros((300, 64)), np.zeros((64, 10))
    table, router = mo.f64(block.table), mo.f64(block.router)
    size_t, size_r = np.zeros_like(want_t), np.zeros_like(want_r)
    for _ in range(3):
        ids = torch.from_numpy(rng.integers(0, 300, 400))
        wg = torch.from_numpy(rng.normal(size=(400, 3)).astype(np.float32))
        chosen = example.train_step(block, ids.cuda(), wg.cuda()).cpu().numpy()
        x = table[ids.numpy()] * block.scale
        d, size = mo.route_grad(x @ router, chosen, mo.f64(wg), "softmax", True, 1.0)
        want_r += x.T @ d
        size_r += np.abs(x).T @ size
        np.add.at(want_t, ids.numpy(), block.scale * (d @ router.T))
        np.add.at(size_t, ids.numpy(), block.scale * (size @ np.abs(router).T))
    # the logits' own 32-bit sums of 64 terms (a product of that size is off by 64 U |x| |w|, which moves a score by as
    # much, relatively), the router's gradient (route_terms), sums of 400 x 3 and of 10 terms: 2^12 U covers their sum
    steps = 2.0 ** 12 * mo.U
    mo.within(block.router_grad, want_r, steps * size_r + 2.0 ** -120, "router")
    mo.within(block.table_grad, want_t, steps * size_t + 2.0 ** -120, "table")


def test_smallest_step(example):
    block = example.Block(rows=5, dim=8, hidden=4, experts=2, top_k=1, seed=7)
    y = example.decode_step(block, torch.tensor([3]).cuda())[-1]
    assert y.shape == (1, 8) and bool(torch.isfinite(y.float()).all())
    empty = example.decode_step(block, torch.zeros(0, dtype=torch.int64).cuda())
    assert empty[-1].shape == (0, 8) and ds.query_timeout() == 0
