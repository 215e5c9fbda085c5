"""The language-model entry points refuse bad arguments on the host before any HIP call (CPU only), and the 64-bit
definitions that the GPU tests compare with are themselves held to differences and to hand-worked cases."""
import os

import numpy as np
import pytest
import torch

import model_oracle as mo

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INV, DTY, OVL, OOM, HIPERR, MIS, BIG, CAPT = range(9)
F32, BF16, FP16, FP8 = 2, 5, 6, 7
# Fake addresses, never dereferenced, 4 GiB apart.
A, B, C, D, E, F, G, H = (0x7F0000000000 + (i << 32) for i in range(8))


@pytest.fixture(scope="module")
def lib():
    path = os.path.join(ROOT, "primitives_device_scan_amd", "libdevscan.so")
    if not os.path.exists(path):
        import __graft_entry__
        __graft_entry__.build()
    from primitives_device_scan_amd import _binding
    return _binding.load_library(path)


def test_embedding_refusals(lib):
    def f(dtype=F32, table=A, rows=100, dim=8, ts=8, ids=B, idb=4, n=10, out=C, os_=8):
        return lib.ds_embedding(dtype, table, rows, dim, ts, ids, idb, n, 1.0, out, os_, None)
    assert f(dtype=0) == DTY and f(dtype=FP8) == DTY and f(dtype=-1) == DTY and f(dtype=3) == DTY
    assert f(rows=-1) == INV and f(dim=-1) == INV and f(n=-1) == INV and f(idb=2) == INV
    assert f(ts=7) == INV and f(os_=7) == INV                     # rows that overlap
    assert f(table=None) == INV and f(ids=None) == INV and f(out=None) == INV
    assert f(n=0, table=None, ids=None, out=None) == OK and f(dim=0, ts=0, os_=0, table=None, out=None) == OK
    assert f(table=A + 2) == MIS and f(out=C + 2) == MIS and f(ids=B + 2) == MIS and f(ids=B + 4, idb=8) == MIS
    assert f(out=A + 32) == OVL and f(out=B + 8) == OVL
    assert f(n=1 << 41) == BIG
    assert f(n=1 << 39, out=C, os_=1 << 30) == BIG                # past any address


def test_embedding_grad_refusals(lib):
    def f(dtype=BF16, dout=A, ds=8, ids=B, idb=4, n=10, gd=F32, grad=C, rows=100, dim=8, gs=8, acc=0):
        return lib.ds_embedding_grad(dtype, dout, ds, ids, idb, n, 1.0, gd, grad, rows, dim, gs, acc, None)
    assert f(dtype=1) == DTY and f(gd=FP16) == DTY and f(dtype=F32, gd=BF16) == DTY and f(gd=0) == DTY
    assert f(rows=-1) == INV and f(dim=-1) == INV and f(n=-1) == INV and f(idb=3) == INV and f(acc=2) == INV
    assert f(ds=7) == INV and f(gs=7) == INV
    assert f(dout=None) == INV and f(ids=None) == INV and f(grad=None) == INV
    assert f(rows=0, grad=None) == OK and f(dim=0, ds=0, gs=0) == OK and f(n=0, acc=1) == OK
    assert f(dout=A + 1) == MIS and f(grad=C + 2) == MIS and f(ids=B + 2) == MIS
    assert f(grad=A + 16) == OVL and f(grad=B) == OVL
    assert f(n=1 << 31) == BIG and f(rows=1 << 27) == BIG


def test_moe_route_refusals(lib):
    def f(dtype=F32, logits=A, t=10, e=16, stride=16, bias=B, k=2, score=0, renorm=1, w=C, ids=D):
        return lib.ds_moe_route(dtype, logits, t, e, stride, bias, k, score, renorm, 1.0, w, ids, None)
    assert f(dtype=0) == DTY and f(dtype=FP8) == DTY
    assert f(t=-1) == INV and f(e=0) == INV and f(e=512, stride=512) == INV and f(stride=15) == INV
    assert f(k=0) == INV and f(k=17) == INV and f(e=100, stride=100, k=65) == INV
    assert f(score=2) == INV and f(score=-1) == INV and f(renorm=2) == INV
    assert f(logits=None) == INV and f(w=None) == INV and f(ids=None) == INV
    assert f(t=0, logits=None, w=None, ids=None) == OK
    assert f(logits=A + 2) == MIS and f(bias=B + 2) == MIS and f(w=C + 2) == MIS
    assert f(w=A + 64) == OVL and f(ids=C + 16) == OVL and f(ids=B) == OVL
    assert f(t=1 << 40) == BIG


def test_moe_route_grad_refusals(lib):
    def f(dtype=F32, logits=A, t=10, e=16, stride=16, ids=B, dw=C, k=2, score=0, renorm=1, dl=D, dls=16):
        return lib.ds_moe_route_grad(dtype, logits, t, e, stride, ids, dw, k, score, renorm, 1.0, dl, dls, None)
    assert f(dtype=1) == DTY
    assert f(t=-1) == INV and f(e=0) == INV and f(k=0) == INV and f(dls=15) == INV and f(score=3) == INV
    assert f(ids=None) == INV and f(dw=None) == INV and f(dl=None) == INV
    assert f(t=0, logits=None) == OK
    assert f(dl=D + 2) == MIS
    assert f(dl=A) == OVL and f(dl=C + 8) == OVL
    assert f(t=1 << 40) == BIG


def test_moe_experts_refusals(lib):
    def f(dtype=BF16, x=A, t=4, dim=64, xs=64, wd=BF16, wi=B, si=None, wo=C, so=None, e=8, hid=32, ids=D, w=E, k=2,
          y=F, ys=64):
        return lib.ds_moe_experts(dtype, x, t, dim, xs, wd, wi, si, wo, so, e, hid, ids, w, k, y, ys, None)
    assert f(dtype=F32, wd=F32) == DTY and f(wd=FP16) == DTY and f(dtype=FP16) == DTY and f(dtype=FP8, wd=FP8) == DTY
    assert f(t=-1) == INV and f(dim=0) == INV and f(hid=0) == INV and f(e=0) == INV and f(k=0) == INV
    assert f(e=8193) == INV and f(xs=63) == INV and f(ys=63) == INV
    assert f(t=0, x=None, y=None, ids=None, w=None) == OK
    for name in ("x", "wi", "wo", "ids", "w", "y"):
        assert f(**{name: None}) == INV, name
    assert f(wd=FP8) == INV and f(wd=FP8, si=G) == INV            # 8-bit weights without their scales
    assert f(x=A + 1) == MIS and f(wi=B + 1) == MIS and f(w=E + 2) == MIS and f(wd=FP8, si=G + 2, so=H) == MIS
    assert f(y=A) == OVL and f(y=B + 64) == OVL and f(y=D) == OVL
    assert f(t=4097) == BIG and f(t=1 << 62) == BIG and f(dim=(1 << 20) + 1, xs=1 << 21, ys=1 << 21) == BIG


def test_other_entry_points_refuse_the_new_types(lib):
    for t in (BF16, FP16, FP8):
        assert lib.scan_exclusive(t, A, B, 10, None) == DTY
        assert lib.compact_if(t, A, B, C, 10, 0, 0, None) == DTY


def test_binding_refuses_host_tensors_and_wrong_types():
    import primitives_device_scan_amd as ds
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        ds.embedding(x, ids)
    with pytest.raises(TypeError):
        ds.embedding(x.double(), ids)
    with pytest.raises(ValueError):
        ds.embedding_grad(x, ids, 10)
    with pytest.raises(ValueError):
        ds.moe_route(x, 2)
    with pytest.raises(ValueError):
        ds.moe_route_grad(x, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(TypeError):
        ds.moe_experts(x, x, x, ids, x)
    with pytest.raises(ValueError):
        ds.moe_experts(x.bfloat16(), x[None].bfloat16(), x[None].bfloat16(), ids[:, None], x)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_oracle_route_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(3)
    T, E, k, scale = 3, 7, 3, 2.5
    l = torch.from_numpy(rng.normal(size=(T, E)).astype(np.float32))
    l[0, 2] = float("-inf")
    dw = rng.normal(size=(T, k))
    _, ids = mo.route(l, None, k, score, renorm, scale)
    grad, _ = mo.route_grad(mo.f64(l), ids, dw, score, renorm, scale)

    def loss(x):
        p = mo.scores(x, x > -np.inf, score)
        w = np.take_along_axis(p, ids.astype(np.int64), 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return float((w * scale * dw).sum())

    step = 1e-5
    for t in range(T):
        for e in range(E):
            if not np.isfinite(mo.f64(l)[t, e]):
                assert grad[t, e] == 0
                continue
            up, down = mo.f64(l).copy(), mo.f64(l).copy()
            up[t, e] += step
            down[t, e] -= step
            assert abs((loss(up) - loss(down)) / (2 * step) - grad[t, e]) < 1e-8


def test_oracle_hand_worked_cases():
    l = torch.tensor([[1.0, 3.0, 3.0, 2.0], [float("-inf"), float("nan"), 0.0, float("-inf")]])
    w, ids = mo.route(l, None, 2, "softmax", True, 1.0)
    assert ids.tolist() == [[1, 2], [2, -1]] and w.tolist() == [[0.5, 0.5], [1.0, 0.0]]
    w, ids = mo.route(l, torch.tensor([5.0, 0, 0, 0]), 2, "sigmoid", False, 2.0)
    assert ids.tolist() == [[0, 1], [2, -1]] and abs(w[0, 0] - 2 / (1 + np.exp(-1.0))) < 1e-15 and w[1, 0] == 1.0
    g, c, s = mo.embedding_grad(np.array([[1.0], [2.0], [4.0], [8.0]]), np.array([1, -1, 1, 3]), 3, 10.0)
    assert g.tolist() == [[0.0], [50.0], [0.0]] and c.tolist() == [0, 2, 0]
    one = torch.ones(1, 1, dtype=torch.float16)
    y, _ = mo.experts(one, torch.ones(2, 2, 1), torch.ones(2, 1, 1), torch.tensor([[1, 5]]), torch.tensor([[3.0, 9.0]]))
    assert abs(y[0, 0] - 3 / (1 + np.exp(-1.0))) < 1e-15
