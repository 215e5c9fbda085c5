"""The router's gradient with a bias refuses bad arguments on the host before any HIP call (CPU only)."""
import pytest
import torch

from test_model_ops_abi import A, B, BIG, C, D, DTY, E, F32, INV, MIS, OK, OVL, lib  # noqa: F401


def test_moe_route_grad_biased_refusals(lib):  # noqa: F811
    def f(dtype=F32, logits=A, t=10, e=16, stride=16, bias=E, ids=B, dw=C, k=2, score=0, renorm=1, dl=D, dls=16):
        return lib.ds_moe_route_grad_biased(dtype, logits, t, e, stride, bias, ids, dw, k, score, renorm, 1.0, dl, dls,
                                            None)
    assert f(dtype=1) == DTY
    assert f(t=-1) == INV and f(e=0) == INV and f(k=0) == INV and f(dls=15) == INV and f(score=3) == INV
    assert f(ids=None) == INV and f(dw=None) == INV and f(dl=None) == INV
    assert f(t=0, logits=None, bias=None) == OK
    assert f(dl=D + 2) == MIS and f(bias=E + 2) == MIS
    assert f(dl=A) == OVL and f(dl=C + 8) == OVL and f(bias=D + 32) == OVL
    assert f(t=1 << 40) == BIG


def test_binding_refuses_a_bias_on_the_host():
    import primitives_device_scan_amd as ds
    with pytest.raises(ValueError):
        ds.moe_route_grad(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), bias=torch.zeros(8))
