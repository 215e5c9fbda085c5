"""The language-model operators have no autograd history: they refuse tensors that require grad while it is enabled, so that
no gradient is lost without a word (CPU: the refusal comes before any other check; GPU: what is not refused runs)."""
import pytest
import torch

import primitives_device_scan_amd as ds


def calls(dev):
    """Each entry point with one of its inputs as it is given."""
    f = lambda *shape: torch.ones(shape, device=dev)
    b = lambda *shape: torch.ones(shape, device=dev, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int64, device=dev)
    chosen = torch.zeros(4, 2, dtype=torch.int32, device=dev)
    ex = lambda x=None, w_in=None, w_out=None, w=None: ds.moe_experts(
        b(4, 8) if x is None else x, b(3, 8, 8) if w_in is None else w_in, b(3, 8, 4) if w_out is None else w_out, chosen,
        f(4, 2) if w is None else w)
    return [(f(5, 8), lambda t: ds.embedding(t, ids)), (f(4, 8), lambda t: ds.embedding(f(5, 8), ids, out=t)),
            (f(4, 8), lambda t: ds.embedding_grad(t, ids, 5)),
            (f(5, 8), lambda t: ds.embedding_grad(f(4, 8), ids, 5, out=t, accumulate=True)),
            (f(4, 6), lambda t: ds.moe_route(t, 2)), (f(6), lambda t: ds.moe_route(f(4, 6), 2, bias=t)),
            (f(4, 6), lambda t: ds.moe_route_grad(t, chosen, f(4, 2))),
            (f(4, 2), lambda t: ds.moe_route_grad(f(4, 6), chosen, t)),
            (b(4, 8), lambda t: ex(x=t)), (b(3, 8, 8), lambda t: ex(w_in=t)), (b(3, 8, 4), lambda t: ex(w_out=t)),
            (f(4, 2), lambda t: ex(w=t))]


@pytest.mark.parametrize("case", range(12))
def test_refused_on_the_host(case):
    t, call = calls("cpu")[case]
    with pytest.raises(ValueError, match="requires grad"):
        call(t.requires_grad_())
    with torch.no_grad(), pytest.raises(ValueError, match="GPU tensor"):
        call(t)


@pytest.mark.gpu
@pytest.mark.parametrize("case", range(12))
def test_refused_and_allowed_on_the_gpu(case):
    t, call = calls("cuda")[case]
    want = call(t.clone())
    t.requires_grad_()
    with pytest.raises(ValueError, match="requires grad"):
        call(t)
    with torch.no_grad():
        got = call(t)
    same = lambda a, b: all(map(torch.equal, a, b)) if isinstance(a, tuple) else torch.equal(a, b)
    assert same(got, want) if got is not t else True
    call(t.detach())
