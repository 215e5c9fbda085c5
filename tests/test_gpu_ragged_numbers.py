"""Numbers that do not fit the library's 32 bits are refused, not cut."""
import pytest
import torch

import primitives_device_scan_amd as ds

pytestmark = pytest.mark.gpu

FAR = [0, -1, 1 << 31, (1 << 32) + 2]


def ints(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("top_k", FAR)
def test_top_k(top_k):
    x, w = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((4, 8), (1, 8, 8)))
    for call in (lambda: ds.grouped_matmul(x, w, ints(0, 4), index=ints(0, 1, 2, 3), top_k=top_k),
                 lambda: ds.grouped_matmul_grad(x, x, ints(0, 4), index=ints(0, 1, 2, 3), top_k=top_k)):
        with pytest.raises(ValueError, match="top_k"):
            call()


@pytest.mark.parametrize("page", FAR)
def test_page(page):
    with pytest.raises(ValueError, match="page"):
        ds.page_slots(ints(0), ints(1), ints(0).view(1, 1), ints(5), ints(1), page, 1)


def test_the_largest():
    x, w = (torch.ones(s, dtype=torch.bfloat16, device="cuda") for s in ((4, 8), (1, 8, 8)))
    y = ds.grouped_matmul(x, w, ints(0, 4), index=ints(0, 1, -1, (1 << 31) - 1), top_k=(1 << 31) - 1)
    assert y[:, 0].tolist() == [8, 8, 0, 8]  # the last is assignment 0 of token 1
    offsets, slots, positions, left = ds.page_slots(ints(5), ints(2), ints(3).view(1, 1), ints(9), ints(1), (1 << 31) - 1, 2)
    assert slots.tolist() == [3 * ((1 << 31) - 1) + 5, 3 * ((1 << 31) - 1) + 6] and left.tolist() == [1]
