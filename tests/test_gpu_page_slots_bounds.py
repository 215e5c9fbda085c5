"""Requests that need far more pages than their tables have entries: the work is bounded by the tables, whatever the lengths
are. What is entered equals what is worked out request by request."""
import numpy as np
import pytest
import torch

import primitives_device_scan_amd as ds
from test_gpu_page_slots import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("count", [0, 7, 95, 200])
def test_more_pages_than_entries(count):
    tables = np.arange(1000, 1015, dtype=np.int32).reshape(5, 3)
    free = np.arange(200, dtype=np.int32)
    run([0, 3, 7, 1, 0], [40, 50, 1, 0, 9], tables, free, count, 1, 120)
    run([0, 3, 7, 1, 0], [40, 50, 1, 0, 9], tables[:, :1], free, count, 2, 60, extra=2)
    run([0, 3, 7, 1, 0], [40, 50, 1, 0, 9], tables[:, :0], free, count, 2, 100)


@pytest.mark.parametrize("longest", [500, (1 << 31) - 1])
def test_far_lengths(longest):
    """3,000 requests in three chunks; of 2^31 - 1 tokens each they name 6 * 10^12 pages."""
    n, width, held = 3000, 40, 3
    new = torch.full((n,), longest, dtype=torch.int32, device="cuda")
    new[1::7] = 0
    new[2::7] = 5
    tables = torch.full((n, width), 77, dtype=torch.int32, device="cuda")
    free = torch.arange(2_000_000, dtype=torch.int32, device="cuda")
    count = torch.tensor([free.numel()], dtype=torch.int32, device="cuda")
    context = torch.full((n,), held, dtype=torch.int32, device="cuda")
    _, slots, positions, left = ds.page_slots(context, new, tables, free, count, 1, 64)
    need = new.long().cpu()
    first = need.cumsum(0) - need
    col = torch.arange(width)
    q = first[:, None] + col - held
    page = torch.where(q < free.numel(), free.numel() - 1 - q, -1)
    want = torch.where((col >= held) & (col - held < need[:, None]), page, 77)
    assert torch.equal(tables.cpu().long(), want)
    assert left.item() == max(free.numel() - int(need.sum()), -(1 << 31))
    assert positions.tolist() == list(range(held, held + 64))
    assert slots.tolist() == [free.numel() - 1 - i if i < width - held else -1 for i in range(64)]
