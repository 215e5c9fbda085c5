"""Page tables and slot maps on the GPU, equal to those worked out request by request and token by token."""
import numpy as np
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro

pytestmark = pytest.mark.gpu


def run(context, new, tables, free, count, page, tokens, extra=0):
    cuda = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    want = ro.pages(np.array(context, dtype=np.int64), np.array(new, dtype=np.int64), tables, free, count, page, tokens)
    buf = torch.full((len(context), tables.shape[1] + extra), 77, dtype=torch.int32, device="cuda")
    view = buf[:, :tables.shape[1]]
    view.copy_(cuda(tables))
    args = (cuda(context), cuda(new), view, cuda(free), cuda([count]), page, tokens)
    for _ in range(2):  # again with the same inputs: the same
        offsets, slots, positions, left = ds.page_slots(*args)
        assert slots.dtype == torch.int64 and left.shape == (1,)
        assert np.array_equal(offsets.cpu().numpy(), want[0])
        assert np.array_equal(slots.cpu().numpy(), want[1])
        assert np.array_equal(positions.cpu().numpy(), want[2])
        assert int(left) == want[3]
        assert np.array_equal(view.cpu().numpy(), want[4])
        assert (buf[:, tables.shape[1]:] == 77).all()


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("requests,longest,deepest,spare", [(1, 1, 0, 0), (1, 300, 5, 3), (7, 1, 50, 0), (64, 20, 40, 9),
                                                            (1024, 3, 9, 0), (1025, 2, 70, 100), (3000, 5, 30, 1)])
def test_slots(requests, longest, deepest, spare, page):
    rng = np.random.default_rng(requests + page)
    context, new = rng.integers(0, deepest + 1, requests), rng.integers(0, longest + 1, requests)
    width = -(-(deepest + longest) // page)
    pages = rng.permutation(requests * width + 50).astype(np.int32)
    tables, free = pages[:requests * width].reshape(requests, width), rng.permutation(pages)
    run(context, new, tables, free, len(free), page, int(new.sum()) + spare, extra=page % 3)


def test_too_few_pages_and_short_tables():
    tables = np.arange(12, dtype=np.int32).reshape(4, 3)
    free = np.array([100, 101, 102, 103, 104], dtype=np.int32)
    for count in (5, 3, 1, 0, -2, 99):
        run([4, 0, 5, 1], [5, 3, 9, 0], tables, free, count, 2, 17)          # pages missing, columns past the width
        run([4, 0, 5, 1], [5, 3, 9, 0], tables, free, count, 2, 6)           # tokens past the batch
    run([4, 0], [3, 2], np.zeros((2, 0), dtype=np.int32), free, 5, 2, 5)     # no columns at all
    run([0, 0], [3, 2], np.full((2, 2), -1, dtype=np.int32), np.zeros(0, dtype=np.int32), 4, 4, 5)
    run([9, -4, 2], [-3, 2, 1], np.arange(30, dtype=np.int32).reshape(3, 10), free, 5, 1, 5)  # negative counts as 0
    run([6, 6], [2, 2], np.full((2, 2), -1, dtype=np.int32), free, 5, 4, 4)  # tables that have no page where one should be


def test_far_positions_and_slots():
    """Positions near 2^31 and slots past 2^32."""
    tables = np.zeros((2, 40000), dtype=np.int32)
    tables[0, 32767] = 2000000000
    run([32767 * 65536 + 65000, 3], [500, 2], tables, np.array([1999999999], dtype=np.int32), 1, 65536, 502)


def test_many_tokens():
    rng = np.random.default_rng(5)
    new = np.array([100000, 1, 0, 30000, 7])
    context = np.array([5, 16, 7, 0, 31])
    tables = rng.integers(0, 1 << 20, (5, 7000)).astype(np.int32)
    run(context, new, tables, rng.permutation(20000).astype(np.int32), 20000, 16, int(new.sum()) + 5000)


def test_no_requests():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    c = torch.tensor([3], dtype=torch.int32, device="cuda")
    off, slots, pos, left = ds.page_slots(e, e, e.view(0, 4), torch.arange(5, device="cuda", dtype=torch.int32), c, 8, 2)
    assert off.tolist() == [0] and slots.tolist() == [-1, -1] and pos.tolist() == [0, 0] and left.tolist() == [3]


def test_graph_and_streams():
    """A decoding loop out of a graph: lengths and free pages move on from step to step on the GPU alone."""
    requests, page, width = 40, 4, 16
    context = torch.arange(requests, dtype=torch.int32, device="cuda") % 7
    held = (context + page - 1) // page
    tables = torch.full((requests, width), -1, dtype=torch.int32, device="cuda")
    tables[torch.arange(width, device="cuda") < held[:, None]] = 900 + torch.arange(int(held.sum()), dtype=torch.int32, device="cuda")
    free = torch.randperm(700, device="cuda").int()
    count = torch.tensor([700], dtype=torch.int32, device="cuda")
    new = torch.ones(requests, dtype=torch.int32, device="cuda")
    want = [(t.clone()) for t in (context, tables, count)]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        offsets, slots, positions, left = ds.page_slots(context, new, tables, free, count, page, requests + 3)
        context += new
        count.copy_(left)
    for step in range(12):
        g.replay()
        torch.cuda.synchronize()
        ref = ro.pages(want[0].cpu().numpy(), np.ones(requests, dtype=np.int64), want[1].cpu().numpy(), free.cpu().numpy(),
                       int(want[2]), page, requests + 3)
        mine = ds.page_slots(want[0], new, want[1], free, want[2], page, requests + 3, stream=side)
        side.synchronize()
        assert np.array_equal(slots.cpu().numpy(), ref[1]) and torch.equal(mine[1], slots)
        assert np.array_equal(positions.cpu().numpy(), ref[2]) and np.array_equal(tables.cpu().numpy(), ref[4])
        assert int(left) == ref[3] == int(count)
        want = [want[0] + 1, want[1], left.clone()]
