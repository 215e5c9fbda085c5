"""The gradient of the embedding over so many tokens that the radix passes' count table has more than one tile: its scan
waits for nothing, so that no wait that gives up can leave positions and rows unwritten which the sums then follow."""
import numpy as np
import pytest
import torch

import model_oracle as mo
import primitives_device_scan_amd as ds
from test_gpu_embedding import normal, token_ids

pytestmark = pytest.mark.gpu

N = 1_000_003  # 256 digits x 41 groups of tiles: 10,496 words, where a tile of the scan has 8,192


def reference(dout, ids, rows):
    g, s = np.zeros((rows, dout.shape[1])), np.zeros((rows, dout.shape[1]))
    live = (ids >= 0) & (ids < rows)
    np.add.at(g, ids[live], dout[live])
    np.add.at(s, ids[live], np.abs(dout[live]))
    return g, np.bincount(ids[live], minlength=rows).astype(float), s


@pytest.mark.parametrize("rows", [70, 70_000])
def test_grad_of_a_million_ids(rows):
    dout, ids = normal(1, (N, 3), torch.bfloat16), token_ids(2, N, rows)
    ref, c, s = reference(mo.f64(dout), ids.numpy(), rows)
    got = ds.embedding_grad(dout.cuda(), ids.cuda(), rows, dtype=torch.float32)
    mo.within(got, ref, mo.embedding_grad_bound(ref, c, s, torch.float32), f"{N} ids, {rows} rows")


def test_no_wait_of_the_gradient_can_give_up():
    rows = 70_000
    dout, ids = normal(3, (N, 3), torch.bfloat16).cuda(), token_ids(4, N, rows).cuda()
    want = ds.embedding_grad(dout, ids, rows)
    torch.cuda.synchronize()
    ds.set_spin_limit(1)
    try:
        got = ds.embedding_grad(dout, ids, rows)
        assert ds.query_timeout() is False
    finally:
        ds.set_spin_limit(0)
    assert torch.equal(got, want)


def test_grad_of_a_million_ids_replays():
    rows = 5000
    dout, ids = normal(5, (N, 3), torch.bfloat16).cuda(), token_ids(6, N, rows).cuda()
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        ds.embedding_grad(dout, ids, rows)
    cap.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        got = ds.embedding_grad(dout, ids, rows)
    for r in range(3):
        ids.copy_(token_ids(10 + r, N, rows))
        want = ds.embedding_grad(dout, ids, rows)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), f"replay {r}"
