"""A larger call after a capture grows the stream's workspace. The graph still replays on the one that it recorded, which
is kept until ds_release_workspace, whichever entry point recorded it."""
import numpy as np
import pytest
import torch

import datagen
import oracle
import primitives_device_scan_amd as ds
from gpu_util import check_scan, say, tile_of, to_dev

pytestmark = pytest.mark.gpu


def record_then_grow(call, larger):
    """A graph of call(), recorded on a stream whose workspace larger() then outgrows."""
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        call()
    cap.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        got = call()
    with torch.cuda.stream(cap):
        larger()
    cap.synchronize()
    # memory that was freed would be taken and overwritten here
    fill = [torch.full((1 << 18,), -1, dtype=torch.int64, device="cuda") for _ in range(64)]
    torch.cuda.synchronize()
    return g, got, cap, fill


def larger_scan():
    x = torch.ones(2000 * tile_of(np.int32), dtype=torch.int32, device="cuda")
    return ds.scan_exclusive(x)


def test_scan():
    n = 40 * tile_of(np.int32) + 3
    x = datagen.uniform_int(81, n, -1000, 1000)
    xin = to_dev(x)
    g, got, cap, _keep = record_then_grow(lambda: ds.scan_exclusive(xin), larger_scan)
    for r in range(3):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_scan(x, False, got.cpu().numpy(), f"replay {r}")
        assert ds.query_timeout(stream=cap) is False


def test_moe_align_of_many_ids():
    experts, n = 500, 60_000      # 500 x 30 counts: two tiles of the look-back
    ids = torch.from_numpy(np.random.default_rng(3).integers(0, experts, n).astype(np.int32)).cuda()
    wc, wo, ws = oracle.moe_align(ids.cpu().numpy(), experts, 16)
    g, got, cap, _keep = record_then_grow(lambda: ds.moe_align(ids, experts, 16), larger_scan)
    for r in range(3):
        for t in got:
            t.fill_(-9)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(got[0].cpu().numpy(), wc) and np.array_equal(got[1].cpu().numpy(), wo), f"replay {r}"
        assert np.array_equal(got[2].cpu().numpy()[:int(wo[-1])], ws)
        assert ds.query_timeout(stream=cap) is False
    say("growth after a captured moe_align")


def test_compaction():
    n = 30 * tile_of(np.int32, compact=True) + 7
    x = datagen.uniform_int(82, n, -1000, 1000)
    xin = to_dev(x)
    want = oracle.compact(x, "<", 0)
    g, got, cap, _keep = record_then_grow(lambda: ds.compact_if(xin, "<", 0), larger_scan)
    for r in range(3):
        got[0].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(got[1].item()) == want.size and np.array_equal(got[0].cpu().numpy()[:want.size], want), f"replay {r}"
        assert ds.query_timeout(stream=cap) is False
