"""A look-back wait that gives up inside the alignment's table scan makes its outputs invalid and nothing else: every kernel
finishes, nothing is written outside the outputs, the call reports it, and the next one is right."""
import numpy as np
import pytest
import torch

import oracle
import primitives_device_scan_amd as ds
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [1, 16, 128])
def test_moe_align_after_a_give_up(block):
    experts, n = 500, 400_000        # 500 x 196 counts: 12 tiles of the look-back
    ids = torch.from_numpy(np.random.default_rng(block).integers(0, experts, n).astype(np.int32)).cuda()
    cap = n + experts * (block - 1)
    room = torch.full((cap + 2 * 65536,), -77, dtype=torch.int32, device="cuda")
    sorted_ids = room[65536:65536 + cap]
    counts, offsets = (torch.empty(experts + k, dtype=torch.int32, device="cuda") for k in (0, 1))

    def call():
        st = ds.lib.ds_moe_align(ids.data_ptr(), n, experts, block, counts.data_ptr(), offsets.data_ptr(),
                                 sorted_ids.data_ptr(), cap, torch.cuda.current_stream().cuda_stream)
        assert st == ds.DS_OK
        return ds.query_timeout()

    ds.set_spin_limit(1)
    try:
        gave_up = [call() for _ in range(3)]
    finally:
        ds.set_spin_limit(0)
    say("gave up:", gave_up)
    assert bool((room[:65536] == -77).all()) and bool((room[65536 + cap:] == -77).all())
    assert call() is False
    wc, wo, ws = oracle.moe_align(ids.cpu().numpy(), experts, block)
    assert np.array_equal(counts.cpu().numpy(), wc) and np.array_equal(offsets.cpu().numpy(), wo)
    assert np.array_equal(sorted_ids.cpu().numpy()[:int(wo[-1])], ws)
