"""The gradient of the grouped matrices leaves out the rows for which the index names no row of x: dy's values there, infinities
and NaN among them, have no part in it. Against 64-bit sums over the other rows, in every tile size."""
import pytest
import torch

import primitives_device_scan_amd as ds
from test_gpu_grouped_matmul import big_close, big_reference, choose, setting

pytestmark = pytest.mark.gpu

# (rows, cols, lengths of the groups): tiles of 64, 128 and 256, and rows that are no whole 16 bytes
SHAPES = [(72, 64, [40, 0, 3, 100, 33]), (1032, 1024, [700, 9, 400, 33, 250, 0, 500, 80]),
          (2056, 2056, [600] * 14 + [3000, 0]), (77, 100, [17, 40, 0, 70])]
IDS = [f"{r}x{c}-{len(g)}" for r, c, g in SHAPES]


@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("rows,cols,lengths", SHAPES, ids=IDS)
def test_gradient_of_the_matrices(rows, cols, lengths, dtype, bad):
    offsets, m = setting(lengths, 0, 6)
    tokens, top_k = m // 3 + 5, 3
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, dy = (torch.randn(s, generator=g, device="cuda").to(dtype) for s in ((tokens, cols), (m, rows)))
    index = choose(m, tokens, top_k, 3).cuda()
    index[offsets[2]:offsets[2] + 40] = tokens * top_k  # a run of padding longer than a stage
    if lengths[0] > 1:
        index[offsets[1] - 1] = -1                       # a group's last row
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    padding = (index < 0) | (index >= tokens * top_k)
    assert padding[:offsets[-1]].sum() > 40
    clean = torch.where(padding[:, None], 0, dy)
    spoilt = torch.where(padding[:, None], bad, dy)
    w = torch.zeros((len(lengths), rows, cols), dtype=dtype, device="cuda")
    _, _, want, err = big_reference(x, w, clean, offsets, index, top_k, False)
    kw = dict(index=index, top_k=top_k)
    big_close(ds.grouped_matmul_grad(spoilt, x, off, **kw), want, err, dtype, "gradient")
    old = torch.randn(want.shape, generator=g, device="cuda")
    got = ds.grouped_matmul_grad(spoilt, x, off, out=old.clone(), accumulate=True, **kw)
    big_close(got, want + old.double(), err + 4 * 2.0 ** -24 * old.abs().double(), torch.float32, "added gradient")
    assert torch.equal(ds.grouped_matmul_grad(spoilt, x, off, dtype=torch.float32, **kw),
                       ds.grouped_matmul_grad(clean, x, off, dtype=torch.float32, **kw))


def test_a_group_of_padding():
    x = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    dy = torch.full((96, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    dy[64:] = 1
    off = torch.tensor([0, 32, 64, 96], dtype=torch.int32, device="cuda")
    index = torch.full((96,), 4, dtype=torch.int32, device="cuda")
    index[64:] = 0
    dw = ds.grouped_matmul_grad(dy, x, off, index=index)
    assert (dw[:2] == 0).all() and (dw[2] == 32).all()
