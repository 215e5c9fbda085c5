"""The 64-bit definitions of the operators on ragged batches are held to hand-worked cases and to differences (CPU)."""
import numpy as np
import pytest
import torch

import ragged_oracle as ro


def test_scan_by_hand():
    a = torch.tensor([[0.5], [0.25], [0.5], [0.0], [0.5]])
    x = torch.tensor([[1.0], [2.0], [3.0], [4.0], [5.0]])
    h, final, _, _ = ro.scan(a, x, [0, 2, 2, 4], "decay", False, torch.tensor([[8.0], [7.0], [6.0]]))
    assert h[:4, 0].tolist() == [5.0, 3.25, 6.0, 4.0] and final[:, 0].tolist() == [3.25, 7.0, 4.0]
    assert h[4].isnan()
    h, final, _, _ = ro.scan(a[:2], x[:2], None, "decay", True, None)
    assert h[:, 0].tolist() == [0.5, 0.125 + 1.5] and final[0, 0] == 1.625


@pytest.mark.parametrize("mix", [False, True])
@pytest.mark.parametrize("form", ["decay", "log", "sigmoid"])
def test_gradients_match_differences(form, mix):
    g = torch.Generator().manual_seed(3)
    n, d, offsets = 9, 2, [1, 4, 4, 9]
    gate = torch.rand((n, d), generator=g, dtype=torch.float64) * (0.9 if form == "decay" else -2.0)
    x = torch.randn((n, d), generator=g, dtype=torch.float64)
    initial, dfinal = torch.randn((2, 3, d), generator=g, dtype=torch.float64)
    dh = torch.randn((n, d), generator=g, dtype=torch.float64)

    def loss(gate, x, initial):
        h, final, _, _ = ro.scan(gate, x, offsets, form, mix, initial)
        return (h.nan_to_num() * dh).sum() + (final * dfinal).sum()

    h = ro.scan(gate, x, offsets, form, mix, initial)[0]
    got, _ = ro.scan_grad(gate, h, dh, x, offsets, form, mix, initial, dfinal)
    for i, grad in enumerate(got):
        at = [gate, x, initial]
        for k in range(at[i].numel()):
            e = torch.zeros_like(at[i]).reshape(-1)
            e[k] = 1e-6
            up, down = [list(at), list(at)]
            up[i], down[i] = at[i] + e.view(at[i].shape), at[i] - e.view(at[i].shape)
            want = (loss(*up) - loss(*down)) / 2e-6
            mine = grad.reshape(-1)[k].nan_to_num()
            assert abs(mine - want) <= 1e-6 * (1 + abs(want)), (i, k)


def test_grouped_matches_differences():
    g = torch.Generator().manual_seed(4)
    x = torch.randn((4, 3), generator=g, dtype=torch.float64)
    w = torch.randn((3, 5, 3), generator=g, dtype=torch.float64)
    index, offsets = torch.tensor([6, 1, 8, 0, 3, -1, 2]), [0, 3, 3, 6]
    y = ro.grouped(x, w, offsets, index, 2, False)[0]
    assert torch.allclose(y[0], w[0] @ x[3]) and (y[2] == 0).all() and y[6].isnan().all() and (y[5] == 0).all()
    dy = torch.randn((7, 5), generator=g, dtype=torch.float64)
    dw = ro.grouped_grad(dy, x, offsets, index, 2, None)[0]
    dx = ro.grouped(dy, w, offsets, None, 1, True)[0]
    for e, i, j in ((0, 1, 2), (1, 0, 0), (2, 4, 1)):
        d = torch.zeros_like(w)
        d[e, i, j] = 1e-6
        up = (ro.grouped(x, w + d, offsets, index, 2, False)[0] - ro.grouped(x, w - d, offsets, index, 2, False)[0])
        assert abs((up[:6] * dy[:6]).sum() / 2e-6 - dw[e, i, j]) < 1e-6
    assert torch.allclose(dx[4], w[2].T @ dy[4])


def test_pages_by_hand():
    tables = np.full((3, 3), 90, dtype=np.int32)
    tables[0, :2] = [4, 5]
    tables[2, 0] = 6
    off, slots, pos, left, out = ro.pages(np.array([3, 0, 2]), np.array([2, 3, 1]), tables,
                                          np.array([10, 11, 12, 13, 14]), 4, 2, 8)
    assert off.tolist() == [0, 2, 5, 6] and left == 4 - 4
    assert out.tolist() == [[4, 5, 13], [12, 11, 90], [6, 10, 90]]
    assert slots.tolist() == [11, 26, 24, 25, 22, 20, -1, -1] and pos.tolist() == [3, 4, 0, 1, 2, 2, 0, 0]
    off, slots, pos, left, out = ro.pages(np.array([0, 0]), np.array([2, 3]), np.full((2, 1), 7), np.array([1, 2, 3]), 2, 1, 4)
    assert left == 2 - 5 and slots.tolist() == [2, -1, -1, -1] and out.tolist() == [[2], [-1]]
