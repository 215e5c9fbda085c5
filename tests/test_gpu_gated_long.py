"""Gates near 1 over 32,768 steps, the same at every step, so that what is lost in one tile's product of gates is lost in every
tile's: a state that only decays, forward and back, against a^t in 64 bits.

u = 2^-24. Between 0.9 and 1 a rounding is at most u / 2. What passes from a sequence's one end to the other is rounded once
for each tile (512 at most), part of the last tile (16) and row of the last part (8), 540 in all. A tile's product is held as
1 - a, formed over 8 rows and then 16 parts: 24 roundings of it, and 24 of the factors before them, each relative to 1 - a;
with the gate's own error they are taken of the whole sum of 1 - a, which is t (1 - a)."""
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro
from test_gpu_gated_scan import TYPES, close

pytestmark = pytest.mark.gpu

N, D = 32_768, 64


def decaying(dtype, form):
    """(gate [N, D], a^t for t = 1 .. N and its bound): 32,768 (1 - a) from 0.005 to 0.1."""
    lost = torch.logspace(-2.3, -1.0, D, dtype=torch.float64) / N  # 1 - a
    gate = (-lost if form == "log" else torch.log(1 / lost - 1)).to(dtype)
    _, rest, _, off = ro.gates(gate, form)
    t = torch.arange(1, N + 1, dtype=torch.float64)[:, None]
    power = torch.exp(t * (gate.double() if form == "log" else torch.log1p(-rest)))
    assert power.min() > 0.9
    return gate.expand(N, D).contiguous().cuda(), power, 540 / 2 * ro.U + t * rest * (off + 48 * ro.U)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form", ["log", "sigmoid"])
@pytest.mark.parametrize("mix", [False, True])
def test_states(mix, form, dtype):
    gate, want, err = decaying(dtype, form)
    h, final = ds.gated_scan(gate, torch.zeros_like(gate), form=form, mix=mix, initial=torch.ones((1, D), device="cuda"))
    close(h, want, err, dtype, "h")
    close(final, want[-1:], err[-1:], torch.float32, "final")


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form", ["log", "sigmoid"])
@pytest.mark.parametrize("mix", [False, True])
def test_gradient_of_the_initial_states(mix, form, dtype):
    gate, want, err = decaying(dtype, form)
    zero, one = torch.zeros_like(gate), torch.ones((1, D), device="cuda")
    _, dx, dinitial = ds.gated_scan_grad(gate, zero, zero, x=zero if mix else None, form=form, mix=mix, dfinal=one)
    close(dinitial, want[-1:], err[-1:], torch.float32, "dinitial")
    if not mix:  # what reaches step t from the end
        back, bound = torch.cat([torch.ones_like(want[:1]), want[:-1]]).flip(0), err.flip(0)
        close(dx, back, bound, dtype, "dx")
