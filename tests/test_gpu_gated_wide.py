"""The gated recurrence and its gradient where a lane has 16 bytes of channels, as in large batches (with few workgroups it has
4): odd widths, whose last lanes overlap, odd strides and starts, bad values and offsets. Each test first asks what lanes its
shape takes."""
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro
from test_gpu_gated_scan import TYPES, check_grad, check_scan, close, make, off, states, wide

pytestmark = pytest.mark.gpu

CODE = {torch.float32: ds.DS_FP32, torch.bfloat16: ds.DS_BF16, torch.float16: ds.DS_FP16}
FORMS = [(form, mix) for form in ("decay", "log", "sigmoid") for mix in (False, True)]
SHAPE = (2100, 1029, [3, 700, 700, 701, 1500, 2095])


def lane_bytes(dtype, grad, mix, n, d):
    """Bytes of channels that a lane has, from the scratch that the call asks for: a word for each tile and group of eight tiles
    and each channel, the channels rounded up to 16 lanes', and a word a tile. Tiles have 128 rows, 64 in the gradient of mixed
    inputs in 16 bits; the scratch is for that one where the two differ, so half as many rows make as many tiles."""
    size = torch.finfo(dtype).bits // 8
    short = grad and size == 2
    tiles = -(-n // (64 if short and mix else 128))
    room = ds.lib.ds_gated_scan_scratch_bytes(CODE[dtype], int(grad), tiles * (64 if short else 128), d)
    fits = []
    for lane in (16, 4, size):
        span = 16 * lane // size
        words = (tiles + -(-tiles // 8)) * (-(-d // span) * span) + tiles
        if room == (words * 8 + 15) // 16 * 16:
            fits.append(lane)
    assert len(set(fits)) == 1, (fits, "the shape does not tell, or tiles are other than this test takes them to be")
    return fits[0]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", FORMS)
def test_scan(form, mix, dtype):
    assert lane_bytes(dtype, False, mix, *SHAPE[:2]) == 16
    check_scan(*SHAPE, dtype, form, mix, initial=True, extra=(1, 3, 6), lead=1)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", FORMS)
def test_grad(form, mix, dtype):
    assert lane_bytes(dtype, True, mix, *SHAPE[:2]) == 16
    check_grad(*SHAPE, dtype, form, mix, given=True, extra=1, lead=3)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_between_the_rows(dtype):
    n, d, offsets = SHAPE
    gate, x, _ = (t.cuda() for t in make(n, d, dtype, "sigmoid"))
    out = wide(torch.full((n, d), 77.0).to(dtype), 5, 1)
    ds.gated_scan(gate, x, off(offsets), out=out)
    memory = out._base.clone()
    memory[1:1 + n * (d + 5)].view(n, d + 5)[offsets[0]:offsets[-1], :d] = 77
    assert (memory == 77).all()


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix,offsets", [("sigmoid", True, None), ("decay", False, [0, 4000, 4100, 8999])])
def test_many_tiles(form, mix, offsets, dtype):
    n, d = 9000, 133
    assert lane_bytes(dtype, False, mix, n, d) == 16 == lane_bytes(dtype, True, mix, n, d)
    check_scan(n, d, offsets, dtype, form, mix, initial=False, extra=(2, 0, 1))
    check_grad(n, d, offsets, dtype, form, mix, given=False, extra=3)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("offsets", [None, [0, 2, 2, 5, 6]])
def test_one_tile(offsets, dtype):
    """So wide that one tile's rows fill 128 workgroups (of at most 128 channels each) at 16 bytes a lane."""
    n, d = 6, 16_645
    assert d > 127 * 128 and ds.lib.ds_gated_scan_scratch_bytes(CODE[dtype], 1, n, d) == 0
    check_scan(n, d, offsets, dtype, "sigmoid", True, initial=True, extra=(1, 0, 3), lead=1)
    check_grad(n, d, offsets, dtype, "sigmoid", True, given=True, extra=1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")], ids=str)
def test_a_bad_value_stays_in_its_sequence_and_channel(bad, dtype):
    n, d, offsets = 2100, 1029, [0, 900, 900, 1260, 2100]
    assert lane_bytes(dtype, False, True, n, d) == 16 == lane_bytes(dtype, True, True, n, d)
    at, channels = 940, [5, d - 6, d - 1]  # the last two in lanes that overlap
    gate, x, dh = make(n, d, dtype, "sigmoid")
    want = ro.scan(gate, x, offsets, "sigmoid", True, None)
    kept = want[0].to(dtype)
    ref = ro.scan_grad(gate, kept, dh, x, offsets, "sigmoid", True, None, None)
    spoilt, spoilt_dh = x.clone(), dh.clone()
    spoilt[at, channels] = spoilt_dh[at, channels] = bad
    h, final = ds.gated_scan(gate.cuda(), spoilt.cuda(), off(offsets), mix=True)
    hit = torch.zeros((n, d), dtype=torch.bool)
    hit[at:1260, channels] = True
    h = h.cpu()
    assert not torch.isfinite(h[hit]).any() and torch.isfinite(h[~hit]).all()
    close(torch.where(hit, 0, h), torch.where(hit, 0.0, want[0]), want[2], dtype, "h")
    assert (~torch.isfinite(final.cpu())).nonzero().tolist() == [[2, c] for c in channels]
    dgate, dx, dinitial = ds.gated_scan_grad(gate.cuda(), kept.cuda(), spoilt_dh.cuda(), off(offsets), x=x.cuda(), mix=True)
    hit[:] = False
    hit[900:at + 1, channels] = True
    for got, w, e, name in ((dgate, ref[0][0], ref[1][0], "dgate"), (dx, ref[0][1], ref[1][1], "dx")):
        got = got.cpu()
        assert torch.isfinite(got[~hit]).all()
        close(torch.where(hit, 0, got), torch.where(hit, 0.0, w), e, dtype, name)
    assert not torch.isfinite(dx.cpu()[hit]).any()
    assert (~torch.isfinite(dinitial.cpu())).nonzero().tolist() == [[2, c] for c in channels]
    # what lies in rows outside all sequences is not taken into them
    outside = x.clone()
    outside[:10] = outside[2090:] = bad
    h, final = ds.gated_scan(gate.cuda(), outside.cuda(), off([10, 900, 2090]), mix=True)
    assert torch.isfinite(h[10:2090]).all() and torch.isfinite(final).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
def test_offsets_that_are_not_offsets_stay_inside(dtype):
    """Bad offsets give undefined results, but nothing outside the matrices is touched."""
    n, d = 2100, 1029
    assert lane_bytes(dtype, False, False, n, d) == 16 == lane_bytes(dtype, True, False, n, d)
    gate, x, dh = (t.cuda() for t in make(n, d, dtype, "sigmoid"))
    for bad in ([-5, 1000, 500, 1 << 30], [3000, 4000, -1], [0, 1500, 200, 1900, 100]):
        buf = torch.full((n + 64, d), 77.0, device="cuda", dtype=dtype)
        init = states(bad, d, 1).cuda()
        ds.gated_scan(gate, x, off(bad), out=buf[32:32 + n], initial=init)
        ds.gated_scan_grad(gate, x, dh, off(bad), initial=init, dfinal=init)
        torch.cuda.synchronize()
        assert (buf[:32] == 77).all() and (buf[32 + n:] == 77).all()
