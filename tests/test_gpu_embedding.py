"""Token embedding and its gradient on the GPU against the definitions in 64 bits (tests/model_oracle.py).

The lookup is one 32-bit product and one rounding, so it has to be equal bit for bit to the same two roundings on the
host. The gradient's bound counts the additions of each row (model_oracle.embedding_grad_bound)."""
import numpy as np
import pytest
import torch

import model_oracle as mo
import primitives_device_scan_amd as ds
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
RANK_MAX = 8192  # ids that one launch sorts


def normal(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype)


def token_ids(seed, n, rows, dtype=torch.int64, bad=0.1):
    """Skewed ids, some of them outside the table on either side."""
    rng = np.random.default_rng(seed)
    ids = np.minimum((rows ** rng.random(n)).astype(np.int64) - 1, rows - 1)
    out = rng.random(n)
    ids[out < bad] = -1
    ids[out < bad / 2] = rows
    if n > 4:
        ids[n // 2] = -(1 << 31)
        ids[n // 3] = (1 << 31) - 1 if dtype == torch.int32 else (1 << 40) + 1
    return torch.from_numpy(ids).to(dtype)


def lookup_reference(table, ids, scale):
    live = (ids >= 0) & (ids < table.shape[0])
    y = table[torch.where(live, ids.long(), 0)].float() * torch.tensor(scale, dtype=torch.float32)
    y[~live] = 0
    return y.to(table.dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,dim,rows", [(1, 1, 1), (1, 2048, 5), (5, 3, 7), (64, 128, 100), (257, 1000, 50),
                                        (130, 513, 1000), (33, 4097, 11), (700, 8, 3)])
def test_lookup(dtype, idt, n, dim, rows):
    say("lookup", dtype, idt, n, dim, rows)
    table, ids = normal(n, (rows, dim), dtype), token_ids(n + 1, n, rows, idt)
    for scale in (1.0, 45.254833):
        got = ds.embedding(table.cuda(), ids.cuda(), scale=scale)
        assert torch.equal(got.cpu(), lookup_reference(table, ids, scale))


@pytest.mark.parametrize("dtype", DTYPES)
def test_lookup_strides_offsets_and_shape(dtype):
    big = normal(1, (40, 150), dtype).cuda()
    table = big[3:, 1:102]                       # rows 150 apart, starting off any 16-byte boundary
    ids = token_ids(2, 60, 37)
    room = torch.full((60, 130), 7.0, dtype=dtype, device="cuda")
    got = ds.embedding(table, ids.cuda(), scale=3.0, out=room[:, 5:106])
    want = lookup_reference(table.cpu(), ids, 3.0)
    assert torch.equal(got.cpu(), want) and torch.equal(room[:, 5:106].cpu(), want)
    assert bool((room[:, :5] == 7).all()) and bool((room[:, 106:] == 7).all())   # nothing else is written
    got = ds.embedding(table, ids.view(3, 4, 5).cuda())
    assert got.shape == (3, 4, 5, 101) and torch.equal(got.cpu().view(60, 101), lookup_reference(table.cpu(), ids, 1.0))


def test_lookup_special_values_and_empty():
    table = torch.tensor([[float("inf"), float("nan"), -0.0, 1e-40], [1.0, 2.0, 3.0, 4.0]]).cuda()
    got = ds.embedding(table, torch.tensor([0, 5, 1, -1]).cuda(), scale=2.0).cpu()
    assert got[0, 0] == float("inf") and got[0, 1] != got[0, 1] and bool(torch.signbit(got[0, 2]))
    assert bool((got[1] == 0).all()) and bool((got[3] == 0).all()) and got[2].tolist() == [2, 4, 6, 8]
    assert ds.embedding(table, torch.zeros(0, dtype=torch.int64).cuda()).shape == (0, 4)
    assert ds.embedding(table[:, :0], torch.tensor([1]).cuda()).shape == (1, 0)
    got = ds.embedding(table[:0], torch.tensor([0, 1]).cuda())
    assert got.shape == (2, 4) and bool((got == 0).all())


def test_lookup_past_32_bit_offsets():
    rows, dim = 2_200_000, 2048                 # 4.5G elements, 9 GB
    table = torch.empty((rows, dim), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 1_048_576, 2_097_151, 2_097_152, rows - 1])
    table[at.cuda()] = normal(3, (5, dim), torch.bfloat16).cuda()
    assert torch.equal(ds.embedding(table, at.cuda()), table[at.cuda()])


def check_grad(dout, ids, rows, scale, out_dtype, old=None, what=""):
    """One call; every element against the definition, and the same bits from a second call."""
    g = old.cuda() if old is not None else None
    got = ds.embedding_grad(dout.cuda(), ids.cuda(), rows, scale=scale, dtype=out_dtype, out=g,
                            accumulate=old is not None)
    ref, c, s = mo.embedding_grad(mo.f64(dout), ids.numpy(), rows, float(np.float32(scale)),
                                  None if old is None else mo.f64(old))
    worst = mo.within(got, ref, mo.embedding_grad_bound(ref, c, s, out_dtype), what)
    if old is None:
        assert bool((got.cpu()[torch.from_numpy(c == 0)] == 0).all())
        again = ds.embedding_grad(dout.cuda(), ids.cuda(), rows, scale=scale, dtype=out_dtype)
        assert torch.equal(got, again), "two runs differ"
    else:
        untouched = torch.from_numpy(c == 0)
        assert torch.equal(got.cpu()[untouched], old[untouched])
    say(what, "worst share of the bound %.2f" % worst)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("idt", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,dim,rows", [(1, 1, 1), (1, 700, 9), (7, 3, 5), (8, 64, 2), (9, 1000, 300), (63, 2100, 7000),
                                         (64, 9, 30), (128, 260, 900), (129, 260, 900), (63, 40, 64),
                                        (64, 513, 31), (65, 520, 33), (500, 33, 20), (1003, 1000, 400),
                                        (4097, 24, 100)])
def test_grad(dtype, idt, n, dim, rows):
    dout, ids = normal(n, (n, dim), dtype), token_ids(n + 5, n, rows, idt)
    check_grad(dout, ids, rows, 1.0, dtype, what=f"grad {dtype} {n}x{dim} rows {rows}")
    check_grad(dout, ids, rows, 3.7, torch.float32, normal(n + 2, (rows, dim), torch.float32), "added in 32 bits")
    check_grad(dout, ids, rows, 0.5, dtype, normal(n + 3, (rows, dim), dtype), "added in place")


@pytest.mark.parametrize("n", [RANK_MAX - 1, RANK_MAX, RANK_MAX + 1, 20_000])
@pytest.mark.parametrize("rows", [2, 600, 262_000])
def test_grad_both_sorts(n, rows):
    # up to RANK_MAX ids are sorted by rank, more by counting passes over 9 bits: one for 2 rows, two for the others
    dout, ids = normal(n, (n, 12), torch.bfloat16), token_ids(n + 7, n, rows)
    check_grad(dout, ids, rows, 1.0, torch.float32, what=f"{n} ids, {rows} rows")


@pytest.mark.parametrize("n,rows", [(9_000, 600_000), (131_072, 5000), (131_073, 262_143), (150_001, 262_144),
                                    (262_144, 70), (262_145, 70), (300_001, 70_000)])
def test_grad_long_sorts(n, rows):
    # three passes, tiles of 1,024 and of 2,048 ids, and above 262,144 ids the radix passes
    dout, ids = normal(n, (n, 3), torch.bfloat16), token_ids(n + 9, n, rows)
    check_grad(dout, ids, rows, 1.0, torch.float32, what=f"{n} ids, {rows} rows")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,dim", [(1, 1), (1, 7), (2, 1), (2, 3), (3, 2), (5, 9), (40, 15), (33, 531)])
def test_grad_reads_stay_inside(dtype, n, dim):
    # the gradient of the last rows of a buffer that ends with them; what lies behind is NaN and must not be seen
    room = torch.full((n * dim + 64,), float("nan"), dtype=dtype, device="cuda")
    dout = room[:n * dim].view(n, dim)
    dout.copy_(normal(n + dim, (n, dim), dtype))
    ids = token_ids(dim, n, 4, bad=0.0)
    got = ds.embedding_grad(dout, ids.cuda(), 4)
    ref, c, s = mo.embedding_grad(mo.f64(dout), ids.numpy(), 4, 1.0)
    mo.within(got, ref, mo.embedding_grad_bound(ref, c, s, dtype), f"{n} x {dim}")


@pytest.mark.parametrize("n", [64, 65, 127, 128, 129, 3000, 12_001])
def test_grad_one_row_distinct_rows_and_none(n):
    dout = normal(n, (n, 70), torch.float32)
    check_grad(dout, torch.full((n,), 4), 9, 1.0, torch.float32, what="one row takes all")
    check_grad(dout, torch.from_numpy(np.random.default_rng(n).permutation(n)), n, 1.0, torch.float32, what="distinct")
    check_grad(dout, torch.full((n,), -1), 9, 1.0, torch.float32, what="all left out")
    two = torch.full((n,), 8)
    two[::2] = 0
    check_grad(dout, two, 9, 1.0, torch.float32, what="first and last row")
    # every run crosses chunks, runs of 64 + 1 and of many chunks in turn
    runs = torch.repeat_interleave(torch.arange(6 * n), torch.tensor([65, 1, 64, 200, 7, 128]).repeat(n))[:n]
    check_grad(dout, runs, n, 1.0, torch.float32, what="runs")


def test_grad_strides_shape_and_guards():
    n, dim, rows = 300, 45, 20
    dout, ids = normal(1, (n, 64), torch.bfloat16).cuda(), token_ids(2, n, rows)
    room = torch.full((rows, 50), 7.0, device="cuda")
    got = ds.embedding_grad(dout[:, 3:48], ids.cuda(), rows, out=room[:, 2:47])
    ref, c, s = mo.embedding_grad(mo.f64(dout)[:, 3:48], ids.numpy(), rows, 1.0)
    mo.within(got, ref, mo.embedding_grad_bound(ref, c, s, torch.float32), "strided")
    assert bool((room[:, :2] == 7).all()) and bool((room[:, 47:] == 7).all())
    got3 = ds.embedding_grad(dout[:, :dim].contiguous().view(3, 100, dim), ids.view(3, 100).cuda(), rows)
    ref, c, s = mo.embedding_grad(mo.f64(dout)[:, :dim], ids.numpy(), rows, 1.0)
    mo.within(got3, ref, mo.embedding_grad_bound(ref, c, s, torch.bfloat16), "shaped")
    assert bool((ds.embedding_grad(dout[:0], ids[:0].cuda(), rows) == 0).all())
    kept = room.clone()
    assert torch.equal(ds.embedding_grad(dout[:0, :50], ids[:0].cuda(), rows, out=room, accumulate=True), kept)
    assert ds.embedding_grad(dout, ids.cuda(), 0).shape == (0, 64)


def test_grad_past_32_bit_offsets():
    # 2.8G values of dout; then 2.25G values of the gradient
    n, dim = 70_000, 40_000
    dout = torch.ones((n, dim), dtype=torch.bfloat16, device="cuda")
    ids = torch.arange(n, device="cuda") % 5
    ids[-3:] = 4
    got = ds.embedding_grad(dout, ids, 6, dtype=torch.float32)
    assert torch.equal(got[:, 0], torch.bincount(ids, minlength=6).float())
    assert torch.equal(got, got[:, :1].expand(6, dim))
    del dout, got
    rows, dim = 1_100_000, 2048
    grad = torch.full((rows, dim), 3.0, device="cuda")
    ids = torch.tensor([rows - 1, 5, 1_048_576, rows - 1], device="cuda")
    d = normal(9, (4, dim), torch.float32).cuda()
    got = ds.embedding_grad(d, ids, rows, out=grad)
    assert torch.equal(got[rows - 1], d[0] + d[3]) and torch.equal(got[5], d[1]) and torch.equal(got[1_048_576], d[2])
    got[ids] = 0
    assert not bool(got.any())


def test_grad_infinities_stay_in_their_rows():
    dout = torch.ones(200, 8)
    ids = torch.arange(200) % 5
    dout[7] = float("inf")       # row 2
    dout[9] = float("nan")       # row 4
    ids[11] = -1
    dout[11] = float("nan")      # left out
    got = ds.embedding_grad(dout.cuda(), ids.cuda(), 6).cpu()
    assert bool((got[2] == float("inf")).all()) and bool((got[4] != got[4]).all())
    assert got[0, 0] == 40 and got[1, 0] == 39 and got[3, 0] == 40 and got[5, 0] == 0


def test_grad_against_differences():
    # <d, W -> sum of embedding(W) * dout> is linear, so one difference of any size gives it exactly but for rounding
    table, ids, dout = normal(1, (50, 33), torch.float32), token_ids(2, 90, 50), normal(3, (90, 33), torch.float32)
    d = normal(4, (50, 33), torch.float32)
    up, down = (mo.f64(ds.embedding((table + s * d).cuda(), ids.cuda(), scale=2.0)) for s in (0.5, -0.5))
    slope = ((up - down) * mo.f64(dout)).sum()
    grad = mo.f64(ds.embedding_grad(dout.cuda(), ids.cuda(), 50, scale=2.0))
    size = (np.abs(mo.f64(dout)).sum(1)[:, None] * 2 * (np.abs(mo.f64(table)).max() + 1)).sum()
    assert abs(slope - (grad * mo.f64(d)).sum()) <= 8 * mo.U * size


def test_two_streams_and_raw_handles():
    ids = [token_ids(k, 9000 + k, 700) for k in (1, 2)]
    dout = [normal(k, (9000 + k, 40), torch.bfloat16) for k in (1, 2)]
    dev = [(i.cuda(), d.cuda()) for i, d in zip(ids, dout)]
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        got = [ds.embedding_grad(dev[k][1], dev[k][0], 700, stream=s[0] if k == 0 else s[1].cuda_stream)
               for k in (0, 1)]
    torch.cuda.synchronize()
    for k in (0, 1):
        ref, c, a = mo.embedding_grad(mo.f64(dout[k]), ids[k].numpy(), 700, 1.0)
        mo.within(got[k], ref, mo.embedding_grad_bound(ref, c, a, torch.bfloat16), f"stream {k}")


@pytest.mark.parametrize("n", [40, 900, 9001, 270_000])
def test_graph_replays(n):
    rows, dim = 500, 72
    ids, dout, table = token_ids(1, n, rows).cuda(), normal(2, (n, dim), torch.bfloat16).cuda(), \
        normal(3, (rows, dim), torch.bfloat16).cuda()
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        ds.embedding_grad(dout, ids, rows)          # sizes the workspace
    cap.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        y = ds.embedding(table, ids, scale=2.0)
        dw = ds.embedding_grad(dout, ids, rows)
    for r in range(4):
        ids.copy_(token_ids(10 + r, n, rows))
        dout.copy_(normal(20 + r, (n, dim), torch.bfloat16))
        want = ds.embedding(table, ids, scale=2.0), ds.embedding_grad(dout, ids, rows)   # eager, on another stream
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[0]) and torch.equal(dw, want[1]), f"replay {r}"


def test_workspace_growth_keeps_captured_graphs():
    # a larger call after the capture grows the stream's workspace; the graph still replays on the one it recorded
    rows, dim, n = 100, 40, 300
    ids, dout = token_ids(1, n, rows).cuda(), normal(2, (n, dim), torch.float32).cuda()
    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        want = ds.embedding_grad(dout, ids, rows)
    cap.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        got = ds.embedding_grad(dout, ids, rows)
    big = token_ids(3, 60_000, 5000).cuda()
    wide = torch.ones(60_000, 600, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(cap):
        ds.embedding_grad(wide, big, 5000)
    torch.cuda.synchronize()
    for _ in range(2):
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals_on_the_gpu():
    x = torch.zeros(4, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (lambda: ds.embedding(x.t(), ids), lambda: ds.embedding(x, ids.cpu()),
                lambda: ds.embedding(x, ids, out=x[:3]), lambda: ds.embedding(x[:1].expand(4, 8), ids),
                lambda: ds.embedding_grad(x, ids[:3], 5), lambda: ds.embedding_grad(x, ids, 5, accumulate=True),
                lambda: ds.embedding_grad(x, ids, 5, out=torch.zeros(4, 8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ds.embedding(x, ids.short()), lambda: ds.embedding(x, ids, out=x.bfloat16()),
                lambda: ds.embedding_grad(x, ids, 5, dtype=torch.bfloat16)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ds.DevscanError):
        ds.embedding(x, ids, out=x)             # over its own table
