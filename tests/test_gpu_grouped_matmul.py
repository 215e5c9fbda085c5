"""Products grouped by expert and the gradient of their matrices on the GPU, against 64-bit sums within the error that
32-bit sums of as many products may have; rows outside the groups stay as they were."""
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
# (rows, cols, lengths of the groups, rows before and behind them)
SHAPES = [(1, 1, [1], 0, 0), (16, 32, [3, 0, 5], 0, 0), (64, 64, [64], 0, 0), (65, 33, [1, 63, 2], 2, 3),
          (128, 256, [0, 0, 130], 0, 7), (77, 100, [17, 40, 0, 1], 1, 0), (200, 8, [9, 300], 0, 0), (8, 520, [33, 31], 0, 1),
          (256, 192, [200, 5, 270], 0, 0), (130, 72, [1] * 40, 0, 0), (96, 1024, [40, 0, 25], 0, 0)]
IDS = [f"{r}x{c}-{len(g)}" for r, c, g, _, _ in SHAPES]


def rand(*shape, dtype, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def wide(x, extra):
    buf = torch.full((x.shape[0], x.shape[1] + extra), 77.0, dtype=x.dtype, device="cuda")
    buf[:, :x.shape[1]] = x
    return buf[:, :x.shape[1]]


def setting(lengths, before, behind):
    offsets = [before]
    for v in lengths:
        offsets.append(offsets[-1] + v)
    return offsets, offsets[-1] + behind


def choose(m, tokens, top_k, seed):
    """An index of m rows: assignments of the tokens, one in five padding or nonsense."""
    g = torch.Generator().manual_seed(seed)
    index = torch.randint(0, tokens * top_k, (m,), generator=g, dtype=torch.int32)
    index[torch.rand(m, generator=g) < 0.1] = tokens * top_k
    index[torch.rand(m, generator=g) < 0.1] = -3
    return index


def close(got, want, err, dtype, what):
    got = got.double().cpu()
    there = ~want.isnan()
    bad = ((got - want).abs() > ro.rounded(err, want, dtype)) & there
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs()[there].max()), bad.nonzero()[:4].tolist())


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_products(shape, gather, transposed, dtype):
    rows, cols, lengths, before, behind = shape
    offsets, m = setting(lengths, before, behind)
    depth, width = (rows, cols) if transposed else (cols, rows)
    tokens, top_k = (max(1, m // 2), 3) if gather else (m, 1)
    x, w = rand(tokens, depth, dtype=dtype, seed=1), rand(len(lengths), rows, cols, dtype=dtype, seed=2)
    index = choose(m, tokens, top_k, 3) if gather else None
    want, err = ro.grouped(x, w, offsets, index, top_k, transposed)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for extra in (0, 8, 5):
        out = wide(torch.full((m, width), 77.0).to(dtype), extra)
        y = ds.grouped_matmul(wide(x, extra), w.cuda(), off, index=None if index is None else index.cuda(), top_k=top_k,
                              transposed=transposed, out=out)
        assert y is out
        close(y, want, err, dtype, f"extra {extra}")
        assert (y.cpu()[want.isnan()] == 77).all(), "rows outside the groups"
    again = ds.grouped_matmul(x.cuda(), w.cuda(), off, index=None if index is None else index.cuda(), top_k=top_k,
                              transposed=transposed)
    inside = ~want.isnan()
    assert torch.equal(again.cpu()[inside], ds.grouped_matmul(
        x.cuda(), w.cuda(), off, index=None if index is None else index.cuda(), top_k=top_k, transposed=transposed).cpu()[inside])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("out_dtype,add", [(None, False), (torch.float32, False), (torch.float32, True), (None, True)])
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_gradient_of_the_matrices(shape, gather, out_dtype, add, dtype):
    rows, cols, lengths, before, behind = shape
    offsets, m = setting(lengths, before, behind)
    out_dtype = out_dtype or dtype
    tokens, top_k = (max(1, m // 2), 3) if gather else (m, 1)
    x, dy = rand(tokens, cols, dtype=dtype, seed=1), rand(m, rows, dtype=dtype, seed=2)
    index = choose(m, tokens, top_k, 3) if gather else None
    old = rand(len(lengths), rows, cols, dtype=out_dtype, seed=4) if add else None
    want, err = ro.grouped_grad(dy, x, offsets, index, top_k, old)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for extra in (0, 8, 5):
        out = old.cuda() if add else None
        args = (wide(dy, extra), wide(x, extra), off)
        kw = dict(index=None if index is None else index.cuda(), top_k=top_k, dtype=out_dtype)
        dw = ds.grouped_matmul_grad(*args, out=out, accumulate=add, **kw)
        assert dw.dtype == out_dtype and (not add or dw is out)
        close(dw, want, err, out_dtype, f"extra {extra}")
        if not add:
            assert torch.equal(ds.grouped_matmul_grad(*args, **kw), dw)


def test_after_the_alignment():
    """moe_align's offsets and indices, padded parts and all, as they come; the combination by embedding_grad."""
    tokens, top_k, experts, rows, cols = 50, 3, 7, 72, 64
    g = torch.Generator().manual_seed(9)
    x, w = rand(tokens, cols, dtype=torch.bfloat16, seed=1), rand(experts, rows, cols, dtype=torch.bfloat16, seed=2)
    ids = torch.stack([torch.randperm(experts, generator=g)[:top_k] for _ in range(tokens)]).int()
    counts, offsets, index = ds.moe_align(ids.cuda(), experts, 16)
    y = ds.grouped_matmul(x.cuda(), w.cuda(), offsets, index=index, top_k=top_k)
    total = int(offsets[-1])
    owner = torch.full((index.numel(),), -1, dtype=torch.int32, device="cuda")
    owner[:total] = index[:total] // top_k  # padding: tokens, past the last row
    got = ds.embedding_grad(y, owner, tokens, dtype=torch.float32).double().cpu()
    for t in range(tokens):
        each = torch.stack([w[e].double() @ x[t].double() for e in ids[t].long()])
        size = torch.stack([w[e].double().abs() @ x[t].double().abs() for e in ids[t].long()])
        bound = 2 * ro.U * (cols + 8) * size.sum(0) + ro.STEP[torch.bfloat16] * 1.01 * each.abs().sum(0)
        assert ((got[t] - each.sum(0)).abs() <= bound).all(), t


def test_nothing_to_do():
    b = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
    zero = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert ds.grouped_matmul(b(0, 8), b(3, 5, 8), zero).shape == (0, 5)
    assert (ds.grouped_matmul_grad(b(0, 5), b(0, 8), zero) == 0).all()
    out = torch.full((4, 5), 77.0, dtype=torch.bfloat16, device="cuda")
    assert (ds.grouped_matmul(b(4, 8), b(3, 5, 8), zero, out=out) == 77).all()
    off = torch.tensor([0, 1, 1, 4], dtype=torch.int32, device="cuda")
    assert (ds.grouped_matmul(b(4, 0), b(3, 5, 0), off) == 0).all()              # sums of no products
    assert ds.grouped_matmul(b(4, 8), b(3, 0, 8), off).shape == (4, 0)
    none = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    assert (ds.grouped_matmul(b(0, 8), b(3, 5, 8), off, index=none, top_k=2) == 0).all()


def test_offsets_that_are_not_offsets_stay_inside():
    x, w, dy = (rand(*s, dtype=torch.bfloat16, seed=1).cuda() for s in ((100, 40), (4, 48, 40), (100, 48)))
    for bad in ([-9, 50, 20, 1 << 30, 100], [200, 300, 100, -4, -8], [0, 90, 10, 80, 5]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf = torch.full((140, 48), 77.0, dtype=torch.bfloat16, device="cuda")
        ds.grouped_matmul(x, w, off, out=buf[20:120])
        ds.grouped_matmul_grad(dy, x, off)
        torch.cuda.synchronize()
        assert (buf[:20] == 77).all() and (buf[120:] == 77).all()


@pytest.mark.parametrize("lengths", [[5, 0, 30], [400, 0, 700]])
def test_graph_and_streams(lengths):
    offsets, m = setting(lengths, 0, 0)
    x, w, dy = (rand(*s, dtype=torch.bfloat16, seed=1).cuda() for s in ((m, 256), (3, 384, 256), (m, 384)))
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")

    def call(stream=None):
        return (ds.grouped_matmul(x, w, off, stream=stream), ds.grouped_matmul(dy, w, off, transposed=True, stream=stream),
                ds.grouped_matmul_grad(dy, x, off, dtype=torch.float32, stream=stream))

    want = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(call())
        graphs.append(g)
    other = torch.cuda.Stream()
    for _ in range(4):
        for out in outs:
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        eager = call()
        torch.cuda.synchronize()
        for out in (*outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(out, want))


# ---------------------------------------------------------------------------------------------------------------------
# Sizes that take the larger tiles, several tiles to a workgroup, groups of very different lengths; the 64-bit sums on the GPU
# ---------------------------------------------------------------------------------------------------------------------
def big_reference(x, w, dy, offsets, index, top_k, transposed):
    """(y, bound, dw, bound) in 64 bits, from products of whole groups."""
    rows = x if index is None else torch.cat([x, torch.zeros_like(x[:1])])[
        torch.where(index < 0, len(x), torch.div(index, top_k, rounding_mode="floor")).clamp(max=len(x)).long()]
    rows, dy = rows.double(), dy.double()
    y = torch.zeros((len(rows), w.shape[1 if not transposed else 2]), dtype=torch.float64, device="cuda")
    ye, dw = torch.zeros_like(y), torch.zeros((len(w), dy.shape[1], x.shape[1]), dtype=torch.float64, device="cuda")
    dwe = torch.zeros_like(dw)
    for e in range(len(w)):
        part = slice(offsets[e], offsets[e + 1])
        if offsets[e + 1] > offsets[e]:
            m = w[e].double() if transposed else w[e].double().T.contiguous()
            y[part], ye[part] = rows[part] @ m, rows[part].abs() @ m.abs() * (len(m) + 2)
            d = dy[part].T.contiguous()
            dw[e], dwe[e] = d @ rows[part], d.abs() @ rows[part].abs() * (offsets[e + 1] - offsets[e] + 2)
    return y, 2 * ro.U * ye, dw, 2 * ro.U * dwe


def big_close(got, want, err, dtype, what):
    bad = (got.double() - want).abs() > ro.rounded(err, want, dtype)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:4].tolist())


BIG = [(520, 264, [700, 0, 1, 257, 3000] + [130] * 250, 8), (1032, 1024, [2100, 9, 4000, 33, 2050, 0, 500, 8000], 0),
       (264, 520, [5] * 300 + [0] * 20 + [700], 3), (128, 136, [1000, 1, 300], 0), (2056, 1032, [600] * 16, 16),
       (2056, 2056, [600] * 14 + [3000, 0], 2), (1031, 517, [300, 0, 900, 1], 5)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("rows,cols,lengths,behind", BIG, ids=[f"{r}x{c}-{len(g)}" for r, c, g, _ in BIG])
def test_large(rows, cols, lengths, behind, gather, dtype):
    offsets, m = setting(lengths, 0, behind)
    g = torch.Generator(device="cuda").manual_seed(rows)
    rand_ = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    tokens, top_k = (m // 3 + 5, 3) if gather else (m, 1)
    index = choose(m, tokens, top_k, 3).cuda() if gather else None
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    w, dy = rand_(len(lengths), rows, cols), rand_(m, rows)
    end = offsets[-1]
    for transposed in (False, True):
        x = rand_(tokens, rows if transposed else cols)
        kw = dict(index=index, top_k=top_k)
        want, err, dw, dwe = big_reference(x, w, dy if not transposed else rand_(m, 1), offsets, index, top_k, transposed)
        out = torch.full((m, want.shape[1]), 77.0, dtype=dtype, device="cuda")
        ds.grouped_matmul(x, w, off, transposed=transposed, out=out, **kw)
        big_close(out[:end], want[:end], err[:end], dtype, f"transposed {transposed}")
        assert (out[end:] == 77).all()
        if not transposed:
            big_close(ds.grouped_matmul_grad(dy, x, off, **kw), dw, dwe, dtype, "gradient")
            old = torch.randn(dw.shape, generator=g, device="cuda")
            got = ds.grouped_matmul_grad(dy, x, off, out=old.clone(), accumulate=True, **kw)
            big_close(got, dw + old.double(), dwe + 2 * ro.U * old.abs().double(), torch.float32, "added gradient")


def test_most_experts_and_one_more():
    off = torch.arange(2049, dtype=torch.int32, device="cuda")
    x, w = rand(2048, 16, dtype=torch.bfloat16, seed=1).cuda(), rand(2048, 8, 16, dtype=torch.bfloat16, seed=2).cuda()
    want = (x.double()[:, None] * w.double()).sum(2)
    err = 2 * ro.U * 18 * (x.double().abs()[:, None] * w.double().abs()).sum(2)
    big_close(ds.grouped_matmul(x, w, off), want, err, torch.bfloat16, "2,048 experts")
    dy = rand(2048, 8, dtype=torch.bfloat16, seed=3).cuda()
    big_close(ds.grouped_matmul_grad(dy, x, off), dy.double()[:, :, None] * x.double()[:, None], torch.zeros(1, device="cuda"),
              torch.bfloat16, "gradient")
    with pytest.raises(ds.DevscanError):
        ds.grouped_matmul(x, torch.zeros((2049, 8, 16), dtype=torch.bfloat16, device="cuda"),
                          torch.zeros(2050, dtype=torch.int32, device="cuda"))


def test_rows_past_32_bit_offsets():
    """x, y and the matrices each beyond 4 GiB: 2^21 rows of 1,056 columns, two of them used at either end."""
    n, cols, rows = (1 << 21) + 40, 1056, 64
    x = torch.zeros((n, cols), dtype=torch.bfloat16, device="cuda")
    x[:3] = x[-3:] = 1
    w = rand(2, rows, cols, dtype=torch.bfloat16, seed=2).cuda()
    off = torch.tensor([0, n - 20, n], dtype=torch.int32, device="cuda")
    y = ds.grouped_matmul(x, w, off)
    want = w.double().sum(2)
    err = 2 * ro.U * (cols + 2) * w.double().abs().sum(2)
    big_close(y[:3], want[:1].expand(3, -1), err[:1], torch.bfloat16, "first")
    big_close(y[-3:], want[1:].expand(3, -1), err[1:], torch.bfloat16, "last")
    assert (y[3:-3] == 0).all()
    index = torch.tensor([n - 1, 0, n - 2, n], dtype=torch.int32, device="cuda")
    y = ds.grouped_matmul(x, w, torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"), index=index)
    big_close(y[:3], torch.stack([want[0], want[1], want[1]]), err.amax(0, keepdim=True), torch.bfloat16, "index")
    assert (y[3] == 0).all()
    dy = torch.ones((4, rows), dtype=torch.bfloat16, device="cuda")
    dw = ds.grouped_matmul_grad(dy, x, torch.tensor([0, 1, 4], dtype=torch.int32, device="cuda"), index=index)
    assert (dw[0] == 1).all() and (dw[1] == 2).all()


@pytest.mark.parametrize("stride", [8, 11])
def test_offsets_that_name_all_rows_for_each_expert(stride):
    """1,024 times 2^29 rows: more blocks of rows than 31 bits count, of offsets that decrease. Undefined results, all inside."""
    m, guard = 1 << 29, 4096
    x = torch.ones((m * stride,), dtype=torch.bfloat16, device="cuda").view(m, stride)[:, :8]
    w = torch.ones((2048, 8, 8), dtype=torch.bfloat16, device="cuda")
    buf = torch.full((m + 2 * guard, 8), 77.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, m] * 1024 + [0], dtype=torch.int32, device="cuda")
    ds.grouped_matmul(x, w, off, out=buf[guard:-guard])
    assert (buf[:guard] == 77).all() and (buf[-guard:] == 77).all()
    assert bool(((buf == 77) | (buf == 8)).all())


def test_no_rows_of_x():
    """Only padding: rows of zeros, and a gradient of zeros, from an x without rows."""
    x = torch.zeros((0, 24), dtype=torch.bfloat16, device="cuda")
    w, dy = rand(3, 16, 24, dtype=torch.bfloat16, seed=1).cuda(), rand(40, 16, dtype=torch.bfloat16, seed=2).cuda()
    off = torch.tensor([0, 16, 16, 32], dtype=torch.int32, device="cuda")
    index = torch.arange(40, dtype=torch.int32, device="cuda")
    out = torch.full((40, 16), 77.0, dtype=torch.bfloat16, device="cuda")
    y = ds.grouped_matmul(x, w, off, index=index, top_k=2, out=out)
    assert (y[:32] == 0).all() and (y[32:] == 77).all()
    assert (ds.grouped_matmul_grad(dy, x, off, index=index, top_k=2) == 0).all()
    old = torch.ones((3, 16, 24), device="cuda")
    assert (ds.grouped_matmul_grad(dy, x, off, index=index, top_k=2, out=old, accumulate=True) == 1).all()
