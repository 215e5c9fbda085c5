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
