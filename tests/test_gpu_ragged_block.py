"""The operators on ragged batches together, as a recurrent layer with a mixture of experts behind it uses them: a batch of
requests of different lengths forward and back, then single tokens from a pool of states. Each operator is held against its
64-bit definition on the inputs that it had."""
import numpy as np
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
DIM, HIDDEN, EXPERTS, TOP_K, ROWS, PAGE, POOL, BLOCK = 192, 96, 12, 3, 500, 16, 11, 16
CONTEXT, NEW, SPARE = [0, 5, 16, 40, 0, 7], [37, 1, 16, 0, 290, 3], 9


def rand(*shape, seed, std=1.0, dtype=BF):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Layer:
    def __init__(self):
        self.table, self.gates = rand(ROWS, DIM, seed=1), rand(ROWS, DIM, seed=2, std=2.0)
        self.router = rand(1, EXPERTS, DIM, seed=3, std=DIM ** -0.5)
        self.w_in = rand(EXPERTS, 2 * HIDDEN, DIM, seed=4, std=DIM ** -0.5)
        self.w_out = rand(EXPERTS, DIM, HIDDEN, seed=5, std=HIDDEN ** -0.5)
        self.pool = rand(POOL, DIM, seed=6, dtype=torch.float32)
        self.places = ints([7, 2, 9, 0, 10, 4])
        self.tables = torch.full((len(NEW), 30), -1, dtype=torch.int32)
        taken = 0
        for r, c in enumerate(CONTEXT):
            held = -(-c // PAGE)
            self.tables[r, :held] = torch.arange(100 + taken, 100 + taken + held)
            taken += held
        self.tables = self.tables.cuda()
        self.free, self.count = torch.arange(64, dtype=torch.int32, device="cuda").flip(0).contiguous(), ints([60])

    def experts(self, h):
        """Everything behind the recurrence, and what its backward pass needs."""
        k = {"h": h}
        k["logits"] = ds.grouped_matmul(h, self.router, ints_of(0, len(h)))
        k["weights"], k["chosen"] = ds.moe_route(k["logits"].float(), TOP_K)
        _, k["off"], k["index"] = ds.moe_align(k["chosen"], EXPERTS, BLOCK)
        m = k["index"].numel()
        inside = torch.arange(m, device="cuda") < k["off"][-1]
        there = inside & (k["index"] >= 0) & (k["index"] < len(h) * TOP_K)  # else padding of a block
        at = torch.where(there, k["index"], 0).long()
        k["owner"] = torch.where(there, at // TOP_K, -1).int()
        k["share"] = torch.where(there, k["weights"].reshape(-1)[at], 0.0)[:, None]
        k["u"] = ds.grouped_matmul(h, self.w_in, k["off"], index=k["index"], top_k=TOP_K,
                                   out=torch.zeros((m, 2 * HIDDEN), dtype=BF, device="cuda"))
        gate, up = k["u"].float().split(HIDDEN, 1)
        k["a"] = (torch.nn.functional.silu(gate) * up).to(BF)
        k["e"] = ds.grouped_matmul(k["a"], self.w_out, k["off"], out=torch.zeros((m, DIM), dtype=BF, device="cuda"))
        k["y"] = ds.embedding_grad((k["e"].float() * k["share"]).to(BF), k["owner"], len(h), dtype=torch.float32)
        return k

    def prefill(self, ids):
        n = ids.numel()
        offsets, slots, positions, left = ds.page_slots(ints_of(*CONTEXT), ints_of(*NEW), self.tables, self.free, self.count,
                                                        PAGE, n)
        x, gate = ds.embedding(self.table, ids), ds.embedding(self.gates, ids)
        initial = self.pool[self.places.long()]
        h, final = ds.gated_scan(gate, x, offsets, mix=True, initial=initial, out=torch.zeros_like(x))
        k = self.experts(h)
        k.update(offsets=offsets, slots=slots, positions=positions, left=left, x=x, gate=gate, initial=initial, final=final)
        return k

    def backward(self, k, ids, dy):
        """The gradients of both tables, the matrices and the initial states, from that of y."""
        g = {}
        spread = torch.where(k["owner"][:, None] >= 0, dy[k["owner"].long().clamp(min=0)], 0.0)
        g["de"] = (spread * k["share"]).to(BF)
        g["w_out"] = ds.grouped_matmul_grad(g["de"], k["a"], k["off"])
        g["da"] = ds.grouped_matmul(g["de"], self.w_out, k["off"], transposed=True, out=torch.zeros_like(k["a"]))
        gate, up = k["u"].float().split(HIDDEN, 1)
        s, da = torch.sigmoid(gate), g["da"].float()
        g["du"] = torch.cat([da * up * s * (1 + gate * (1 - s)), da * gate * s], 1).to(BF)
        g["w_in"] = ds.grouped_matmul_grad(g["du"], k["h"], k["off"], index=k["index"], top_k=TOP_K, dtype=torch.float32)
        g["dhe"] = ds.grouped_matmul(g["du"], self.w_in, k["off"], transposed=True, out=torch.zeros_like(k["e"]))
        g["dh"] = ds.embedding_grad(g["dhe"], k["owner"], len(k["h"]))
        g["gate"], g["x"], g["initial"] = ds.gated_scan_grad(k["gate"], k["h"], g["dh"], k["offsets"], x=k["x"], mix=True,
                                                             initial=k["initial"])
        inside = torch.where(torch.arange(ids.numel(), device="cuda") < k["offsets"][-1], ids, -1)
        g["table"] = ds.embedding_grad(g["x"], inside, ROWS, dtype=torch.float32)
        return g


_CONST = {}


def ints_of(*x):
    """int32 constants on the GPU, made once: a recorded call has them already."""
    if x not in _CONST:
        _CONST[x] = ints(list(x))
    return _CONST[x]


def close(got, want, err, dtype, what, rows=slice(None)):
    bad = ((got.detach().double().cpu() - want).abs() > ro.rounded(err, want, dtype))[rows]
    assert not bad.any(), (what, int(bad.sum()))


def check_experts(layer, k):
    off, index = k["off"].tolist(), k["index"].cpu()
    part = slice(0, off[-1])
    want, err = ro.grouped(k["h"].cpu(), layer.router.cpu(), [0, len(k["h"])], None, 1, False)
    close(k["logits"], want, err, BF, "logits")
    want, err = ro.grouped(k["h"].cpu(), layer.w_in.cpu(), off, index, TOP_K, False)
    close(k["u"], want, err, BF, "first product", part)
    want, err = ro.grouped(k["a"].cpu(), layer.w_out.cpu(), off, None, 1, False)
    close(k["e"], want, err, BF, "second product", part)
    # the sum over a token's choices: TOP_K products rounded to bfloat16, then added in 32 bits
    e, share, owner = k["e"].double().cpu(), k["share"].double().cpu(), k["owner"].cpu()
    y, size = (torch.zeros((len(k["h"]), DIM), dtype=torch.float64) for _ in range(2))
    live = owner >= 0
    y.index_add_(0, owner[live].long(), (e * share)[live])
    size.index_add_(0, owner[live].long(), (e * share)[live].abs())
    assert ((k["y"].double().cpu() - y).abs() <= (ro.STEP[BF] + 8 * ro.U) * size + ro.TINY[BF] * TOP_K).all()
    assert live.sum() == len(k["h"]) * TOP_K


@pytest.fixture(scope="module")
def setting():
    n = sum(NEW) + SPARE
    ids = torch.from_numpy(np.random.default_rng(3).integers(0, ROWS, n)).cuda()
    return ids, rand(n, DIM, seed=8, dtype=torch.float32)


def test_batch_forward_and_back(setting):
    ids, dy = setting
    layer = Layer()
    before = layer.tables.cpu().numpy()
    k = layer.prefill(ids)
    live = sum(NEW)
    ref = ro.pages(np.array(CONTEXT), np.array(NEW), before, layer.free.cpu().numpy(), 60, PAGE, len(ids))
    assert k["offsets"].tolist() == ref[0].tolist() and k["left"].item() == ref[3]
    assert np.array_equal(k["slots"].cpu().numpy(), ref[1]) and np.array_equal(k["positions"].cpu().numpy(), ref[2])
    assert np.array_equal(layer.tables.cpu().numpy(), ref[4])
    offsets = k["offsets"].tolist()
    h, final, he, fe = ro.scan(k["gate"].cpu(), k["x"].cpu(), offsets, "sigmoid", True, k["initial"].cpu())
    close(k["h"], h, he, BF, "h", slice(0, live))
    assert (k["h"][live:] == 0).all()
    close(k["final"], final, fe, torch.float32, "final")
    check_experts(layer, k)

    g = layer.backward(k, ids, dy)
    off, index = k["off"].tolist(), k["index"].cpu()
    part = slice(0, off[-1])
    close(g["w_out"], *ro.grouped_grad(g["de"].cpu(), k["a"].cpu(), off, None, 1, None), BF, "w_out")
    close(g["w_in"], *ro.grouped_grad(g["du"].cpu(), k["h"].cpu(), off, index, TOP_K, None), torch.float32, "w_in")
    close(g["da"], *ro.grouped(g["de"].cpu(), layer.w_out.cpu(), off, None, 1, True), BF, "da", part)
    close(g["dhe"], *ro.grouped(g["du"].cpu(), layer.w_in.cpu(), off, None, 1, True), BF, "dh of the experts", part)
    want, err = ro.scan_grad(k["gate"].cpu(), k["h"].cpu(), g["dh"].cpu(), k["x"].cpu(), offsets, "sigmoid", True,
                             k["initial"].cpu(), None)
    close(g["gate"], want[0], err[0], BF, "dgate", slice(0, live))
    close(g["x"], want[1], err[1], BF, "dx", slice(0, live))
    close(g["initial"], want[2], err[2], torch.float32, "dinitial")
    table, size = (torch.zeros((ROWS, DIM), dtype=torch.float64) for _ in range(2))
    dx = g["x"][:live].double().cpu()
    table.index_add_(0, ids[:live].cpu(), dx)
    size.index_add_(0, ids[:live].cpu(), dx.abs())
    assert ((g["table"].double().cpu() - table).abs() <= 2 * ro.U * live * size).all()


def test_single_tokens_after_the_batch(setting):
    """Two steps of every request from the pool that the batch's last states went into: the batch one token longer."""
    ids, _ = setting
    layer = Layer()
    k = layer.prefill(ids)
    layer.pool[layer.places.long()] = k["final"]
    pool = layer.pool.cpu()
    context, count = ints_of(*[c + n for c, n in zip(CONTEXT, NEW)]), k["left"]
    for step in range(2):
        tables = layer.tables.cpu().numpy()
        ref = ro.pages(context.cpu().numpy(), np.ones(6, int), tables, layer.free.cpu().numpy(), count.item(), PAGE, 6)
        offsets, slots, positions, left = ds.page_slots(context, ints_of(1, 1, 1, 1, 1, 1), layer.tables, layer.free, count,
                                                        PAGE, 6)
        assert offsets.tolist() == list(range(7)) and np.array_equal(slots.cpu().numpy(), ref[1])
        assert torch.equal(positions, context) and left.item() == ref[3]
        assert np.array_equal(layer.tables.cpu().numpy(), ref[4])
        assert len(set(slots.tolist())) == 6 and not set(slots.tolist()) & set(k["slots"].tolist())
        tok = ids[step * 6:step * 6 + 6]
        x, gate = ds.embedding(layer.table, tok), ds.embedding(layer.gates, tok)
        h = ds.gated_step(gate, x, layer.pool, layer.places, mix=True)
        want, pool64, he, se = ro.step(gate.cpu(), x.cpu(), pool, layer.places.cpu(), "sigmoid", True)
        close(h, want, he, BF, "h")
        close(layer.pool, pool64, se, torch.float32, "states")
        pool = layer.pool.cpu()
        check_experts(layer, layer.experts(h))
        context, count = context + 1, left


def test_recorded(setting):
    """Forward and back in one graph, replayed with other batches and the program's own work in between."""
    ids, dy = setting
    layer = Layer()
    batches = [ids, ids.flip(0).contiguous(), ids.roll(11)]

    def run(tok):
        k = layer.prefill(tok)
        g = layer.backward(k, tok, dy)
        return [k["y"], k["final"], k["slots"], g["table"], g["w_in"], g["w_out"], g["gate"][:sum(NEW)], g["initial"]]

    want = [[t.clone() for t in run(b)] for b in batches]
    fixed = ids.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(fixed)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = run(fixed)
    for r in range(6):
        fixed.copy_(batches[r % 3])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[r % 3])), r
        assert all(torch.equal(a, b) for a, b in zip(run(batches[(r + 1) % 3]), want[(r + 1) % 3])), r
    assert not ds.query_timeout()
