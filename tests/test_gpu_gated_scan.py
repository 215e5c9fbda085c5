"""The gated recurrence, its gradient and its step on the GPU against their 64-bit definitions, within the bounds that count
their roundings; rows outside the sequences stay as they were; every run gives the same bits."""
import pytest
import torch

import primitives_device_scan_amd as ds
import ragged_oracle as ro

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# (tokens, dim, offsets): one token, odd sizes, rows before and behind the sequences, empty ones, more steps than one tile
SHAPES = [(1, 1, None), (1, 130, [0, 1]), (5, 7, [0, 0, 3, 3, 5, 5]), (64, 64, None), (37, 65, [2, 9, 9, 30]),
          (300, 129, [0, 1, 2, 130, 131, 300]), (1000, 33, None), (515, 200, [0, 256, 512, 515]), (3, 1030, None),
          (2100, 17, [5, 2099]), (130, 8, list(range(131)))]
IDS = [f"{n}x{d}-{'one' if o is None else len(o) - 1}" for n, d, o in SHAPES]


def make(n, d, dtype, form, seed=0, stride=None):
    g = torch.Generator().manual_seed(seed)
    gate = torch.randn((n, d), generator=g) * 2 + 2 * torch.randn((1, d), generator=g) + 1.5
    if form == "log":
        gate = -torch.log1p(torch.exp(-gate))
    elif form == "decay":
        gate = torch.sigmoid(gate) * (1 - 2 * (torch.rand((n, d), generator=g) < 0.1).float())
    return gate.to(dtype), torch.randn((n, d), generator=g).to(dtype), torch.randn((n, d), generator=g).to(dtype)


def states(offsets, d, seed):
    return torch.randn((1 if offsets is None else len(offsets) - 1, d), generator=torch.Generator().manual_seed(seed))


def wide(x, extra, lead=0):
    """x on the GPU as a matrix whose rows lie `extra` elements further apart, `lead` elements into their memory."""
    n, d = x.shape
    buf = torch.full((n * (d + extra) + lead + extra,), 77.0, dtype=x.dtype, device="cuda")
    view = buf[lead:lead + n * (d + extra)].view(n, d + extra)[:, :d]
    view.copy_(x)
    return view


def off(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")


def close(got, want, err, dtype, what):
    got = got.detach().double().cpu()
    there = ~want.isnan()
    bad = (got - want).abs() > ro.rounded(err, want, dtype)
    assert not (bad & there).any(), (what, int((bad & there).sum()), float((got - want).abs()[there].max()))


def check_scan(n, d, offsets, dtype, form, mix, initial, seed=0, extra=(0, 0, 0), lead=0):
    gate, x, _ = make(n, d, dtype, form, seed)
    init = states(offsets, d, seed + 1) if initial else None
    want = ro.scan(gate, x, offsets, form, mix, init)
    out = wide(torch.full((n, d), 77.0).to(dtype), extra[2], lead)
    args = (wide(gate, extra[0], lead), wide(x, extra[1], lead), off(offsets))
    kw = dict(form=form, mix=mix, initial=None if init is None else init.cuda())
    h, final = ds.gated_scan(*args, out=out, **kw)
    assert h is out and final.dtype == torch.float32
    close(h, want[0], want[2], dtype, "h")
    close(final, want[1], want[3], torch.float32, "final")
    outside = want[0].isnan()
    assert (h.cpu()[outside] == 77).all(), "rows outside the sequences"
    again = ds.gated_scan(*args, **kw)
    assert torch.equal(again[0].cpu()[~outside], h.cpu()[~outside]) and torch.equal(again[1], final)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", [("decay", False), ("log", True), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_scan(shape, form, mix, dtype):
    check_scan(*shape, dtype, form, mix, initial=(shape[0] % 2 == 1))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("extra,lead", [((8, 16, 24), 0), ((1, 3, 5), 0), ((1, 0, 2), 3)])
def test_scan_strides(extra, lead, dtype):
    check_scan(150, 96, [0, 70, 150], dtype, "sigmoid", True, True, extra=extra, lead=lead)
    check_scan(33, 257, None, dtype, "log", False, True, extra=extra, lead=lead)


@pytest.mark.parametrize("form,mix", [("log", False), ("sigmoid", True)])
def test_long_memory(form, mix):
    """Gates that keep their state for 1e5 steps: 1 - a has to be exact, a alone does not hold it."""
    n, d = 6000, 16
    gate = torch.full((n, d), 11.5 if form == "sigmoid" else -1e-5)
    x = torch.ones((n, d))
    init = torch.ones((1, d))
    want = ro.scan(gate, x, None, form, mix, init)
    h, final = ds.gated_scan(gate.cuda(), x.cuda(), form=form, mix=mix, initial=init.cuda())
    close(h, want[0], want[2], torch.float32, "h")
    close(final, want[1], want[3], torch.float32, "final")


def test_extreme_gates():
    """Gates that open and shut entirely, and values next to a reset of a large state."""
    gate = torch.tensor([[30.0, -30.0, float("inf"), -float("inf"), 200.0, -200.0, 0.0, 88.0]]).repeat(6, 1)
    gate[3] = -float("inf")
    x = torch.full((6, 8), 1e-3)
    x[0] = 1e6
    for mix in (False, True):
        want = ro.scan(gate, x, None, "sigmoid", mix, None)
        h, final = ds.gated_scan(gate.cuda(), x.cuda(), form="sigmoid", mix=mix)
        close(h, want[0], want[2], torch.float32, "h")
        assert (h[3].cpu() == x[3]).all(), "a shut gate forgets everything"
    log = torch.where(gate > 0, 0.0, gate)
    want = ro.scan(log, x, None, "log", False, None)
    close(ds.gated_scan(log.cuda(), x.cuda(), form="log")[0], want[0], want[2], torch.float32, "log")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_value_stays_in_its_sequence_and_channel(bad):
    n, d, offsets = 700, 130, [0, 300, 300, 420, 700]
    gate, x, dh = make(n, d, torch.float32, "sigmoid")
    want = ro.scan(gate, x, offsets, "sigmoid", True, None)
    ref = ro.scan_grad(gate, want[0], dh, x, offsets, "sigmoid", True, None, None)
    spoilt, spoilt_dh = x.clone(), dh.clone()
    spoilt[310, 5] = spoilt_dh[310, 5] = bad
    h, _ = ds.gated_scan(gate.cuda(), spoilt.cuda(), off(offsets), mix=True)
    hit = torch.zeros((n, d), dtype=torch.bool)
    hit[310:420, 5] = True
    assert not torch.isfinite(h.cpu()[hit]).any() and torch.isfinite(h.cpu()[~hit]).all()
    dgate, dx, _ = ds.gated_scan_grad(gate.cuda(), want[0].float().cuda(), spoilt_dh.cuda(), off(offsets), x=x.cuda(), mix=True)
    hit[:] = False
    hit[300:311, 5] = True
    assert not torch.isfinite(dx.cpu()[hit]).any() and torch.isfinite(dx.cpu()[~hit]).all()
    close(torch.where(hit, 0.0, dx.cpu()), torch.where(hit, 0.0, ref[0][1]), ref[1][1], torch.float32, "dx")
    # what lies in rows outside all sequences is not read into them
    outside = x.clone()
    outside[:10] = outside[690:] = bad
    h, final = ds.gated_scan(gate.cuda(), outside.cuda(), off([10, 300, 690]), mix=True)
    assert torch.isfinite(h[10:690]).all() and torch.isfinite(final).all()


def check_grad(n, d, offsets, dtype, form, mix, given, seed=0, extra=0, lead=0):
    gate, x, dh = make(n, d, dtype, form, seed)
    init, dfinal = (states(offsets, d, seed + 1), states(offsets, d, seed + 2)) if given else (None, None)
    h = ro.scan(gate, x, offsets, form, mix, init)[0].nan_to_num().to(dtype)
    want, err = ro.scan_grad(gate, h, dh, x, offsets, form, mix, init, dfinal)
    cuda = lambda t: None if t is None else t.cuda()
    args = [wide(t, extra + i, lead) for i, t in enumerate((gate, h, dh, x))]
    kw = dict(x=args[3] if mix else None, form=form, mix=mix, initial=cuda(init), dfinal=cuda(dfinal))
    got = ds.gated_scan_grad(*args[:3], off(offsets), **kw)
    for g, w, e, t, name in zip(got, want, err, (dtype, dtype, torch.float32), ("dgate", "dx", "dinitial")):
        close(g, w, e, t, name)
    again = ds.gated_scan_grad(*args[:3], off(offsets), **kw)
    inside = ~want[0].isnan()
    assert all(torch.equal(a.cpu()[inside], g.cpu()[inside]) for a, g in zip(again[:2], got[:2]))
    assert torch.equal(again[2], got[2])


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", [("decay", True), ("log", False), ("log", True), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_grad(shape, form, mix, dtype):
    check_grad(*shape, dtype, form, mix, given=(shape[0] % 2 == 1))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("extra,lead", [(8, 0), (1, 0), (3, 1)])
def test_grad_strides(extra, lead, dtype):
    check_grad(150, 96, [0, 70, 150], dtype, "sigmoid", True, True, extra=extra, lead=lead)
    check_grad(33, 257, None, dtype, "log", False, True, extra=extra, lead=lead)


@pytest.mark.parametrize("form,mix", [("decay", False), ("log", True), ("sigmoid", True)])
def test_grad_matches_differences_of_the_scan(form, mix):
    n, d, offsets = 12, 5, [0, 5, 12]
    gate, x, dh = make(n, d, torch.float32, form, seed=5)
    init, dfinal = states(offsets, d, 6), states(offsets, d, 7)

    def loss(gate, x, init):
        h, final = ds.gated_scan(gate.cuda(), x.cuda(), off(offsets), form=form, mix=mix, initial=init.cuda())
        return float((h.cpu().double() * dh).sum() + (final.cpu().double() * dfinal).sum())

    h, _ = ds.gated_scan(gate.cuda(), x.cuda(), off(offsets), form=form, mix=mix, initial=init.cuda())
    got = ds.gated_scan_grad(gate.cuda(), h, dh.cuda(), off(offsets), x=x.cuda(), form=form, mix=mix, initial=init.cuda(),
                             dfinal=dfinal.cuda())
    # a difference over 2 step of sums of about 100 terms of size 1: 2e-5 / (2 step) of rounding, step^2 of curvature
    step = 2.0 ** -6
    for i, grad in enumerate(got):
        for k in (0, 7, 3):
            at = [gate, x, init]
            e = torch.zeros_like(at[i]).reshape(-1)
            e[k] = step
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + e.view(at[i].shape), at[i] - e.view(at[i].shape)
            want = (loss(*up) - loss(*down)) / (2 * step)
            assert abs(float(grad.reshape(-1)[k]) - want) < 2e-3 + 20 * step ** 2, (i, k)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", [("decay", False), ("log", True), ("sigmoid", True)])
@pytest.mark.parametrize("rows,dim,pool,slots", [
    (1, 1, 1, None), (3, 1000, 5, None), (64, 256, 64, None), (1, 77, 3, [2]),
    (7, 130, 9, [8, -1, 0, 3, 9, 1, 2]), (6, 40, 4, [1, 2, 1, 1, -5, 2]), (300, 33, 20, [i * i % 23 for i in range(300)])])
def test_step(rows, dim, pool, slots, form, mix, dtype):
    gate, x, _ = make(rows, dim, dtype, form)
    state = states(list(range(pool + 1)), dim, 1)
    want = ro.step(gate, x, state, slots, form, mix)
    for extra in (0, 3):
        mine = wide(state, extra)
        h = ds.gated_step(wide(gate, extra), wide(x, extra), mine,
                          None if slots is None else torch.tensor(slots, dtype=torch.int32, device="cuda"), form=form, mix=mix)
        close(h, want[0], want[2], dtype, "h")
        close(mine, want[1], want[3], torch.float32, "state")
        unused = [k for k in range(pool) if k not in (range(rows) if slots is None else slots)]
        assert torch.equal(mine.cpu()[unused], state[unused])


def test_steps_are_the_scan():
    """Tokens one by one through a pool give what the scan gives for the whole sequences."""
    n, d, seqs = 20, 96, 3
    gate, x, _ = make(n * seqs, d, torch.float32, "sigmoid")
    gate, x = gate.cuda(), x.cuda()
    h, final = ds.gated_scan(gate, x, off([0, n, 2 * n, 3 * n]), mix=True)
    pool = torch.zeros((5, d), device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    for t in range(n):
        got = ds.gated_step(gate[t::n], x[t::n], pool, slots, mix=True)
        assert torch.allclose(got, h[t::n], rtol=1e-5, atol=1e-6)
    assert torch.allclose(pool[slots.long()], final, rtol=1e-5, atol=1e-6)


def test_nothing_to_do():
    e = torch.empty((0, 8), device="cuda")
    h, final = ds.gated_scan(e, e, off([0, 0, 0]), initial=torch.ones((2, 8), device="cuda"))
    assert h.shape == (0, 8) and (final == 1).all()
    assert ds.gated_scan(e, e)[1].abs().sum() == 0
    d = ds.gated_scan_grad(e, e, e, off([0, 0]), dfinal=torch.full((1, 8), 3.0, device="cuda"))
    assert d[0].shape == (0, 8) and (d[2] == 3).all()
    z = torch.empty((4, 0), device="cuda")
    assert ds.gated_scan(z, z)[0].shape == (4, 0) and ds.gated_scan(torch.ones(4, 8).cuda(), torch.ones(4, 8).cuda(), off([0]))[1].shape == (0, 8)
    assert ds.gated_step(e, e, torch.ones((2, 8), device="cuda")).shape == (0, 8)


def test_offsets_that_are_not_offsets_stay_inside():
    """Bad offsets give undefined results, but nothing outside the matrices is touched."""
    n, d = 200, 64
    gate, x, dh = (t.cuda() for t in make(n, d, torch.float32, "sigmoid"))
    for bad in ([-5, 100, 50, 1 << 30], [300, 400, -1], [0, 150, 20, 190, 10]):
        buf = torch.full((n + 64, d), 77.0, device="cuda")
        ds.gated_scan(gate, x, off(bad), out=buf[32:32 + n])
        ds.gated_scan_grad(gate, x, dh, off(bad))
        torch.cuda.synchronize()
        assert (buf[:32] == 77).all() and (buf[32 + n:] == 77).all()


@pytest.mark.parametrize("n", [40, 3000])
def test_graph_and_streams(n):
    d, offsets = 200, [0, 1, n // 3, n]
    gate, x, dh = (t.cuda() for t in make(n, d, torch.bfloat16, "sigmoid"))
    o = off(offsets)
    state = torch.zeros((8, d), device="cuda")

    def call():
        h, final = ds.gated_scan(gate, x, o, mix=True)
        return h, final, *ds.gated_scan_grad(gate, h, dh, o, x=x, mix=True)

    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, final = ds.gated_scan(gate, x, o, mix=True, stream=side)
    rest = ds.gated_scan_grad(gate, h, dh, o, x=x, mix=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h, final, *rest), want))
    graphs, outs = [], []
    for _ in range(2):  # two graphs of one stream, replayed side by side
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(call())
            ds.gated_step(gate[:5], x[:5], state)
        graphs.append(g)
    other = torch.cuda.Stream()
    for _ in range(4):
        for out in outs:
            for t in out:
                t.zero_()
        eager = call()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0].replay()
        with torch.cuda.stream(other):
            graphs[1].replay()
        torch.cuda.synchronize()
        for out in (*outs, eager):
            assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert not ds.query_timeout()


# ---------------------------------------------------------------------------------------------------------------------
# Many tiles and groups of tiles, the caller's scratch, a wait that gives up, matrices and states beyond 4 GiB
# ---------------------------------------------------------------------------------------------------------------------
LONG = [0, 7000, 7000, 7129, 20_021]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("form,mix", [("log", False), ("sigmoid", True)])
def test_many_tiles(form, mix, dtype):
    check_scan(20_030, 136, LONG, dtype, form, mix, initial=True)
    check_grad(20_030, 136, LONG, dtype, form, mix, given=True)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_scratch_of_the_callers(dtype):
    n, d, code = 3001, 136, {torch.float32: ds.DS_FP32, torch.bfloat16: ds.DS_BF16, torch.float16: ds.DS_FP16}[dtype]
    gate, x, dh = (t.cuda() for t in make(n, d, dtype, "sigmoid"))
    want, final = ds.gated_scan(gate, x)
    grads = ds.gated_scan_grad(gate, want, dh)
    stream = torch.cuda.current_stream().cuda_stream
    for grad in (0, 1):
        room = ds.lib.ds_gated_scan_scratch_bytes(code, grad, n, d)
        assert room > 0 and ds.lib.ds_gated_scan_scratch_bytes(code, grad, 5, d) == 0
        buf = torch.full((room + 512,), 0x5A, dtype=torch.uint8, device="cuda")
        outs = [torch.empty_like(t) for t in ((want, final) if grad == 0 else grads)]
        for r in (room, room - 1):
            if grad == 0:
                st = ds.lib.ds_gated_scan(code, gate.data_ptr(), d, x.data_ptr(), d, n, d, None, 1, ds.GATES["sigmoid"], 0,
                                          None, outs[0].data_ptr(), d, outs[1].data_ptr(), buf.data_ptr() + 256, r, stream)
            else:
                st = ds.lib.ds_gated_scan_grad(code, gate.data_ptr(), d, want.data_ptr(), d, dh.data_ptr(), d, None, 0, n, d,
                                               None, 1, ds.GATES["sigmoid"], 0, None, None, outs[0].data_ptr(), d,
                                               outs[1].data_ptr(), d, outs[2].data_ptr(), buf.data_ptr() + 256, r, stream)
            assert (st == ds.DS_OK) == (r == room)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, (want, final) if grad == 0 else grads))
        assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + room:] == 0x5A).all())


def test_after_a_give_up():
    """Every wave ends; what the wait would have given is NaN, what needs no wait is right, and so is the next call."""
    n, d, offsets = 9000, 256, [0, 5000, 5100, 9000]
    gate, x, dh = (t.cuda() for t in make(n, d, torch.float32, "sigmoid"))
    o = off(offsets)
    want = ds.gated_scan(gate, x, o)
    grads = ds.gated_scan_grad(gate, want[0], dh, o)
    ds.set_spin_limit(1)
    try:
        got, got_grads = ds.gated_scan(gate, x, o), ds.gated_scan_grad(gate, want[0], dh, o)
        torch.cuda.synchronize()
    finally:
        ds.set_spin_limit(0)
    for a, b in zip((*got, *got_grads), (*want, *grads)):
        assert bool((torch.isnan(a) | (a == b)).all())
    assert torch.equal(got[0][:128], want[0][:128]) and torch.equal(got[0][5000:5100], want[0][5000:5100])
    again = (*ds.gated_scan(gate, x, o), *ds.gated_scan_grad(gate, want[0], dh, o))
    assert all(torch.equal(a, b) for a, b in zip(again, (*want, *grads)))


def test_matrices_and_states_past_4_gib():
    """Gates of 0 forget everything: h is x, dx is dh and dgate dh h_{t-1}, bit for bit."""
    n, d = (1 << 21) + 40, 1056
    x = torch.randn((n, d), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda", dtype=torch.bfloat16)
    gate = torch.zeros_like(x)
    h, final = ds.gated_scan(gate, x, off([0, n - 200, n]), form="decay")
    assert torch.equal(h, x) and torch.equal(final[1], x[-1].float())
    dgate, dx, _ = ds.gated_scan_grad(gate, h, x, off([0, n - 200, n]), form="decay")
    assert torch.equal(dx, x)
    before = torch.cat([torch.zeros_like(h[:1]), h[n - 300:n - 201], torch.zeros_like(h[:1]), h[n - 200:-1]])
    assert torch.equal(dgate[n - 299:], (x[n - 299:].float() * before[1:].float()).to(torch.bfloat16))
    del h, dgate, dx, gate
    pool = torch.zeros(((1 << 20) + 5, 1030), device="cuda")
    pool[-1], pool[0] = 3.0, 5.0
    got = ds.gated_step(torch.ones((3, 1030), device="cuda"), torch.ones((3, 1030), device="cuda"), pool,
                        torch.tensor([len(pool) - 1, 0, len(pool) - 1], dtype=torch.int32, device="cuda"), form="decay")
    assert got[:, 0].tolist() == [4.0, 6.0, 5.0] and (got == got[:, :1]).all()
    assert (pool[-1] == 5).all() and (pool[0] == 6).all() and pool.sum().item() == 11 * 1030


def test_step_of_many_rows():
    """The most rows that name slots: 2,000 of them slot 5's, the last ones too; one row more is refused."""
    n = 65536
    slots = torch.arange(10, 10 + n, dtype=torch.int32)
    slots[100:n:33] = 5
    slots[-1] = 5
    gate, x, _ = make(n, 24, torch.float32, "sigmoid", 3)
    state = states([0] * (n + 21), 24, 4)
    pool = state.cuda()
    h = ds.gated_step(gate.cuda(), x.cuda(), pool, slots.cuda())
    rows = (slots == 5).nonzero()[:, 0]
    want, after, he, se = ro.step(gate[rows], x[rows], state, slots[rows], "sigmoid", False)
    close(h[rows.cuda()], want, he, torch.float32, "rows of one slot")
    close(pool[5:6], after[5:6], se[5:6], torch.float32, "its state")
    a = torch.sigmoid(gate.double())
    other = slots != 5
    want = (a * state.double()[slots.long()] + x.double())[other]
    size = (a * state.double()[slots.long()].abs() + x.double().abs())[other]
    assert ((h.double().cpu()[other] - want).abs() <= (2 * float(gate.abs().max()) + 12) * ro.U * size).all()
    with pytest.raises(ds.DevscanError):
        ds.gated_step(torch.ones((n + 1, 8), device="cuda"), torch.ones((n + 1, 8), device="cuda"), pool[:, :8],
                      torch.zeros(n + 1, dtype=torch.int32, device="cuda"))
