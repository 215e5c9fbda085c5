"""The mixture-of-experts router, its gradient and the experts' products on the GPU against the definitions in 64 bits
(tests/model_oracle.py), which also gives the bounds."""
import numpy as np
import pytest
import torch

import model_oracle as mo
import oracle
import primitives_device_scan_amd as ds
from gpu_util import say

pytestmark = pytest.mark.gpu

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def normal(seed, shape, dtype=torch.float32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype)


def masked_logits(seed, tokens, experts, dtype):
    """Logits with ties (few distinct values in 16 bits), experts at -inf, at the type's lowest value and at NaN, and
    tokens with no expert left, one or a few."""
    l = normal(seed, (tokens, experts), dtype, 2.0)
    rng = np.random.default_rng(seed)
    r = torch.from_numpy(rng.random((tokens, experts)))
    l[r < 0.2] = float("-inf")
    l[(r > 0.2) & (r < 0.25)] = float("nan")
    l[(r > 0.25) & (r < 0.3)] = torch.finfo(dtype).min
    l[(r > 0.9)] = 0.5
    l[::7] = float("-inf")
    l[1::7, 1:] = float("-inf")
    l[2::7] = torch.finfo(dtype).min
    l[3::7] = 1.25
    return l


def check_route(l, top_k, score, renorm, scale, bias=None, what=""):
    w, ids = ds.moe_route(l.cuda(), top_k, score=score, renormalize=renorm, scale=scale,
                          bias=None if bias is None else bias.cuda())
    rw, rids = mo.route(l, bias, top_k, score, renorm, float(np.float32(scale)))
    assert np.array_equal(ids.cpu().numpy(), rids), what
    mo.within(w, rw, mo.route_terms(l) * mo.U * np.abs(rw) + 2.0 ** -120, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (1, 2, 2), (3, 5, 5), (17, 8, 2), (33, 60, 4), (9, 64, 6),
                                                  (5, 65, 64), (40, 128, 8), (66, 256, 8), (7, 300, 16), (12, 511, 8)])
def test_route(dtype, score, renorm, tokens, experts, top_k):
    say("route", dtype, score, renorm, tokens, experts, top_k)
    l = normal(tokens + experts, (tokens, experts), dtype, 1.5)
    check_route(l, top_k, score, renorm, 1.0, what="plain")
    check_route(l, top_k, score, renorm, 2.5, normal(5, (experts,), std=0.5), "bias")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("experts,top_k", [(6, 6), (70, 5), (256, 8), (400, 33)])
def test_route_masks_and_ties(dtype, score, experts, top_k):
    l = masked_logits(experts, 50, experts, dtype)
    finite = l.clone()
    finite[~torch.isfinite(finite) | (finite == torch.finfo(dtype).min)] = 0
    # the lowest value of a type is far from the other logits: its scores are exactly 0 and its own rows equal shares,
    # so the bound goes by the other logits
    for renorm in (True, False):
        w, ids = ds.moe_route(l.cuda(), top_k, score=score, renormalize=renorm)
        rw, rids = mo.route(l, None, top_k, score, renorm, 1.0)
        assert np.array_equal(ids.cpu().numpy(), rids)
        mo.within(w, rw, mo.route_terms(finite) * mo.U * np.abs(rw) + 2.0 ** -120, "masked")
    # what cannot be chosen is dropped by the alignment too
    c, o, s = ds.moe_align(ids, experts, 16)
    wc, wo, ws = oracle.moe_align(rids, experts, 16)
    assert np.array_equal(c.cpu().numpy(), wc) and np.array_equal(s.cpu().numpy()[:int(wo[-1])], ws)


def test_route_strides_and_bias_that_switches_off():
    l = normal(1, (30, 50), torch.bfloat16).cuda()[:, 3:36]
    bias = normal(2, (33,))
    bias[4] = float("-inf")
    bias[5] = float("nan")
    w, ids = ds.moe_route(l, 31, bias=bias.cuda())
    rw, rids = mo.route(l, bias, 31, "softmax", True, 1.0)
    assert np.array_equal(ids.cpu().numpy(), rids) and not np.isin(rids, [4, 5]).any()
    mo.within(w, rw, mo.route_terms(l) * mo.U * np.abs(rw) + 2.0 ** -120, "strided")
    w, ids = ds.moe_route(l[:0], 4)
    assert w.shape == (0, 4) and ids.shape == (0, 4)


def test_route_past_32_bit_offsets():
    tokens, experts = 4_300_000, 511          # 2.2G logits
    l = torch.zeros((tokens, experts), dtype=torch.bfloat16, device="cuda")
    l[-2:] = normal(3, (2, experts), torch.bfloat16).cuda()
    w, ids = ds.moe_route(l, 2)
    rw, rids = mo.route(l[-2:], None, 2, "softmax", True, 1.0)
    assert np.array_equal(ids[-2:].cpu().numpy(), rids) and ids[:-2].unique(dim=0).tolist() == [[0, 1]]
    mo.within(w[-2:], rw, mo.route_terms(l[-2:]) * mo.U * np.abs(rw) + 2.0 ** -120, "last tokens")
    dw = torch.zeros((tokens, 2), device="cuda")
    dw[-2:, 0] = 1.0
    got = ds.moe_route_grad(l, ids, dw)
    ref, size = mo.route_grad(mo.f64(l[-2:]), rids, np.array([[1.0, 0.0]] * 2), "softmax", True, 1.0)
    mo.within(got[-2:], ref, 2 * mo.route_terms(l[-2:]) * mo.U * size + mo.rounding(ref, l.dtype), "last gradients")
    assert not bool(got[:-2].any())


def check_route_grad(l, ids, score, renorm, scale, seed, what):
    dw = normal(seed, tuple(ids.shape))
    got = ds.moe_route_grad(l.cuda(), ids.cuda(), dw.cuda(), score=score, renormalize=renorm, scale=scale)
    ref, size = mo.route_grad(mo.f64(l), ids.numpy(), mo.f64(dw), score, renorm, float(np.float32(scale)))
    bound = 2 * mo.route_terms(l) * mo.U * size + mo.rounding(ref, l.dtype)
    return mo.within(got, ref, bound, what)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k", [(1, 1, 1), (4, 3, 2), (33, 60, 4), (5, 65, 64), (21, 256, 8),
                                                  (6, 511, 16)])
def test_route_grad(dtype, score, renorm, tokens, experts, top_k):
    l = normal(tokens * experts, (tokens, experts), dtype, 1.5)
    _, ids = ds.moe_route(l.cuda(), top_k)
    worst = check_route_grad(l, ids.cpu(), score, renorm, 2.5, 3, "chosen ids")
    say("route grad", dtype, score, renorm, tokens, experts, top_k, "worst share of the bound %.2f" % worst)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_masks_and_dropped_ids(score, renorm):
    l = normal(4, (20, 90), torch.float32, 1.5)
    l[:, 3::9] = float("-inf")
    l[5] = float("-inf")
    l[6, 1:] = float("-inf")
    l[7, 8] = float("nan")
    _, ids = ds.moe_route(l.cuda(), 6)
    ids = ids.cpu()
    ids[0, 2] = -1
    ids[1, 1] = 90
    ids[2] = -5
    check_route_grad(l, ids, score, renorm, 1.0, 5, "masked")
    got = ds.moe_route_grad(l.cuda(), ids.cuda(), torch.ones(20, 6, device="cuda"), score=score, renormalize=renorm)
    assert bool((got[:, 3::9] == 0).all()) and bool((got[5] == 0).all()) and bool((got[2] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_grad_against_differences(score, renorm):
    # a symmetric difference of the kernel's own weights along one direction: its error is the step's square times the
    # third derivative (under 20 for these sums of products of scores) and the weights' rounding over the step
    l, d = normal(8, (16, 40)), normal(9, (16, 40))
    step = 2.0 ** -7
    _, ids = ds.moe_route(l.cuda(), 5)
    dw = normal(10, (16, 5))
    grad = mo.f64(ds.moe_route_grad(l.cuda(), ids, dw.cuda(), score=score, renormalize=renorm))

    def along(s):
        p = mo.scores(mo.f64(l + s * d), np.ones((16, 40), bool), score)
        w = np.take_along_axis(p, ids.cpu().numpy().astype(np.int64), 1)
        return w / w.sum(1, keepdims=True) if renorm else w

    slope = ((along(step) - along(-step)) / (2 * step) * mo.f64(dw)).sum(1)
    size = np.abs(mo.f64(dw)).sum(1) * np.abs(mo.f64(d)).max(1) ** 3
    assert bool((np.abs(slope - (grad * mo.f64(d)).sum(1)) <= 20 * step ** 2 * size).all())


# ---------------------------------------------------------------------------------------------------------------------
def layer(seed, tokens, experts, top_k, dim, hidden, dtype, eight=False):
    x = normal(seed, (tokens, dim), dtype)
    w_in, w_out = normal(seed + 1, (experts, 2 * hidden, dim)), normal(seed + 2, (experts, dim, hidden))
    s_in = s_out = None
    if eight:
        w_in, w_out = (32 * w_in).to(torch.float8_e4m3fn), (32 * w_out).to(torch.float8_e4m3fn)
        up = lambda v: -(-v // 128)
        g = torch.Generator().manual_seed(seed + 3)
        s_in = (torch.rand((experts, up(2 * hidden), up(dim)), generator=g) + 0.5) / (32 * dim ** 0.5)
        s_out = (torch.rand((experts, up(dim), up(hidden)), generator=g) + 0.5) / (32 * hidden ** 0.5)
    else:
        w_in, w_out = (w_in * dim ** -0.5).to(dtype), (w_out * hidden ** -0.5).to(dtype)
    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]).astype(np.int32)
    weights = torch.from_numpy(rng.random((tokens, top_k)).astype(np.float32)) + 0.1
    return x, w_in, w_out, torch.from_numpy(ids), weights, s_in, s_out


def on_gpu(x, w_in, w_out, ids, weights, s_in, s_out, **more):
    up = lambda v: None if v is None else v.cuda()
    return ds.moe_experts(x.cuda(), w_in.cuda(), w_out.cuda(), ids.cuda(), weights.cuda(), w_in_scale=up(s_in),
                          w_out_scale=up(s_out), **more)


def check_experts(args, what):
    got = on_gpu(*args)
    ref, bound = mo.experts(*args)
    worst = mo.within(got, ref, bound, what)
    assert torch.equal(got, on_gpu(*args)), "two runs differ"
    say(what, "worst share of the bound %.2f" % worst)
    return got


@pytest.mark.parametrize("dtype,eight", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True),
                                         (torch.float16, True)])
@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden", [
    (1, 1, 1, 1, 1), (1, 4, 2, 64, 32), (1, 300, 8, 128, 48), (2, 3, 3, 7, 5), (5, 8, 2, 130, 33), (16, 4, 1, 256, 128),
    (17, 2, 2, 96, 64), (33, 2, 1, 200, 136), (40, 6, 6, 129, 65), (70, 2, 2, 320, 80), (64, 40, 4, 63, 144),
    (130, 3, 2, 72, 40), (12, 300, 3, 384, 272), (1, 9, 9, 2048, 768), (3, 40, 5, 320, 208), (4, 64, 16, 144, 1040),
    (2, 20, 10, 528, 512), (64, 8, 1, 64, 48), (65, 8, 1, 64, 48), (16, 300, 4, 64, 48), (13, 70, 5, 64, 48), (4, 4, 1, 16, 16), (20, 5, 3, 160, 48), (9, 1, 1, 80, 304), (90, 4, 2, 256, 96)])
def test_experts(dtype, eight, tokens, experts, top_k, dim, hidden):
    say("experts", dtype, eight, tokens, experts, top_k, dim, hidden)
    check_experts(layer(tokens + dim, tokens, experts, top_k, dim, hidden, dtype, eight),
                  f"{tokens} tokens, {top_k} of {experts}, {dim} x {hidden}")


@pytest.mark.parametrize("dtype,eight", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden", [(40, 1, 1, 64, 32), (100, 1, 1, 144, 48), (300, 2, 1, 272, 160),
                                                            (600, 1, 1, 128, 64), (257, 2, 2, 80, 304),
                                                            (129, 4, 4, 192, 128), (200, 3, 1, 1040, 16)])
def test_experts_many_tokens(dtype, eight, tokens, experts, top_k, dim, hidden):
    # the waves of a workgroup split an expert's tokens: up to 16, 32 and 64 to a wave, and blocks of the most
    check_experts(layer(tokens, tokens, experts, top_k, dim, hidden, dtype, eight), f"{tokens} tokens, {experts} experts")


@pytest.mark.parametrize("eight", [False, True])
def test_experts_one_crowded_among_many(eight):
    # enough experts for every wave to have its own rows, one of them with most of the tokens
    x, w_in, w_out, ids, weights, s_in, s_out = layer(31, 180, 130, 2, 272, 1040, torch.bfloat16, eight)
    ids[:150, 0] = 77
    ids[:40, 1] = 3
    ids[150:, 1] = 129
    check_experts((x, w_in, w_out, ids, weights, s_in, s_out), "crowded")


@pytest.mark.parametrize("eight", [False, True])
def test_experts_wide_enough_for_whole_waves(eight):
    # many experts and rows: every wave streams its own rows over the whole depth
    check_experts(layer(3, 24, 64, 8, 544, 1040, torch.bfloat16, eight), "many experts")


@pytest.mark.parametrize("dtype,eight", [(torch.bfloat16, False), (torch.float16, False), (torch.bfloat16, True)])
@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden", [(1, 8, 4, 256, 512), (8, 8, 2, 256, 512),
                                                            (24, 4, 1, 256, 512)])
def test_experts_are_as_exact_as_the_output(dtype, eight, tokens, experts, top_k, dim, hidden):
    # h is held in two halves, so the error is the output's own rounding and that of 32-bit sums, not one more rounding
    args = layer(tokens + 77, tokens, experts, top_k, dim, hidden, dtype, eight)
    ref, _ = mo.experts(*args)
    off = np.linalg.norm(mo.f64(on_gpu(*args)) - ref)
    own = np.linalg.norm(mo.f64(torch.from_numpy(ref).to(dtype)) - ref)
    assert off <= 1.1 * own, (off, own)


def test_experts_few_tokens_dropped_and_repeated_choices():
    x, w_in, w_out, ids, weights, _, _ = layer(21, 3, 40, 9, 96, 64, torch.bfloat16)
    ids[0] = -1
    ids[1, 4:] = 40
    ids[1, 1] = ids[1, 0]
    ids[2, 8] = -(1 << 31)
    weights[1, 2] = 0.0
    got = check_experts((x, w_in, w_out, ids, weights, None, None), "few tokens")
    assert bool((got[0] == 0).all())
    x[1, 5] = float("inf")
    x[2] = float("nan")
    got = on_gpu(x, w_in, w_out, ids, weights, None, None)
    assert bool((got[0] == 0).all()) and not bool(torch.isfinite(got[1].float()).all()) and bool((got[2] != got[2]).all())


def test_experts_dropped_choices_duplicates_and_weights():
    x, w_in, w_out, ids, weights, _, _ = layer(5, 20, 6, 4, 80, 48, torch.bfloat16)
    ids[0] = -1
    ids[1] = 6
    ids[2, 1] = -7
    ids[3] = 2                   # the same expert four times
    ids[4, 0], ids[4, 1] = 1 << 30, -(1 << 31)
    weights[5] = 0.0
    weights[6] = -1.5
    got = check_experts((x, w_in, w_out, ids, weights, None, None), "dropped")
    assert bool((got[0] == 0).all()) and bool((got[1] == 0).all()) and bool((got[5] == 0).all())
    ids[:] = -1
    assert bool((on_gpu(x, w_in, w_out, ids, weights, None, None) == 0).all())


def test_experts_all_tokens_on_one_expert_and_most_assignments():
    x, w_in, w_out, ids, weights, _, _ = layer(6, 200, 5, 1, 64, 32, torch.float16)
    ids[:] = 3
    check_experts((x, w_in, w_out, ids, weights, None, None), "one expert")
    args = layer(7, 1024, 16, 8, 16, 8, torch.bfloat16)      # 8,192 assignments
    check_experts(args, "most assignments")
    with pytest.raises(ds.DevscanError) as e:
        on_gpu(*layer(8, 1025, 16, 8, 16, 8, torch.bfloat16))
    assert e.value.status == ds.DS_ERR_TOO_LARGE


def test_experts_special_values_stay_with_their_token():
    x, w_in, w_out, ids, weights, _, _ = layer(9, 40, 3, 2, 72, 40, torch.bfloat16)
    clean = on_gpu(x, w_in, w_out, ids, weights, None, None)
    x[4] = float("nan")
    x[9, 3] = float("inf")
    got = on_gpu(x, w_in, w_out, ids, weights, None, None)
    keep = torch.ones(40, dtype=torch.bool)
    keep[[4, 9]] = False
    assert torch.equal(got[keep.cuda()], clean[keep.cuda()])
    assert bool((got[4] != got[4]).all()) and not bool(torch.isfinite(got[9].float()).all())


def test_experts_strides_offsets_and_streams():
    x, w_in, w_out, ids, weights, _, _ = layer(10, 30, 4, 2, 100, 60, torch.bfloat16)
    ref, bound = mo.experts(x, w_in, w_out, ids, weights)
    wide = torch.zeros(30, 140, dtype=torch.bfloat16, device="cuda")
    wide[:, 7:107] = x.cuda()
    flat_in = torch.zeros(w_in.numel() + 3, dtype=torch.bfloat16, device="cuda")
    flat_in[3:] = w_in.flatten().cuda()          # weights that start off any 16-byte boundary
    room = torch.full((30, 110), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = ds.moe_experts(wide[:, 7:107], flat_in[3:].view(w_in.shape), w_out.cuda(), ids.cuda(), weights.cuda(),
                         out=room[:, 4:104], stream=s)
    torch.cuda.synchronize()
    mo.within(got, ref, bound, "strided")
    assert bool((room[:, :4] == 7).all()) and bool((room[:, 104:] == 7).all())
    assert ds.moe_experts(x[:0].cuda(), w_in.cuda(), w_out.cuda(), ids[:0].cuda(), weights[:0].cuda()).shape == (0, 100)


def test_experts_past_32_bit_offsets():
    # 4.8G values of w_in; only the last expert is used
    experts, dim, hidden = 1200, 1024, 2048
    w_in = torch.zeros((experts, 2 * hidden, dim), dtype=torch.bfloat16, device="cuda")
    w_out = torch.zeros((experts, dim, hidden), dtype=torch.bfloat16, device="cuda")
    x, a, b, _, weights, _, _ = layer(11, 3, 1, 1, dim, hidden, torch.bfloat16)
    w_in[-1], w_out[-1] = a[0].cuda(), b[0].cuda()
    got = ds.moe_experts(x.cuda(), w_in, w_out, torch.full((3, 1), experts - 1, dtype=torch.int32).cuda(), weights.cuda())
    ref, bound = mo.experts(x, a, b, torch.zeros(3, 1, dtype=torch.int32), weights)
    mo.within(got, ref, bound, "last expert")


def test_router_and_experts_in_a_graph():
    tokens, experts, top_k, dim, hidden = 20, 16, 4, 128, 64
    x, w_in, w_out, _, _, _, _ = (v.cuda() if v is not None else None
                                  for v in layer(12, tokens, experts, top_k, dim, hidden, torch.bfloat16))
    logits = normal(1, (tokens, experts)).cuda()

    def step():
        weights, ids = ds.moe_route(logits, top_k)
        return weights, ids, ds.moe_experts(x, w_in, w_out, ids, weights), \
            ds.moe_route_grad(logits, ids, weights)

    cap = torch.cuda.Stream()
    cap.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(cap):
        step()
    cap.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=cap):
        got = step()
    for r in range(4):
        logits.copy_(normal(30 + r, (tokens, experts)))
        x.copy_(normal(40 + r, (tokens, dim), torch.bfloat16))
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), f"replay {r}"


def test_refused_allocation_then_success():
    args = layer(13, 4, 4, 2, 64, 32, torch.bfloat16)
    s = torch.cuda.Stream()  # a stream with no workspace yet
    torch.cuda.synchronize()
    ds.lib.ds_fail_next_allocations(1)
    try:
        with pytest.raises(ds.DevscanError) as e:
            on_gpu(*args, stream=s)
        assert e.value.status == ds.DS_ERR_OUT_OF_MEMORY
    finally:
        ds.lib.ds_fail_next_allocations(0)
    torch.cuda.synchronize()
    got = on_gpu(*args, stream=s)
    torch.cuda.synchronize()
    ref, bound = mo.experts(*args)
    mo.within(got, ref, bound, "after a refused allocation")


def test_refusals_on_the_gpu():
    x, w_in, w_out, ids, weights, _, _ = (v.cuda() if v is not None else None
                                          for v in layer(14, 4, 4, 2, 64, 32, torch.bfloat16))
    f = ds.moe_experts
    scale = torch.ones(4, 1, 1, device="cuda")
    for bad in (lambda: f(x, w_in[:, :63], w_out, ids, weights), lambda: f(x, w_in, w_out[:3], ids, weights),
                lambda: f(x, w_in.transpose(1, 2), w_out, ids, weights), lambda: f(x, w_in, w_out, ids[:3], weights),
                lambda: f(x, w_in, w_out, ids, weights[:, :1]), lambda: f(x.t(), w_in, w_out, ids, weights),
                lambda: f(x, w_in, w_out, ids, weights, w_in_scale=scale, w_out_scale=scale),
                lambda: f(x, w_in.to(torch.float8_e4m3fn), w_out.to(torch.float8_e4m3fn), ids, weights),
                lambda: ds.moe_route(weights, 3), lambda: ds.moe_route(weights, 1, score="other"),
                lambda: ds.moe_route(weights, 1, bias=torch.zeros(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(x.float(), w_in, w_out, ids, weights), lambda: f(x, w_in.half(), w_out, ids, weights),
                lambda: f(x, w_in, w_out, ids.long(), weights), lambda: f(x, w_in, w_out, ids, weights.half()),
                lambda: ds.moe_route(ids, 1), lambda: ds.moe_route_grad(weights, ids, weights.half())):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ds.DevscanError):
        f(x, w_in, w_out, ids, weights, out=x)
