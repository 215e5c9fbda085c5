"""Scratch of the language-model operators and HIP graphs: every recorded call holds scratch of its own."""
import pytest
import torch

import primitives_device_scan_amd as ds
from test_gpu_embedding import normal, token_ids
from test_gpu_moe_layer import layer

pytestmark = pytest.mark.gpu


def recorded(fn, stream):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        out = fn()
    return g, out


@pytest.mark.parametrize("n", [900, 9001, 270_000])
def test_capture_on_a_stream_of_its_own_needs_no_call_before(n):
    # the usual recipe: one call on a side stream, then torch's own capture stream
    rows = 500
    ids, dout = token_ids(1, n, rows).cuda(), normal(2, (n, 8), torch.float32).cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ds.embedding_grad(dout, ids, rows)
    side.synchronize()
    g, got = recorded(lambda: ds.embedding_grad(dout, ids, rows), torch.cuda.Stream())
    for r in range(3):
        dout.copy_(normal(20 + r, (n, 8), torch.float32))
        want = ds.embedding_grad(dout, ids, rows)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), f"replay {r}"


@pytest.mark.parametrize("tokens", [3, 200])
def test_experts_captured_on_a_stream_of_its_own(tokens):
    args = [v if v is None else v.cuda() for v in layer(12, tokens, 16, 4, 128, 64, torch.bfloat16)]
    run = lambda: ds.moe_experts(*args[:5])
    g, got = recorded(run, torch.cuda.Stream())
    for r in range(3):
        args[0].copy_(normal(40 + r, (tokens, 128), torch.bfloat16))
        want = run()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want), f"replay {r}"


def test_two_graphs_of_one_stream_and_eager_calls_run_side_by_side():
    # gradients and experts recorded on one stream, replayed on two others while the stream itself runs the same calls
    cap, a, b = (torch.cuda.Stream() for _ in range(3))
    rows, n = 700, 20_000
    work = []
    for k in (0, 1, 2):
        ids, dout = token_ids(k, n, rows).cuda(), normal(k, (n, 520), torch.bfloat16).cuda()
        args = [v if v is None else v.cuda() for v in layer(k, 256, 32, 4, 512, 256, torch.bfloat16)][:5]
        work.append(lambda ids=ids, dout=dout, args=args: (ds.embedding_grad(dout, ids, rows), ds.moe_experts(*args)))
    want = [w() for w in work]
    torch.cuda.synchronize()
    with torch.cuda.stream(cap):
        work[0]()
    cap.synchronize()
    graphs = [recorded(w, cap) for w in work[:2]]
    torch.cuda.synchronize()
    for r in range(20):
        for out in (graphs[0][1], graphs[1][1]):
            for t in out:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(a):
                graphs[0][0].replay()
            with torch.cuda.stream(b):
                graphs[1][0].replay()
            with torch.cuda.stream(cap):
                eager = work[2]()
        torch.cuda.synchronize()
        for got, ref in zip((graphs[0][1], graphs[1][1], eager), want):
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1]), f"round {r}"


@pytest.mark.parametrize("n,dim", [(129, 40), (9001, 24), (270_000, 8)])
def test_gradient_in_scratch_of_the_callers(n, dim):
    rows = 300
    ids, dout = token_ids(5, n, rows).cuda(), normal(6, (n, dim), torch.float32).cuda()
    want = ds.embedding_grad(dout, ids, rows)
    room = ds.lib.ds_embedding_grad_scratch_bytes(ds.DS_FP32, n, rows, dim)
    assert room > 0 and ds.lib.ds_embedding_grad_scratch_bytes(ds.DS_FP32, 128, rows, dim) == 0
    buf = torch.full((room + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(want)
    st = ds.lib.ds_embedding_grad_scratch(ds.DS_FP32, dout.data_ptr(), dim, ids.data_ptr(), 8, n, 1.0, ds.DS_FP32,
                                          got.data_ptr(), rows, dim, dim, 0, buf.data_ptr() + 256, room,
                                          torch.cuda.current_stream().cuda_stream)
    assert st == ds.DS_OK and torch.equal(got, want)
    assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + room:] == 0x5A).all())


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("tokens,experts,top_k,dim,hidden,off", [(1, 4, 2, 64, 32, 0), (70, 300, 2, 72, 40, 0),
                                                                 (300, 2, 1, 272, 160, 0), (300, 2, 1, 272, 160, 1)])
def test_experts_in_scratch_of_the_callers(eight, tokens, experts, top_k, dim, hidden, off):
    # off: weights that start off any 16-byte boundary, which another launch serves
    x, w_in, w_out, ids, weights, s_in, s_out = (v if v is None else v.cuda() for v in
                                                 layer(4, tokens, experts, top_k, dim, hidden, torch.bfloat16, eight))
    if off:
        w_in = torch.cat([w_in.flatten()[:off], w_in.flatten()])[off:].view(w_in.shape)
    want = ds.moe_experts(x, w_in, w_out, ids, weights, w_in_scale=s_in, w_out_scale=s_out)
    kind = ds.DS_FP8_E4M3 if eight else ds.DS_BF16
    room = ds.lib.ds_moe_experts_scratch_bytes(kind, tokens, dim, experts, hidden, top_k)
    buf = torch.full((room + 512,), 0x5A, dtype=torch.uint8, device="cuda")
    got = torch.empty_like(want)
    p = lambda t: None if t is None else t.data_ptr()
    st = ds.lib.ds_moe_experts_scratch(ds.DS_BF16, p(x), tokens, dim, dim, kind, p(w_in), p(s_in), p(w_out), p(s_out),
                                       experts, hidden, p(ids), p(weights), top_k, p(got), dim, buf.data_ptr() + 256,
                                       room, torch.cuda.current_stream().cuda_stream)
    assert st == ds.DS_OK and torch.equal(got, want)
    assert bool((buf[:256] == 0x5A).all()) and bool((buf[256 + room:] == 0x5A).all())
