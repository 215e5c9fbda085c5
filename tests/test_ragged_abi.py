"""The entry points on ragged batches refuse bad arguments on the host before any HIP call, and the binding's functions say
what is wrong (CPU only)."""
import pytest
import torch

import primitives_device_scan_amd as ds
from test_model_ops_abi import A, B, BF16, BIG, C, D, DTY, E, F, F32, FP16, FP8, G, H, INV, MIS, OK, OVL, lib  # noqa: F401

I, J, K = (0x7F8000000000 + (i << 32) for i in range(3))


def test_gated_scan_refusals(lib):
    def f(dtype=F32, gate=A, gs=8, x=B, xs=8, t=10, d=8, off=C, n=3, form=2, mix=0, init=D, h=E, hs=8, final=F, ws=None, room=0):
        return lib.ds_gated_scan(dtype, gate, gs, x, xs, t, d, off, n, form, mix, init, h, hs, final, ws, room, None)
    assert f(dtype=0) == DTY and f(dtype=FP8) == DTY and f(dtype=-1) == DTY
    assert f(t=-1) == INV and f(d=-1) == INV and f(n=-1) == INV and f(form=3) == INV and f(form=-1) == INV and f(mix=2) == INV
    assert f(gs=7) == INV and f(xs=7) == INV and f(hs=7) == INV
    assert f(off=None) == INV                                     # three sequences need offsets
    assert f(gate=None) == INV and f(x=None) == INV and f(h=None) == INV
    assert f(d=0, gs=0, xs=0, hs=0, gate=None, x=None, h=None) == OK and f(n=0) == OK
    assert f(gate=A + 2) == MIS and f(x=B + 1) == MIS and f(off=C + 2) == MIS and f(init=D + 2) == MIS and f(final=F + 1) == MIS
    assert f(h=A + 32) == OVL and f(h=B) == OVL and f(final=D) == OVL and f(final=E + 64) == OVL and f(h=C - 64) == OVL
    assert f(t=1 << 31) == BIG and f(d=1 << 31, gs=1 << 31, xs=1 << 31, hs=1 << 31) == BIG and f(n=1 << 31) == BIG
    assert f(t=1, hs=(1 << 20) + 1) == BIG
    assert f(ws=G, room=-1) == INV and f(ws=G + 8, room=1 << 40) == MIS
    big = dict(dtype=BF16, gate=0x100000000000, x=0x200000000000, h=0x300000000000, t=1 << 16, d=4096, gs=4096, xs=4096, hs=4096)
    need = lib.ds_gated_scan_scratch_bytes(BF16, 0, 1 << 16, 4096)
    assert need > 0 and f(**big, ws=G, room=need - 1) == INV and f(**big, ws=0x100000000100, room=need) == OVL


def test_gated_scan_scratch_bytes(lib):
    f = lib.ds_gated_scan_scratch_bytes
    assert f(F32, 0, 0, 8) == 0 and f(F32, 1, 8, 0) == 0 and f(0, 0, 8, 8) == 0 and f(F32, 0, 1 << 31, 8) == 0
    assert f(BF16, 0, 1, 2048) == 0 and f(BF16, 1, 4000, 2048) > 0


def test_gated_scan_grad_refusals(lib):
    def f(dtype=BF16, gate=A, gs=8, h=B, hs=8, dh=C, dhs=8, x=D, xs=8, t=10, d=8, off=E, n=3, form=2, mix=1, init=F, dfinal=G,
          dg=H, dgs=8, dx=I, dxs=8, dinit=J, ws=None, room=0):
        return lib.ds_gated_scan_grad(dtype, gate, gs, h, hs, dh, dhs, x, xs, t, d, off, n, form, mix, init, dfinal, dg, dgs,
                                      dx, dxs, dinit, ws, room, None)
    assert f(dtype=1) == DTY
    assert f(t=-1) == INV and f(form=5) == INV and f(mix=-1) == INV and f(off=None) == INV
    for name in ("gs", "hs", "dhs", "xs", "dgs", "dxs"):
        assert f(**{name: 7}) == INV, name
    for name in ("gate", "h", "dh", "x", "dg", "dx"):
        assert f(**{name: None}) == INV, name
    assert f(mix=0, x=None, xs=0, n=0) == OK                       # x is not read without mix
    assert f(mix=0, x=None, xs=0, gate=None) == INV
    for name, at in (("gate", A), ("h", B), ("dh", C), ("x", D), ("dg", H), ("dx", I)):
        assert f(**{name: at + 1}) == MIS, name
    for name, at in (("off", E), ("init", F), ("dfinal", G), ("dinit", J)):
        assert f(**{name: at + 2}) == MIS, name
    assert f(dg=A) == OVL and f(dx=B + 16) == OVL and f(dg=I) == OVL and f(dinit=G) == OVL and f(dx=D) == OVL
    assert f(t=1 << 31) == BIG


def test_gated_step_refusals(lib):
    def f(dtype=FP16, gate=A, gs=8, x=B, xs=8, n=4, d=8, slots=C, state=D, pool=9, ss=8, form=1, mix=0, h=E, hs=8):
        return lib.ds_gated_step(dtype, gate, gs, x, xs, n, d, slots, state, pool, ss, form, mix, h, hs, None)
    assert f(dtype=3) == DTY
    assert f(n=-1) == INV and f(d=-1) == INV and f(pool=-1) == INV and f(form=3) == INV and f(mix=3) == INV
    assert f(gs=7) == INV and f(xs=7) == INV and f(ss=7) == INV and f(hs=7) == INV
    assert f(slots=None, pool=3) == INV                            # no state for the last row
    assert f(gate=None) == INV and f(x=None) == INV and f(state=None) == INV and f(h=None) == INV
    assert f(n=0, gate=None, x=None, h=None) == OK and f(d=0, gs=0, xs=0, ss=0, hs=0) == OK
    assert f(gate=A + 1) == MIS and f(slots=C + 2) == MIS and f(state=D + 2) == MIS
    assert f(h=A) == OVL and f(h=D + 8) == OVL and f(state=B) == OVL and f(state=C - 64) == OVL
    assert f(n=1 << 31) == BIG and f(pool=1 << 31) == BIG and f(n=(1 << 16) + 1) == BIG


def test_grouped_refusals(lib):
    def f(dtype=BF16, x=A, xr=20, xs=16, w=B, e=3, rows=24, cols=16, tr=0, off=C, m=30, index=D, k=2, y=E, ys=24):
        return lib.ds_grouped_matmul(dtype, x, xr, xs, w, e, rows, cols, tr, off, m, index, k, y, ys, None)
    assert f(dtype=F32) == DTY and f(dtype=FP8) == DTY and f(dtype=0) == DTY
    assert f(xr=-1) == INV and f(e=-1) == INV and f(e=2049) == INV and f(rows=-1) == INV and f(cols=-1) == INV and f(m=-1) == INV
    assert f(tr=2) == INV and f(k=0) == INV and f(xs=15) == INV and f(ys=23) == INV and f(tr=1) == INV  # a row of x is 24 long then
    assert f(index=None) == INV                                    # 20 rows for a batch of 30
    for name in ("x", "w", "off", "y"):
        assert f(**{name: None}) == INV, name
    assert f(e=0) == OK and f(m=0, index=None) == OK and f(rows=0, ys=0) == OK
    assert f(x=A + 1) == MIS and f(w=B + 1) == MIS and f(off=C + 2) == MIS and f(index=D + 2) == MIS and f(y=E + 1) == MIS
    assert f(y=A) == OVL and f(y=B + 64) == OVL and f(y=C) == OVL and f(y=D) == OVL
    assert f(m=1 << 31) == BIG and f(xr=1 << 31) == BIG and f(cols=(1 << 20) + 1, xs=1 << 21) == BIG


def test_grouped_grad_refusals(lib):
    def f(dtype=FP16, dy=A, m=30, dys=24, x=B, xr=20, xs=16, off=C, e=3, index=D, k=2, rows=24, cols=16, gd=F32, dw=E, acc=0):
        return lib.ds_grouped_matmul_grad(dtype, dy, m, dys, x, xr, xs, off, e, index, k, rows, cols, gd, dw, acc, None)
    assert f(dtype=F32) == DTY and f(gd=BF16) == DTY and f(gd=1) == DTY
    assert f(m=-1) == INV and f(acc=2) == INV and f(dys=23) == INV and f(xs=15) == INV and f(index=None) == INV and f(k=-1) == INV
    for name in ("dy", "x", "off", "dw"):
        assert f(**{name: None}) == INV, name
    assert f(e=0) == OK and f(rows=0, dys=0) == OK and f(cols=0, xs=0) == OK and f(m=0, acc=1) == OK
    assert f(dy=A + 1) == MIS and f(dw=E + 2) == MIS and f(dw=E + 1, gd=FP16) == MIS
    assert f(dw=A) == OVL and f(dw=B) == OVL and f(dw=D + 4) == OVL
    assert f(m=1 << 31) == BIG and f(rows=(1 << 20) + 1, dys=1 << 21) == BIG


def test_page_slots_refusals(lib):
    def f(ctx=A, new=B, r=5, tab=C, w=8, ts=8, free=D, cap=50, cnt=E, page=16, off=F, slots=G, pos=H, t=40, left=I):
        return lib.ds_page_slots(ctx, new, r, tab, w, ts, free, cap, cnt, page, off, slots, pos, t, left, None)
    assert f(r=-1) == INV and f(w=-1) == INV and f(ts=7) == INV and f(cap=-1) == INV and f(page=0) == INV and f(t=-1) == INV
    for name in ("ctx", "new", "tab", "free", "cnt", "off", "slots", "pos", "left"):
        assert f(**{name: None}) == INV, name
    for name, at in (("ctx", A), ("new", B), ("tab", C), ("free", D), ("cnt", E), ("off", F), ("pos", H), ("left", I)):
        assert f(**{name: at + 2}) == MIS, name
    assert f(slots=G + 4) == MIS
    assert f(tab=D) == OVL and f(off=A) == OVL and f(slots=C) == OVL and f(pos=G) == OVL and f(left=E) == OVL
    assert f(r=1 << 31) == BIG and f(t=1 << 31) == BIG and f(cap=1 << 31) == BIG


def test_the_binding_refuses_on_the_host():
    x = torch.ones(4, 8)
    i = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ds.gated_scan(x, x), lambda: ds.gated_scan_grad(x, x, x), lambda: ds.gated_step(x, x, x),
                 lambda: ds.grouped_matmul(x.bfloat16(), torch.ones(3, 8, 8), i), lambda: ds.page_slots(i, i, i.view(1, 4), i, i, 4, 4),
                 lambda: ds.grouped_matmul_grad(x.bfloat16(), x.bfloat16(), i)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda t: ds.gated_scan(t, x), lambda t: ds.gated_scan(x, x, initial=t), lambda t: ds.gated_scan_grad(x, t, x),
                 lambda t: ds.gated_scan_grad(x, x, x, dfinal=t), lambda t: ds.gated_step(x, x, t),
                 lambda t: ds.grouped_matmul(t, x, i), lambda t: ds.grouped_matmul(x, t, i), lambda t: ds.grouped_matmul_grad(t, x, i)):
        with pytest.raises(ValueError, match="requires grad"):
            call(torch.ones(4, 8, requires_grad=True))
    with pytest.raises(TypeError):
        ds.grouped_matmul(x, torch.ones(3, 8, 8), i)


@pytest.mark.gpu
def test_the_binding_refuses():
    f = lambda *s, d=torch.float32: torch.ones(s, dtype=d, device="cuda")
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    x, b = f(4, 8), f(4, 8, d=torch.bfloat16)
    bad = [
        (ValueError, lambda: ds.gated_scan(f(4, 9), x)), (TypeError, lambda: ds.gated_scan(b, x)),
        (TypeError, lambda: ds.gated_scan(f(4, 8, d=torch.float64), f(4, 8, d=torch.float64))),
        (ValueError, lambda: ds.gated_scan(x, x, form="tanh")), (ValueError, lambda: ds.gated_scan(x, x, i(0))),
        (TypeError, lambda: ds.gated_scan(x, x, i(3).long())), (ValueError, lambda: ds.gated_scan(x, x, i(3), initial=f(3, 8))),
        (TypeError, lambda: ds.gated_scan(b, b, initial=f(1, 8, d=torch.bfloat16))), (ValueError, lambda: ds.gated_scan(x, x, out=f(5, 8))),
        (ValueError, lambda: ds.gated_scan(x[:1].expand(4, 8), x)), (ValueError, lambda: ds.gated_scan(f(8, 4).t(), x)),
        (ds.DevscanError, lambda: ds.gated_scan(x, x, out=x)),
        (ValueError, lambda: ds.gated_scan_grad(x, x, x, mix=True)), (ValueError, lambda: ds.gated_scan_grad(x, x, f(3, 8))),
        (ValueError, lambda: ds.gated_scan_grad(x, x, x, dfinal=f(2, 8))),
        (ValueError, lambda: ds.gated_step(x, x, f(3, 8))), (TypeError, lambda: ds.gated_step(b, b, b)),
        (ValueError, lambda: ds.gated_step(x, x, f(9, 8), i(3))), (ValueError, lambda: ds.gated_step(x, x, f(9, 7))),
        (ds.DevscanError, lambda: ds.gated_step(x, x, x)),
        (TypeError, lambda: ds.grouped_matmul(b, f(2, 5, 8), i(3))), (ValueError, lambda: ds.grouped_matmul(b, f(2, 5, 8, d=torch.bfloat16), i(4))),
        (ValueError, lambda: ds.grouped_matmul(b, f(2, 5, 7, d=torch.bfloat16), i(3))),
        (ValueError, lambda: ds.grouped_matmul(b, f(2, 5, 8, d=torch.bfloat16), i(3), transposed=True)),
        (ValueError, lambda: ds.grouped_matmul(b, f(2, 5, 8, d=torch.bfloat16), i(3), index=i(6), top_k=0)),
        (TypeError, lambda: ds.grouped_matmul(b, f(2, 5, 8, d=torch.bfloat16), i(3), out=f(4, 5))),
        (ValueError, lambda: ds.grouped_matmul_grad(b, f(5, 8, d=torch.bfloat16), i(3))),
        (ValueError, lambda: ds.grouped_matmul_grad(b, b, i(3), accumulate=True)),
        (TypeError, lambda: ds.grouped_matmul_grad(b, b, i(3), dtype=torch.float16)),
        (ValueError, lambda: ds.grouped_matmul_grad(b, b, i(3), out=f(2, 8, 7))),
        (ValueError, lambda: ds.page_slots(i(3), i(4), i(3, 2), i(5), i(1), 4, 4)), (ValueError, lambda: ds.page_slots(i(3), i(3), i(2, 2), i(5), i(1), 4, 4)),
        (TypeError, lambda: ds.page_slots(i(3), i(3), i(3, 2).long(), i(5), i(1), 4, 4)),
        (ValueError, lambda: ds.page_slots(i(3), i(3), i(3, 2), i(5), i(2), 4, 4)), (ValueError, lambda: ds.page_slots(i(3), i(3), i(3, 2), i(5), i(1), 0, 4)),
        (ValueError, lambda: ds.page_slots(i(3), i(3), i(3, 2), i(5), i(1), 4, -1)),
    ]
    for k, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {k} was not refused")
