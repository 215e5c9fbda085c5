"""Scratch of the caller's: sizes, and refusals on the host before any HIP call (CPU only)."""
from test_model_ops_abi import A, B, BF16, BIG, C, D, E, F, F32, FP8, G, INV, MIS, OVL, lib  # noqa: F401


def test_embedding_grad_scratch_refusals(lib):  # noqa: F811
    size = lib.ds_embedding_grad_scratch_bytes
    need = size(F32, 1000, 100, 8)

    def f(n=1000, rows=100, scratch=D, have=need):
        return lib.ds_embedding_grad_scratch(BF16, A, 8, B, 4, n, 1.0, F32, C, rows, 8, 8, 0, scratch, have, None)
    assert need > 1000 * 8 and size(F32, 128, 100, 8) == 0 and size(F32, 2000, 100, 8) > need
    assert size(0, 1000, 100, 8) == 0 and size(F32, -1, 100, 8) == 0 and size(F32, 1 << 31, 100, 8) == 0
    assert size(F32, 1000, 1 << 27, 8) == 0
    assert f(have=need - 1) == INV and f(have=-1) == INV and f(scratch=None, have=-1) == INV
    assert f(scratch=D + 16) == MIS
    assert f(scratch=A + 256) == OVL and f(scratch=B) == OVL and f(scratch=C - 256) == OVL
    assert f(n=1 << 31) == BIG


def test_moe_experts_scratch_refusals(lib):  # noqa: F811
    size = lib.ds_moe_experts_scratch_bytes
    need = size(BF16, 4, 64, 8, 32, 2)

    def f(scratch=G, have=need):
        return lib.ds_moe_experts_scratch(BF16, A, 4, 64, 64, BF16, B, None, C, None, 8, 32, D, E, 2, F, 64, scratch,
                                          have, None)
    assert need > 0 and size(FP8, 4, 64, 8, 32, 2) > 0 and size(BF16, 0, 64, 8, 32, 2) == 0
    assert size(BF16, 4097, 64, 8, 32, 2) == 0 and size(BF16, 1 << 62, 64, 8, 32, 2) == 0 and size(BF16, 4, 64, 8193, 32, 2) == 0
    assert f(have=64) == INV and f(have=-1) == INV
    assert f(scratch=G + 128) == MIS
    for p in (A, B, C, D, E, F):
        assert f(scratch=p) == OVL
