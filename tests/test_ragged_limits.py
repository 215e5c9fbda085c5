"""The largest batches that the grouped products take (CPU only): their kernels count rows, with those of a tile or a stage
past the last one, in 32 bits. A call that gets past the limit's check is refused for a pointer instead."""
import pytest

from test_model_ops_abi import A, B, BF16, BIG, C, D, E, F32, MIS, lib  # noqa: F401

MOST = (1 << 31) - 512


@pytest.mark.parametrize("index", [None, D], ids=["rows", "indexed"])
@pytest.mark.parametrize("transposed", [0, 1])
def test_products(lib, index, transposed):
    def f(m, y):
        return lib.ds_grouped_matmul(BF16, A, (1 << 31) - 1, 8, B, 3, 8, 8, transposed, C, m, index, 2, y, 8, None)
    assert f(MOST, E + 1) == MIS and f(MOST + 1, E + 1) == BIG and f((1 << 31) - 1, E) == BIG


@pytest.mark.parametrize("index", [None, D], ids=["rows", "indexed"])
def test_gradient(lib, index):
    def f(m, dw):
        return lib.ds_grouped_matmul_grad(BF16, A, m, 8, B, (1 << 31) - 1, 8, C, 3, index, 2, 8, 8, F32, dw, 0, None)
    assert f(MOST, E + 2) == MIS and f(MOST + 1, E + 2) == BIG and f((1 << 31) - 1, E) == BIG


def test_row_arithmetic_fits_32_bits():
    """At the limit no sum of the kernels' row arithmetic passes 2^31 - 1, whatever rows the group starts from."""
    for high in (64, 128, 256):
        for first in (0, 1, high - 1, high, MOST - 1):
            rows = MOST - first
            blocks = (rows + high - 1) // high
            assert rows + high - 1 < 1 << 31
            assert first + (blocks - 1) * high + high - 1 < 1 << 31   # the last tile's last row, before it is cut to the group
    stages = (MOST + 31) // 32
    assert (stages + 4 + 1) * 32 < 1 << 31                            # rows ahead of the last stage
