"""Sizes at the limits of the mixture-of-experts entry points, before any HIP
call."""
import pytest

from conftest import gpu_available
from test_abi_moe import ERR_DEVICE, ERR_NULL, ERR_SHAPE, OK, bwd, codes, lib  # noqa: F401

ROW, COL = 0, 2


@pytest.mark.parametrize("rows", ["rows", "tokens"])
def test_column_major_scales_count_their_padding(lib, rows):  # noqa: F811
    """One row takes four words of each column: 2^30 columns are past 32 bits."""
    side, other = dict(rows=("fout", "tokens"), tokens=("fin", "rows"))[rows]
    for n, words in ((1, 1 << 30), (1, (1 << 31) - 1)):
        assert codes(lib, **{rows: n, other: 1, "words": words, side: COL}) == ERR_SHAPE, (n, words)
    if not gpu_available():
        for n, words in ((1, (1 << 30) - 1), (3, ((1 << 31) - 1) // 3), (5, ((1 << 31) - 1) // 5)):
            assert codes(lib, **{rows: n, other: 1, "words": words, side: COL}) == ERR_DEVICE, (n, words)
            assert codes(lib, **{rows: n, other: 1, "words": words, side: ROW}) == ERR_DEVICE, (n, words)


def test_column_major_scales_of_one_long_row(lib):  # noqa: F811
    """The same of the casts: 2^30 groups of a single row."""
    A, E4M3 = 0x10000, 1

    def cast(cols, group, flags, rows=1):
        return lib.qcast_per_token_sf(A, rows, cols, E4M3, group, 0.0, flags, A, A, None)
    assert cast(1 << 36, 64, COL) == cast(1 << 37, 128, COL) == ERR_SHAPE
    if not gpu_available():
        assert cast((1 << 36) - 64, 64, COL) == cast(1 << 36, 64, ROW) == cast(1 << 36, 64, COL | 4) == ERR_DEVICE
        assert cast(128 * ((1 << 31) // 3), 128, COL, rows=3) == ERR_DEVICE


def test_combine_backward_without_rows(lib):  # noqa: F811
    """Buffers of no rows have no address; only dw is written then."""
    empty = dict(rows=0, q=None, sf=None, dy=None)
    assert bwd(lib, **empty, dw=None) == bwd(lib, **empty, dw=None, y=None) == OK
    assert bwd(lib, **empty, dw=None, cols=200) == bwd(lib, **empty, dw=None, top_k=65) == ERR_SHAPE
    assert bwd(lib, **empty, dest=None) == ERR_NULL
    if not gpu_available():
        assert bwd(lib, **empty) == bwd(lib, **empty, y=None) == ERR_DEVICE
