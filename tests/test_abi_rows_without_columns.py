"""Sums over no columns: refused rather than left unwritten."""
import pytest

from test_abi_checkpoint_norm import A, ERR_SHAPE, OK, bwd, nbwd, norm


@pytest.fixture(scope="module")
def lib():
    from precision_quantization_amd import _lib
    return _lib.load()


def test_gradient_of_a_token_gate(lib):
    assert nbwd(lib, cols=0, kind=2, dgate=A) == ERR_SHAPE
    assert nbwd(lib, cols=0, kind=2, dgate=None) == OK
    assert nbwd(lib, cols=0, kind=2, rows=0, dgate=A) == OK
    # sums over the rows have no columns, and an elementwise gradient no elements
    assert nbwd(lib, cols=0, kind=1, dgate=A) == nbwd(lib, cols=0, kind=3, dgate=A) == OK


def test_gradient_of_a_row_weight(lib):
    assert bwd(lib, cols=0) == ERR_SHAPE
    assert bwd(lib, cols=0, dw=None) == bwd(lib, cols=0, rows=0) == OK


def test_norm_writes_nothing(lib):
    assert norm(lib, cols=0) == OK
