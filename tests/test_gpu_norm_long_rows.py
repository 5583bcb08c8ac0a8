"""Rows of more than 8192 columns, where a lane of the norm kernels holds two
chunks: every gate, with and without a post-norm, from bf16 and both checkpoint
formats, without a block output, and in the scale layouts, against the 64-bit
formulas within the bounds of block_ref."""
import pytest
import torch

import precision_quantization_amd as pq
import test_gpu_norm as nm

pytestmark = pytest.mark.gpu
PACKED, COL, ROUND = pq.SF_PACKED_UE8M0, pq.SF_COL_MAJOR, pq.SF_ROUND_POW2
KINDS = [None, "channel", "token", "full"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("cols,ckpt", [(8320, "e4m3"), (16384, "e5m2"), (8224, None)])
def test_forward(dev, kind, post, cols, ckpt):
    nm.check_forward(dev, 4, cols, kind, post, group=128 if ckpt else 32, ckpt=ckpt, offset=1.0 if post else 0.0,
                     want_x=True)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("cols,saved", [(8320, "e4m3"), (16384, "e5m2"), (16384, "bf16"), (8224, "bf16")])
def test_backward(dev, kind, post, cols, saved):
    nm.check_backward(dev, 4, cols, kind, post, saved, group=128 if cols % 128 == 0 else 32,
                      offset=1.0 if post else 0.0, want_dy=True)


@pytest.mark.parametrize("kind,saved", [("full", "bf16"), ("token", "e5m2"), (None, "e4m3")])
def test_backward_column_sums_over_several_rows_of_a_workgroup(dev, kind, saved):
    # 256 workgroups: the first 44 carry their sums over a second row
    nm.check_backward(dev, 300, 8320, kind, True, saved)


@pytest.mark.parametrize("cols", [8320, 16384])
def test_without_a_block_output(dev, cols):
    nm.check_forward(dev, 3, cols, has_y=False, kind=None, ckpt="e4m3")
    nm.check_backward(dev, 3, cols, has_y=False, saved="e5m2")
    nm.check_backward(dev, 3, cols, has_y=False, saved="bf16", residual=False)


@pytest.mark.parametrize("fmt,group,flags", [("e4m3", 128, PACKED | COL), ("e2m1", 32, PACKED), ("e5m6", 64, COL),
                                             ("e5m2", 128, COL | ROUND)])
def test_layouts(dev, fmt, group, flags):
    nm.check_forward(dev, 5, 12288, fmt=fmt, group=group, flags=flags, ckpt="e5m2")
    nm.check_backward(dev, 5, 12288, "token", fmt=fmt, group=group, flags=flags)
