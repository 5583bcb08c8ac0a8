"""Refusals of the SwiGLU backward from checkpoints in groups of 32, 64 or 128
elements, before any HIP call."""
import pytest

from conftest import gpu_available

(OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_FORMAT, ERR_GROUP, ERR_LAUNCH, ERR_DEVICE,
 ERR_VALUE) = range(9)
A = 0x10000            # aligned, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from precision_quantization_amd import _lib
    return _lib.load()


def bwd(lib, ckpt=A, ckpt_sf=A, dv=A, rows=4, cols=256, w=None, cf=1, ckpt_group=32, fmt=1, group=128, clamp_min=0.0,
        flags=0, clamp=0.0, q=A, sf=A, dhT=A, dhT_sf=A, vT=A, vT_sf=A, dw=A, ws=A):
    return lib.qcast_swiglu_backward_checkpoint_ex(ckpt, ckpt_sf, dv, rows, cols, w, cf, ckpt_group, fmt, group,
                                                   clamp_min, flags, clamp, q, sf, dhT, dhT_sf, vT, vT_sf, dw, ws, None)


@pytest.mark.parametrize("ckpt_group", [32, 64, 128])
def test_refusals(lib, ckpt_group):
    def call(**kw):
        return bwd(lib, ckpt_group=ckpt_group, **kw)
    assert call(fmt=2) == call(cf=4) == call(flags=8) == ERR_FORMAT
    assert call(group=32) == call(group=64) == ERR_GROUP      # of the outputs
    # the outputs' groups are of 128 channels, whatever the checkpoint's
    assert call(cols=96) == call(cols=64) == call(cols=160) == call(rows=-1) == ERR_SHAPE
    assert call(clamp=float("nan")) == ERR_VALUE
    for k in ("ckpt", "ckpt_sf", "dv", "q", "sf", "ws", "dhT", "vT_sf"):
        assert call(**{k: None}) == ERR_NULL, k
    assert call(ckpt_sf=A + 2) == call(ckpt=A + 8) == ERR_ALIGN
    assert call(rows=0, ckpt=None, ckpt_sf=None, dv=None) == OK
    if not gpu_available():
        assert call() == ERR_DEVICE


def test_refused_groups(lib):
    for g in (0, -32, 8, 16, 48, 96, 256):
        assert bwd(lib, ckpt_group=g) == ERR_GROUP, g
