"""The checkpoint and norm operators on tensors whose byte and element offsets
pass 32 bits: the last rows (or token groups), and rows where an offset passes
2^31 and 2^32, as a call on those rows alone gives them, bit for bit."""
import pytest
import torch

import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
ROWS, COLS = 530001, 8192              # 4.3e9 elements
# multiples of 128: an element offset passes 2^31, 2^32, the ragged end
STARTS = [(1 << 31) // COLS - 128, (1 << 32) // COLS - 128, ROWS // 128 * 128 - 128]


@pytest.fixture()
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    if torch.cuda.mem_get_info()[0] < 90 << 30:
        pytest.skip("needs 90 GB of device memory")
    yield torch.device("cuda:0")
    torch.cuda.empty_cache()


def normal(dev, *shape):
    return torch.empty(*shape, dtype=torch.bfloat16, device=dev).normal_()


def codes(dev, *shape):
    t = torch.empty(*shape, dtype=torch.uint8, device=dev).random_(0, 0x7F)      # no NaN codes
    return t.view(torch.float8_e4m3fn)


def scales(dev, *shape):
    return torch.empty(*shape, dtype=torch.float32, device=dev).uniform_(0.001, 0.01)


def parts():
    for r0 in STARTS:
        yield slice(r0, min(ROWS, r0 + 256))


def same(whole, part, what):
    assert torch.equal(whole.contiguous().view(torch.uint8), part.contiguous().view(torch.uint8)), what


def test_swiglu_checkpoint(dev):
    h = normal(dev, ROWS, COLS)
    whole = pq.qcast_swiglu_checkpoint(h)
    for s in parts():
        for i, (a, b) in enumerate(zip(whole, pq.qcast_swiglu_checkpoint(h[s]))):
            same(a[s], b, (i, s))


def test_swiglu_backward_checkpoint(dev):
    q, sf, dv = codes(dev, ROWS, COLS), scales(dev, ROWS, COLS // 128), normal(dev, ROWS, COLS // 2)
    whole = pq.qcast_swiglu_backward_checkpoint(q, sf, dv)
    for s in parts():
        part = pq.qcast_swiglu_backward_checkpoint(q[s], sf[s], dv[s])
        t = slice(s.start, s.start + 256)
        g = slice(s.start // 128, s.start // 128 + 2)
        for name, a, b in zip(whole._fields, whole, part):
            cut = a[:, t] if name in ("dh_t", "v_t") else a[:, g] if name in ("dh_t_sf", "v_t_sf") else a[s]
            same(cut, b, (name, s))


def test_recast(dev):
    q, sf = codes(dev, ROWS, COLS), scales(dev, ROWS, COLS // 128)
    out, out_sf = pq.qcast_recast_per_channel_T(q, sf)
    for s in parts():
        b, b_sf = pq.qcast_recast_per_channel_T(q[s], sf[s])
        same(out[:, s.start:s.start + 256], b, s)
        same(out_sf[:, s.start // 128:s.start // 128 + 2], b_sf, s)


def test_norm(dev):
    y, h, w = normal(dev, ROWS, COLS), normal(dev, ROWS, COLS), normal(dev, COLS)
    whole = pq.qcast_norm_per_token(h, w, y, w, ckpt_fmt="e4m3")
    for s in parts():
        part = pq.qcast_norm_per_token(h[s], w, y[s], w, ckpt_fmt="e4m3")
        for name, a, b in zip(whole._fields, whole, part):
            if a is not None:
                same(a[s], b, (name, s))


def test_norm_backward(dev):
    dx, dh, w = normal(dev, ROWS, COLS), normal(dev, ROWS, COLS), normal(dev, COLS)
    r = torch.empty(ROWS, device=dev).uniform_(0.5, 2.0)
    qh, qy, sf = codes(dev, ROWS, COLS), codes(dev, ROWS, COLS), scales(dev, ROWS, COLS // 128)

    def call(s):
        return pq.qcast_norm_backward_per_token(dx[s], qh[s], r[s], w, dh=dh[s], saved_h_sf=sf[s], saved_y=qy[s],
                                                saved_y_sf=sf[s], rstd_post=r[s], w_post=w, gate=r[s])
    whole = call(slice(None))
    for s in parts():
        part = call(s)
        for name in ("dh", "out", "out_sf", "dgate"):
            same(getattr(whole, name)[s], getattr(part, name), (name, s))
