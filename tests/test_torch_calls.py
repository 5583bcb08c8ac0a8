"""What the binding takes from torch's C module has public stand-ins."""
import types

import pytest
import torch

import precision_quantization_amd as pq


def test_without_the_private_functions():
    for c in (types.SimpleNamespace(), types.SimpleNamespace(_dynamo=types.SimpleNamespace(guards=types.SimpleNamespace()))):
        strided, here, stream = pq._torch_calls(c)
        assert here is torch.cuda.current_device and callable(strided) and callable(stream)


def bits(t):
    # column-major scales of 67 rows: the padding row is left as it was
    t = t[:, :67] if t.shape[-1] == 68 else t
    return t.contiguous().view(torch.uint8)


@pytest.mark.gpu
def test_calls_through_the_public_functions(monkeypatch):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    h = torch.randn(67, 512, generator=g, device=dev).to(torch.bfloat16)
    w = torch.ones(512, dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream(dev)

    def calls():
        side.wait_stream(torch.cuda.current_stream(dev))
        out = []
        for stream in (None, side):
            f = pq.qcast_norm_per_token(h, w, h, w, ckpt_fmt="e4m3", sf_flags=pq.SF_COL_MAJOR, stream=stream)
            s = pq.qcast_swiglu_checkpoint(h, stream=stream)
            out += [t for t in (*f, *s) if t is not None]
        with torch.cuda.stream(side):
            out += pq.qcast_recast_per_channel_T(s[2], s[3])
        torch.cuda.synchronize()
        return out

    a = calls()
    for name, fn in zip(("_strided", "_current_device", "_current_stream"), pq._torch_calls(types.SimpleNamespace())):
        monkeypatch.setattr(pq, name, fn)
    b = calls()
    assert len(a) == len(b)
    for x, y in zip(a, b):
        assert x.shape == y.shape and x.stride() == y.stride() and x.dtype == y.dtype and x.device == y.device
        assert torch.equal(bits(x), bits(y))
