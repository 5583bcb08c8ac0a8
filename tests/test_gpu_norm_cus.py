"""The compute-unit override and the norm: its grid follows the override, its
results do not."""
import ctypes

import pytest
import torch

import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu


class KernelTimer:
    """Time of the next kernel of the library, from its own dispatch."""

    def __init__(self):
        self.hip = ctypes.CDLL("libamdhip64.so")
        self.hip.hipEventCreateWithFlags.argtypes = [ctypes.POINTER(ctypes.c_void_p), ctypes.c_uint]
        self.hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
        self.hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self.events = [ctypes.c_void_p(), ctypes.c_void_p()]
        for e in self.events:
            assert self.hip.hipEventCreateWithFlags(ctypes.byref(e), 0) == 0

    def ms(self, call):
        pq.qcast_bench_time_next(*self.events)
        out = call()
        torch.cuda.synchronize()
        t = ctypes.c_float()
        assert self.hip.hipEventElapsedTime(ctypes.byref(t), *self.events) == 0
        return t.value, out

    def close(self):
        for e in self.events:
            self.hip.hipEventDestroy(e)


def test_override_past_any_device():
    dev, rows, cols = torch.device("cuda:0"), 200001, 32
    h = torch.randn(rows, cols, generator=torch.Generator(device=dev).manual_seed(2), device=dev).to(torch.bfloat16)
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    a = pq.qcast_norm_per_token(h, w, h, w, group=32)
    try:
        pq.qcast_set_num_cus(2 ** 31 - 1)
        b = pq.qcast_norm_per_token(h, w, h, w, group=32)
    finally:
        pq.qcast_set_num_cus(0)
    for x, y in zip(a, b):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("rows,cols", [(4096, 7168), (2048, 16384)])
def test_forward_follows_the_override(rows, cols):
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(1)
    h, y = (torch.randn(rows, cols, generator=g, device=dev).to(torch.bfloat16) for _ in range(2))
    w = torch.randn(cols, generator=g, device=dev).to(torch.bfloat16)
    timer = KernelTimer()
    results = {}
    try:
        for n in (0, 256, 3, 1):
            pq.qcast_set_num_cus(n)
            timer.ms(lambda: pq.qcast_norm_per_token(h, w, y, w, ckpt_fmt="e4m3"))
            results[n] = timer.ms(lambda: pq.qcast_norm_per_token(h, w, y, w, ckpt_fmt="e4m3"))
    finally:
        pq.qcast_set_num_cus(0)
        timer.close()
    whole = results[0]
    # a workgroup of one compute unit takes all the rows: at least 2048 one
    # after another, where 256 units take at most 16 each
    assert results[1][0] > 4 * whole[0], (results[1][0], whole[0])
    assert results[3][0] > 2 * whole[0], (results[3][0], whole[0])
    for n in (256, 3, 1):
        for a, b in zip(whole[1], results[n][1]):
            assert (a is None) == (b is None)
            assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)), n
