"""The plain mixture-of-experts reference itself: its gradient against autograd
and central differences, its rows against the counts, and the workspace and
row formulas of the binding against those of include/qcast.h."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from conftest import ROOT


def test_gradient_against_autograd_and_differences():
    g = torch.Generator().manual_seed(0)
    ids = moe_ref.routing(5, 3, 4, seed=1)
    dest, source, *_ = moe_ref.sort(ids, 4, 2)
    dest = torch.from_numpy(dest)
    dest[2] = -1                                  # a token without rows
    y = torch.randn(len(source), 6, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(5, 3, generator=g, dtype=torch.float64, requires_grad=True)
    dout = torch.randn(5, 6, generator=g, dtype=torch.float64)

    def loss(y, w):
        total = 0.0
        for t in range(5):
            for k in range(3):
                if dest[t, k] >= 0:
                    total = total + w[t, k] * (y[dest[t, k]] * dout[t]).sum()
        return total

    dy, dw, _ = moe_ref.combine_grad(dout, y.detach(), dest, w.detach())
    gy, gw = torch.autograd.grad(loss(y, w), (y, w))
    assert torch.allclose(dy, gy, rtol=1e-12) and torch.allclose(dw, gw, rtol=1e-12)
    # central differences of a bilinear function: exact up to rounding
    h = 0.5
    with torch.no_grad():
        for at in ((0, 0), (1, 2), (4, 1)):
            up, down = w.clone(), w.clone()
            up[at] += h
            down[at] -= h
            assert abs(float((loss(y, up) - loss(y, down)) / (2 * h) - dw[at])) < 1e-12
        out, _ = moe_ref.combine(y, dest, w)
        assert abs(float((out * dout).sum() - loss(y, w))) < 1e-12


@pytest.mark.parametrize("tokens,top_k,experts,align", [(0, 2, 4, 16), (1, 1, 1, 128), (1, 8, 4, 1),
                                                        (7, 3, 5, 16), (40, 2, 64, 8)])
def test_rows_hold_every_routing(tokens, top_k, experts, align):
    rows = pq.expert_rows(tokens, top_k, experts, align)
    assert rows == moe_ref.bound_rows(tokens, top_k, experts, align) and rows % align == 0
    slots = tokens * top_k
    # one slot for as many experts as can have one, the rest in the last
    ids = np.minimum(np.arange(slots), experts - 1).reshape(tokens, top_k)
    _, _, offsets, counts, _ = moe_ref.sort(ids, experts, align)
    assert counts.sum() == slots and offsets[-1] <= rows


def test_formulas_of_the_header(tmp_path):
    src = tmp_path / "f.c"
    src.write_text('#include "qcast.h"\n'
                   "long rows(long t, long k, long e, long a) { return qcast_expert_rows(t, k, e, a); }\n"
                   "long ws(long t, long k, long e) { return qcast_expert_sort_ws_bytes(t, k, e); }\n")
    so = tmp_path / "f.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(so)],
                   check=True)
    f = ctypes.CDLL(str(so))
    for fn in (f.rows, f.ws):
        fn.restype = ctypes.c_long
        fn.argtypes = [ctypes.c_long] * (4 if fn is f.rows else 3)
    for t, k, e, a in [(0, 1, 1, 1), (1, 8, 256, 128), (8, 8, 256, 16), (16384, 8, 256, 128), (2048, 2, 8, 1),
                       (4097, 1, 8, 4), (1 << 20, 8, 1000, 1024)]:
        assert f.rows(t, k, e, a) == pq.expert_rows(t, k, e, a)
        assert f.ws(t, k, e) == pq._sort_parts(t * k) * e * 4


def test_weights_are_those_of_the_e2m1_cast():
    import oracle
    from precision_quantization_amd import workloads
    x = torch.randn(3, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    q, sf = oracle.e2m1(workloads.bf16_bits(x), 32)
    w = moe_ref.e2m1_weights(torch.from_numpy(q), torch.from_numpy(sf), 32)
    # nearest of a step of 2^-1 relative at most, plus the smallest code's half
    step = torch.from_numpy(np.repeat(sf, 32, 1)).double()
    assert ((w - x.double()).abs() <= x.double().abs() / 4 + step / 4 + 1e-6).all()
