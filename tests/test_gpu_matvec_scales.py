"""Packed UE8M0 scales of E2M1 weights at the ends of their range: byte 0 is
2^-127 (a subnormal fp32), 254 is 2^127, and 255 is NaN. Bounds as in
test_gpu_matvec.py, for which no partial result may leave fp32's normal range.

With x's scales over 128 k, codes' products are summed and scaled by the weights'
scales ahead of x's. E4M3 codes up to 448 give sums up to 4 * 32 * 448 * 6 = 2^18.4
there, and 2^18.4 * 2^127 is past fp32, whatever x's scale: the header excludes
that. Codes of 2^-9 keep 4 * 32 * 2^-9 * 6 = 1.5 below 2, and 1.5 * 2^127 fits."""
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from test_gpu_matvec import activations, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def product(x, x_sf, codes, e, ids):
    return pq.qcast_matvec_e2m1(x.to(DEV), codes.to(DEV), e.view(torch.int32).to(DEV),
                                None if ids is None else ids.to(DEV), x_sf=None if x_sf is None else x_sf.to(DEV),
                                out_dtype=torch.float32).double().cpu()


@pytest.mark.parametrize("low,high,scale", [(0, 3, 2.0 ** 90), (252, 255, 2.0 ** -100)])
@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32), ("e4m3", 128)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,k,experts", [(1, 512, 0), (5, 1536, 0), (9, 9728, 0), (2, 36864, 0), (12, 512, 3),
                                            (40, 9728, 3)])
def test_smallest_and_largest(low, high, scale, x, x_group, group, rows, k, experts):
    g = torch.Generator().manual_seed(rows + k)
    lead = (experts,) if experts else ()
    codes, _ = weights(g, lead, 24, k, group, False)
    e = torch.randint(low, high, (*lead, 24, k // group), generator=g, dtype=torch.uint8)
    xq, x_sf, xv = activations(g, rows, k, x, x_group)
    if x_sf is None:
        xq = (xq.float() * scale).to(torch.bfloat16)         # a power of two: exact
    else:
        if high == 255 and x_group == 128:
            xq = torch.sign(xq.float()).mul(2.0 ** -9).to(xq.dtype)
            xv = xq.double() * x_sf.double().repeat_interleave(x_group, 1)
        x_sf = x_sf * scale
    xv = xv * scale
    ids = torch.randint(0, experts, (rows,), generator=g) if experts else None
    want, mag = moe_ref.matvec(xv, moe_ref.e2m1_weights(codes, e.view(torch.int32), group), ids)
    assert want.abs().max() > 1e-13
    out = product(xq, x_sf, codes, e, ids)
    assert ((out - want).abs() <= mag * ((k / 32 + 66) * 2.0 ** -23)).all()


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("rows,k", [(1, 512), (9, 9728)])
def test_not_a_number(x, x_group, group, rows, k):
    """255 reaches the columns that have it, and no other."""
    g = torch.Generator().manual_seed(rows)
    codes, sf = weights(g, (), 24, k, group, True)
    e = sf.view(torch.uint8).clone()
    xq, x_sf, _ = activations(g, rows, k, x, x_group)
    clean = product(xq, x_sf, codes, e, None)
    bad = [3, 17, 22]
    for i, col in enumerate(bad):
        e[col, i * (k // group - 1) // 2] = 255              # the first group, one in the middle, the last
    out = product(xq, x_sf, codes, e, None)
    rest = [c for c in range(24) if c not in bad]
    assert out[:, bad].isnan().all() and torch.equal(out[:, rest], clean[:, rest]) and not clean.isnan().any()
