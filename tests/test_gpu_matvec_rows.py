"""Products with E2M1 weights where several rows take one row of x, called
through the C entry point (the binding gives rows without ids an x of their
own). Behind x's rows stand NaNs, which no product may meet. Bounds as in
test_gpu_matvec.py."""
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from test_gpu_matvec import activations, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32), ("e5m2", 128)])
@pytest.mark.parametrize("x_rows,per,k", [(1, 2, 512), (2, 2, 512), (3, 7, 1152),     # all of x in LDS
                                          (1, 3, 36992), (2, 2, 36992),               # stages of it
                                          (1, 16, 9728), (5, 3, 9728), (7, 5, 5248)])  # with the weights (stages with ids)
@pytest.mark.parametrize("ids", [False, True])
def test_rows_of_one_row_of_x(x, x_group, x_rows, per, k, ids):
    g = torch.Generator().manual_seed(k + x_rows)
    rows, n, experts = x_rows * per, 40, 2 if ids else 1
    codes, sf = weights(g, (experts,), n, k, 32, False)
    xq, x_sf, xv = activations(g, x_rows, k, x, x_group)
    # NaN codes and scales behind the rows that there are
    held = torch.full((rows, k), float("nan")).to(xq.dtype)
    held[:x_rows] = xq
    held = held.to(DEV)
    held_sf = None
    if x_sf is not None:
        held_sf = torch.full((rows, k // x_group), float("nan"))
        held_sf[:x_rows] = x_sf
        held_sf = held_sf.to(DEV)
    e = torch.randint(0, experts, (rows,), generator=g) if ids else None
    e_dev = None if e is None else e.to(DEV)
    out = torch.full((rows, n), float("nan"), device=DEV)
    w, ws = codes.to(DEV), sf.to(DEV)
    fmt = {"bf16": 0, "e4m3": pq.FMT_E4M3, "e5m2": pq.FMT_E5M2}[x]
    rc = pq.load().qcast_matvec_e2m1(
        held.data_ptr(), fmt, None if held_sf is None else held_sf.data_ptr(), x_group, x_rows, w.data_ptr(),
        ws.data_ptr(), 32, 0, experts, None if e is None else e_dev.data_ptr(), 8, rows, n, k, pq.OUT_F32,
        out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    each = torch.zeros(rows, dtype=torch.int64) if e is None else e
    want, mag = moe_ref.matvec(xv, moe_ref.e2m1_weights(codes, sf, 32), each)
    bound = mag * ((k / 32 + 66) * 2.0 ** -23) + 1e-38
    assert ((out.double().cpu() - want).abs() <= bound).all()
