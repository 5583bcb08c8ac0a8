"""Products with E2M1 weights where a workgroup's waves take several column tiles
one after the other (many experts of long n), and where a workgroup takes more
than one pass of rows without experts (more than 8 passes of 16). Compared with
64-bit products on the GPU; bounds as in test_gpu_matvec.py."""
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from test_gpu_matvec import activations, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(x, x_sf, xv, codes, sf, group, ids=None):
    x, xv, codes, sf = x.to(DEV), xv.to(DEV), codes.to(DEV), sf.to(DEV)
    k, n = xv.shape[1], codes.shape[-2]
    rows = x.shape[0] if ids is None else ids.numel()
    out = torch.full((rows, n), float("nan"), device=DEV)
    pq.qcast_matvec_e2m1(x, codes, sf, None if ids is None else ids.to(DEV),
                         x_sf=None if x_sf is None else x_sf.to(DEV), out_dtype=torch.float32, out=out)
    value = torch.from_numpy(moe_ref.E2M1).to(DEV)
    row = torch.arange(rows, device=DEV) // (rows // x.shape[0])
    flat = torch.zeros(rows, dtype=torch.int64, device=DEV) if ids is None else ids.reshape(-1).to(DEV)
    codes, sf = codes.reshape(-1, n, k // 2), sf.reshape(-1, n, sf.shape[-1])
    seen = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for e in range(codes.shape[0]):
        mine = (flat == e).nonzero()[:, 0]
        seen[mine] = True
        s = sf[e].double() if sf.dtype == torch.float32 else \
            torch.exp2(sf[e].contiguous().view(torch.uint8).double() - 127)
        w = torch.stack([value[(codes[e] & 15).long()], value[(codes[e] >> 4).long()]], dim=2).flatten(1) * \
            s.repeat_interleave(group, 1)
        v = xv[row[mine]]
        bound = (v.abs() @ w.abs().t()) * ((k / 32 + 66) * 2.0 ** -23) + 1e-38
        assert ((out[mine].double() - v @ w.t()).abs() <= bound).all(), e
    assert not out[~seen].any()


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32), ("e5m2", 128)])
@pytest.mark.parametrize("tokens,top_k,experts,n,k,group,packed",
                         [(16, 8, 32, 7003, 2048, 32, True),       # passes of 16: 7 tiles a wave, two waves a tile
                          (16, 8, 32, 7003, 1920, 32, False),      # and k that ends inside a unit
                          (30, 10, 100, 5003, 896, 64, False),     # 8 tiles a wave, one wave a tile
                          (2, 8, 32, 7003, 1152, 128, False),      # passes of 4: two tiles a wave
                          (24, 1, 300, 5003, 768, 32, False),
                          (8, 5, 64, 9003, 512, 128, True)])
def test_several_tiles_of_a_wave(x, x_group, tokens, top_k, experts, n, k, group, packed):
    g = torch.Generator().manual_seed(n + k)
    codes, sf = weights(g, (experts,), n, k, group, packed)
    ids = moe_ref.routing(tokens, top_k, experts, seed=k, total=experts + 3)
    check(*activations(g, tokens, k, x, x_group), codes, sf, group, ids)
    # rows of their own for every slot
    check(*activations(g, tokens * top_k, k, x, x_group), codes, sf, group, ids)


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32), ("e5m2", 128)])
@pytest.mark.parametrize("rows", [128, 129, 200, 300])
@pytest.mark.parametrize("n,k", [(40, 512), (3001, 1152), (40000, 256),        # x in LDS
                                 (40, 5248), (1500, 9728)])                    # x with the weights
def test_many_passes_without_experts(x, x_group, rows, n, k):
    g = torch.Generator().manual_seed(rows + k)
    codes, sf = weights(g, (), n, k, 64 if k % 64 == 0 else 32, False)
    check(*activations(g, rows, k, x, x_group), codes, sf, 64 if k % 64 == 0 else 32)
