"""Products with E2M1 weights against the formula in 64 bits.

Bounds. Every product of an E2M1 value with x (bf16, or an 8-bit code) is exact
in fp32; sums of 32 to 128 of them, the scaled groups' sums and the joins over
lanes and waves are fp32 additions, each counted as off by a whole step, 2^-23,
of the magnitudes' sum: at most 32 inside a matrix instruction, k/32 + 32 over
groups and joins, and two products by the scales. bf16 output adds 2^-8 of the
value. Whole numbers whose sums fit 24 bits have to come out exactly."""
import numpy as np
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def weights(g, lead, n, k, group, packed, spread=0.5):
    codes = torch.randint(0, 256, (*lead, n, k // 2), generator=g, dtype=torch.uint8)
    if packed:
        e = torch.randint(110, 130, (*lead, n, k // group), generator=g, dtype=torch.uint8)
        sf = e.view(torch.int32)
    else:
        sf = torch.exp(torch.randn(*lead, n, k // group, generator=g) * spread)
    return codes, sf


def activations(g, rows, k, x="bf16", x_group=128):
    """(x, x_sf, float64 values)"""
    v = torch.randn(rows, k, generator=g)
    if x == "bf16":
        v = v.to(torch.bfloat16)
        return v, None, v.double()
    q = (v * 50).to(F8[x])
    sf = torch.exp(torch.randn(rows, k // x_group, generator=g)) / 50
    return q, sf, q.float().double() * sf.double().repeat_interleave(x_group, 1)


def check(x, x_sf, xv, codes, sf, group, ids=None, out_dtype=torch.float32, **kw):
    out = pq.qcast_matvec_e2m1(x.to(DEV), codes.to(DEV), sf.to(DEV), None if ids is None else ids.to(DEV),
                               x_sf=None if x_sf is None else x_sf.to(DEV), out_dtype=out_dtype, **kw)
    want, mag = moe_ref.matvec(xv, moe_ref.e2m1_weights(codes, sf, group), ids)
    assert out.dtype == out_dtype and tuple(out.shape) == tuple(want.shape)
    k = xv.shape[1]
    bound = mag * ((k / 32 + 66) * 2.0 ** -23) + 1e-38
    if out_dtype == torch.bfloat16:
        bound = (want.abs() + bound) * 2.0 ** -8 + bound
    worst = ((out.double().cpu() - want).abs() / bound).max().item() if want.numel() else 0.0
    assert worst <= 1.0, f"off by {worst:.3g} of the bound"
    return out


@pytest.mark.parametrize("group,packed", [(32, False), (64, False), (128, False), (32, True), (64, True), (128, True)])
@pytest.mark.parametrize("rows", [1, 2, 5, 16, 17, 40, 64, 100])
@pytest.mark.parametrize("n,k", [(16, 512), (1, 1024), (33, 512), (200, 2560)])
def test_one_weight(group, packed, rows, n, k):
    g = torch.Generator().manual_seed(rows)
    codes, sf = weights(g, (), n, k, group, packed)
    check(*activations(g, rows, k), codes, sf, group)


@pytest.mark.parametrize("k", [32, 64, 96, 160, 224, 1056, 7168, 18432])
@pytest.mark.parametrize("rows", [1, 3, 20])
def test_lengths(k, rows):
    g = torch.Generator().manual_seed(k)
    codes, sf = weights(g, (), 24, k, 32, False)
    check(*activations(g, rows, k), codes, sf, 32)
    check(*activations(g, rows, k, "e4m3", 32), codes, sf, 32)


@pytest.mark.parametrize("x", ["e4m3", "e5m2"])
@pytest.mark.parametrize("group,x_group", [(32, 32), (32, 64), (32, 128), (64, 32), (128, 32), (128, 128)])
@pytest.mark.parametrize("rows", [1, 4, 18])
def test_codes_as_input(x, group, x_group, rows):
    g = torch.Generator().manual_seed(rows)
    codes, sf = weights(g, (), 40, 1152, group, False)
    check(*activations(g, rows, 1152, x, x_group), codes, sf, group)
    codes, sf = weights(g, (3,), 20, 512, group, True)
    ids = torch.randint(-1, 4, (rows,), generator=g)
    check(*activations(g, rows, 512, x, x_group), codes, sf, group, ids, torch.bfloat16)


@pytest.mark.parametrize("tokens,top_k,experts", [(1, 8, 16), (1, 1, 1), (4, 2, 3), (16, 8, 12), (3, 6, 200), (40, 4, 5),
                                                  (130, 1, 2)])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
def test_experts(tokens, top_k, experts, dtype, out_dtype):
    g = torch.Generator().manual_seed(tokens)
    n, k = 52, 384
    codes, sf = weights(g, (experts,), n, k, 32, False)
    # one in a few slots has its expert elsewhere
    ids = moe_ref.routing(tokens, top_k, experts + 2, seed=tokens, repeat=True, dtype=dtype) - 1
    out = check(*activations(g, tokens, k), codes, sf, 32, ids, out_dtype)
    gone = ((ids < 0) | (ids >= experts)).reshape(-1)
    assert not out.cpu()[gone].any()
    # rows of their own for every slot
    check(*activations(g, tokens * top_k, k), codes, sf, 32, ids, out_dtype)


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 32), ("e5m2", 128)])
@pytest.mark.parametrize("group,packed,k", [(32, False, 2816), (32, False, 3200), (32, False, 5248), (64, False, 9856),
                                            (32, False, 20480), (128, True, 2560), (128, True, 5632), (128, True, 9728)])
def test_long_rows_of_experts(x, x_group, group, packed, k):
    """More of x than LDS takes at once: stages, with and without an end of k
    that is no whole unit."""
    g = torch.Generator().manual_seed(k)
    codes, sf = weights(g, (3,), 40, k, group, packed)
    for tokens, top_k in ((30, 2), (7, 1), (2, 2)):      # passes of 16, of 7, and of 4
        ids = moe_ref.routing(tokens, top_k, 4, seed=k, repeat=True) - int(tokens > 7)
        check(*activations(g, tokens, k, x, x_group), codes, sf, group, ids)


@pytest.mark.parametrize("x,x_group", [("bf16", 128), ("e4m3", 64), ("e5m2", 128)])
@pytest.mark.parametrize("group", [32, 64])
@pytest.mark.parametrize("rows", [3, 4, 5, 11, 16, 21])
@pytest.mark.parametrize("k", [5248, 9728, 36992])
def test_long_rows(x, x_group, group, rows, k):
    g = torch.Generator().manual_seed(k + rows)
    codes, sf = weights(g, (), 40, k, group, False)
    check(*activations(g, rows, k, x, x_group), codes, sf, group)


@pytest.mark.parametrize("tokens,top_k,experts", [(5000, 1, 2), (1500, 8, 3), (257, 4, 1024), (65, 1, 1)])
def test_many_rows_of_experts(tokens, top_k, experts):
    """Many passes of an expert, whose rows are thousands of ids apart or next
    to one another."""
    g = torch.Generator().manual_seed(tokens)
    codes, sf = weights(g, (experts,), 20, 64, 32, False)
    ids = moe_ref.routing(tokens, top_k, experts, seed=tokens, repeat=True)
    check(*activations(g, tokens, 64), codes, sf, 32, ids)
    ids = torch.sort(ids.reshape(-1)).values.reshape(tokens, top_k)
    check(*activations(g, tokens * top_k, 64), codes, sf, 32, ids)


def test_ids_far_outside():
    g = torch.Generator().manual_seed(0)
    codes, sf = weights(g, (2,), 16, 128, 64, False)
    ids = torch.tensor([[2 ** 62, -2 ** 63, 1], [(1 << 32) + 1, -1, 0]])
    out = check(*activations(g, 2, 128), codes, sf, 64, ids)
    assert not out.cpu()[[0, 1, 3, 4]].any()


@pytest.mark.parametrize("rows", [1, 7, 16, 50])
@pytest.mark.parametrize("k,group", [(256, 32), (544, 32), (1024, 128), (2048, 64)])
def test_whole_numbers_are_exact(rows, k, group):
    """Every code at every place, x and scales small powers of two and whole
    numbers: each sum fits 24 bits, so any order of adding gives it exactly."""
    g = torch.Generator().manual_seed(rows)
    codes, _ = weights(g, (), 48, k, group, False)
    sf = torch.exp2(torch.randint(-1, 2, (48, k // group), generator=g).float())
    x = torch.randint(-8, 9, (rows, k), generator=g).to(torch.bfloat16)
    out = pq.qcast_matvec_e2m1(x.to(DEV), codes.to(DEV), sf.to(DEV), out_dtype=torch.float32)
    want, _ = moe_ref.matvec(x.double(), moe_ref.e2m1_weights(codes, sf, group))
    assert torch.equal(out.cpu().double(), want)
    # one input at a time: the weights themselves
    eye = torch.eye(min(k, 64), k).to(torch.bfloat16)
    out = pq.qcast_matvec_e2m1(eye.to(DEV), codes.to(DEV), sf.to(DEV), out_dtype=torch.float32)
    assert torch.equal(out.cpu().double(), moe_ref.e2m1_weights(codes, sf, group).t()[:eye.shape[0]])


def test_extremes():
    """Subnormal and huge inputs and scales, infinities and NaN."""
    codes = torch.full((16, 64), 0x22, dtype=torch.uint8)             # every weight 1
    sf = torch.ones(16, 4)
    x = torch.zeros(6, 128, dtype=torch.bfloat16)
    x[0, 5] = 2.0 ** -133                                             # smallest bf16
    x[1, 3], x[1, 70] = 2.0 ** 127, 2.0 ** 127                        # past fp32 when summed
    x[2, 9] = float("inf")
    x[3, 100] = float("nan")
    x[4, 0], x[4, 127] = float("inf"), float("-inf")
    x[5] = 1
    sf2 = sf.clone()
    sf2[:, 1] = 2.0 ** -149
    out = pq.qcast_matvec_e2m1(x.to(DEV), codes.to(DEV), sf.to(DEV), out_dtype=torch.float32).cpu()
    assert (out[0] == 2.0 ** -133).all() and out[1].isinf().all() and out[2].isinf().all()
    assert out[3].isnan().all() and out[4].isnan().all() and (out[5] == 128).all()
    out = pq.qcast_matvec_e2m1(x.to(DEV), codes.to(DEV), sf2.to(DEV), out_dtype=torch.float32).cpu()
    assert (out[5] == 96).all() and (out[1] == 2.0 ** 127).sum() == 0
    # rows do not reach one another
    one = pq.qcast_matvec_e2m1(x[5:].to(DEV), codes.to(DEV), sf.to(DEV), out_dtype=torch.float32).cpu()
    assert (one == 128).all()


@pytest.mark.parametrize("rows,n,k", [(0, 16, 64), (3, 0, 64), (3, 16, 0)])
def test_nothing_to_sum(rows, n, k):
    x = torch.ones(rows, k, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    sf = torch.ones(n, k // 32, device=DEV)
    out = pq.qcast_matvec_e2m1(x, w, sf, out=torch.full((rows, n), 7.0, dtype=torch.bfloat16, device=DEV))
    assert tuple(out.shape) == (rows, n) and not out.any()


def test_the_cast_weight_is_what_is_read():
    """Weights cast by qcast_e2m1 and qcast_per_token_sf: what cast_back gives."""
    g = torch.Generator(device=DEV).manual_seed(1)
    wt = torch.randn(96, 1024, generator=g, device=DEV).to(torch.bfloat16)
    x = torch.randn(3, 1024, generator=g, device=DEV).to(torch.bfloat16)
    for group in (32, 64, 128):
        q, sf = pq.qcast_e2m1(wt, group)
        check(x.cpu(), None, x.cpu().double(), q.cpu(), sf.cpu(), group)
        q, sf = pq.qcast_per_token_sf(wt, "e2m1", group, sf_flags=pq.SF_PACKED_UE8M0)
        check(x.cpu(), None, x.cpu().double(), q.cpu(), sf.cpu(), group)


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(8, 128, dtype=torch.uint8, device=DEV)
    sf = torch.zeros(8, 8, device=DEV)
    w3, sf3 = w.unsqueeze(0), sf.unsqueeze(0)
    ids = torch.zeros(8, dtype=torch.int64, device=DEV)
    for bad in (lambda: pq.qcast_matvec_e2m1(x.float(), w, sf), lambda: pq.qcast_matvec_e2m1(x, w3, sf3),
                lambda: pq.qcast_matvec_e2m1(x, w, sf, ids), lambda: pq.qcast_matvec_e2m1(x, w3, sf3, ids[:6]),
                lambda: pq.qcast_matvec_e2m1(x, w[:, :64].contiguous(), sf), lambda: pq.qcast_matvec_e2m1(x, w, sf[:4]),
                lambda: pq.qcast_matvec_e2m1(x, w, sf[:, :5].contiguous()),
                lambda: pq.qcast_matvec_e2m1(x, w, sf[:, :1].contiguous()),
                lambda: pq.qcast_matvec_e2m1(x, w, sf.double()), lambda: pq.qcast_matvec_e2m1(x, w.to(torch.int8), sf),
                lambda: pq.qcast_matvec_e2m1(x, w3, sf3, ids.float()), lambda: pq.qcast_matvec_e2m1(x, w3, sf3, ids.cpu()),
                lambda: pq.qcast_matvec_e2m1(x, w, sf, x_sf=torch.ones(4, 2, device=DEV)),
                lambda: pq.qcast_matvec_e2m1(x.to(torch.float8_e4m3fn), w, sf),
                lambda: pq.qcast_matvec_e2m1(x.to(torch.float8_e4m3fn), w, sf, x_sf=torch.ones(4, 3, device=DEV)),
                lambda: pq.qcast_matvec_e2m1(x, w, sf, out_dtype=torch.float16),
                lambda: pq.qcast_matvec_e2m1(x, w, sf, out=torch.zeros(4, 9, dtype=torch.bfloat16, device=DEV)),
                lambda: pq.qcast_matvec_e2m1(x.t().contiguous().t(), w, sf),
                lambda: pq.qcast_matvec_e2m1(x, w, sf, out_dtype=torch.bfloat16, out=x)):
        with pytest.raises(pq.QcastError):
            bad()
