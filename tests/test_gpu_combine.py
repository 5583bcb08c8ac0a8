"""Experts' rows weighted and summed, and the gradient of that, against the
formulas in 64 bits.

Bounds. A sum from base on is at most top_k fma of fp32, each off by half a
step of a partial sum that the magnitudes bound (2^-24 of their sum each);
rounding to bf16 adds 2^-8 of the value (half the smallest normal step below
it). dw is a sum of cols exact products (bf16 times bf16 fits fp32's 24 bits):
at most cols/64 + 8 fma in one lane and 16 additions that join the lanes and
waves, each off by 2^-24 of the magnitudes' sum. dy is one fp32 product, cast
(bit for bit the oracle's cast) or rounded to bf16."""
import numpy as np
import pytest
import torch

import moe_ref
import oracle
import precision_quantization_amd as pq
from precision_quantization_amd import workloads
from test_gpu_dispatch import FILL, bytes_of, filled, plan_of, scale_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TINY = 2.0 ** -134              # half a step of bf16's subnormals


def near(got, want, mag, steps, what):
    got = got.double().cpu()
    bound = want.abs() * 2.0 ** -8 + (mag * (steps * 2.0 ** -24) + TINY) * (1 + 2.0 ** -7)
    worst = ((got - want).abs() / bound).max().item() if want.numel() else 0.0
    assert worst <= 1.0, f"{what}: off by {worst:.3g} of the bound"


@pytest.mark.parametrize("tokens,top_k,experts,align", [(1, 1, 1, 1), (1, 8, 16, 128), (3, 2, 4, 16), (67, 4, 16, 16),
                                                        (129, 7, 9, 1), (20, 9, 30, 2), (5, 33, 40, 1)])
@pytest.mark.parametrize("cols", [8, 520, 1024, 7168])
@pytest.mark.parametrize("weighted,based", [(True, True), (False, False), (True, False), (False, True)])
def test_combine(tokens, top_k, experts, align, cols, weighted, based):
    plan, dest, source, *_ = plan_of(tokens, top_k, experts, align, total=experts + 3, first=1)
    g = torch.Generator().manual_seed(tokens)
    y = torch.randn(source.size, cols, generator=g).to(torch.bfloat16)
    y[torch.from_numpy(source < 0)] = float("nan")          # rows that no slot has are not read
    w = torch.randn(tokens, top_k, generator=g) if weighted else None
    base = torch.randn(tokens, cols, generator=g).to(torch.bfloat16) if based else None
    out = filled((tokens, cols), torch.bfloat16)
    got = pq.qcast_combine(y.to(DEV), plan.dest, None if w is None else w.to(DEV),
                           None if base is None else base.to(DEV), out=out)
    assert got is out
    want, mag = moe_ref.combine(y, dest, w, base)
    near(got, want, mag, top_k, "combine")


@pytest.mark.parametrize("top_k,weighted,based", [(1, True, False), (2, True, True), (2, False, False)])
def test_many_tokens_of_few_slots(top_k, weighted, based):
    """A count of tokens that no group of them divides, some without a row."""
    tokens, experts, cols = 8203, 8, 1032
    plan, dest, source, *_ = plan_of(tokens, top_k, experts, 16, total=experts + 3, first=1)
    g = torch.Generator().manual_seed(top_k)
    y = torch.randn(source.size, cols, generator=g).to(torch.bfloat16)
    y[torch.from_numpy(source < 0)] = float("nan")
    w = torch.randn(tokens, top_k, generator=g) if weighted else None
    base = torch.randn(tokens, cols, generator=g).to(torch.bfloat16) if based else None
    out = filled((tokens, cols), torch.bfloat16)
    got = pq.qcast_combine(y.to(DEV), plan.dest, None if w is None else w.to(DEV),
                           None if base is None else base.to(DEV), out=out)
    want, mag = moe_ref.combine(y, dest, w, base)
    near(got, want, mag, top_k, "combine")
    # rows that were never sorted
    flat = torch.randn(tokens * top_k, cols, generator=g).to(torch.bfloat16)
    got = pq.qcast_combine(flat.to(DEV), None, None if w is None else w.to(DEV),
                           None if base is None else base.to(DEV), top_k=top_k)
    want, mag = moe_ref.combine(flat, np.arange(tokens * top_k).reshape(tokens, top_k), w, base)
    near(got, want, mag, top_k, "combine of rows as they are")


def test_tokens_without_rows_and_rows_of_several_slots():
    dest = np.array([[-1, -1, 9], [4, 4, 4], [8, 0, -5], [2 ** 31 - 1, -2 ** 31, 8]], np.int32)
    g = torch.Generator().manual_seed(3)
    y = torch.randn(9, 512, generator=g).to(torch.bfloat16)
    base = torch.randn(4, 512, generator=g).to(torch.bfloat16)
    w = torch.randn(4, 3, generator=g)
    w[0] = float("nan")                                     # the weight of a slot without a row
    d = torch.from_numpy(dest).to(DEV)
    w2 = w.clone()
    w2[0] = 0
    for b in (None, base):
        got = pq.qcast_combine(y.to(DEV), d, w.to(DEV), None if b is None else b.to(DEV)).cpu()
        want, mag = moe_ref.combine(y, dest, w2, b)
        near(got, want, mag, 3, "combine")
        assert torch.equal(got[0], base[0] if b is not None else torch.zeros(512, dtype=torch.bfloat16))


def test_infinities_and_nan_go_where_the_sum_puts_them():
    y = torch.ones(4, 8, dtype=torch.bfloat16)
    y[0, 0], y[1, 0], y[2, 1], y[3, 2] = float("inf"), float("-inf"), float("nan"), float("inf")
    out = pq.qcast_combine(y.to(DEV), None, torch.tensor([[1.0, 1.0], [1.0, 0.0]], device=DEV), top_k=2).cpu().float()
    assert out[0, 0].isnan() and out[1, 1].isnan() and out[1, 2].isnan()
    assert torch.equal(out[0, 1:], torch.full((7,), 2.0)) and out[1, 3] == 1


@pytest.mark.parametrize("tokens,top_k", [(1, 8), (5, 3), (64, 1)])
def test_rows_that_were_never_sorted(tokens, top_k):
    g = torch.Generator().manual_seed(tokens)
    y = torch.randn(tokens * top_k, 1032, generator=g).to(torch.bfloat16)
    w = torch.rand(tokens, top_k, generator=g)
    got = pq.qcast_combine(y.to(DEV), None, w.to(DEV), top_k=top_k)
    dest = np.arange(tokens * top_k).reshape(tokens, top_k)
    want, mag = moe_ref.combine(y, dest, w)
    near(got, want, mag, top_k, "combine")


def test_no_slots():
    y = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    base = torch.full((3, 64), 2.0, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(3, 0, dtype=torch.int32, device=DEV)
    assert torch.equal(pq.qcast_combine(y, none, None, base), base)
    assert not pq.qcast_combine(y, none).any()
    assert not pq.qcast_combine(y[:0], torch.zeros(3, 2, dtype=torch.int32, device=DEV)).any()
    assert pq.qcast_combine(y[:0], none[:0]).shape == (0, 64)


@pytest.mark.parametrize("fmt,group,flags", [("e4m3", 128, 0), ("e5m2", 64, 2), ("e4m3", 32, 4), ("e2m1", 32, 6),
                                             ("e5m6", 128, 1)])
@pytest.mark.parametrize("tokens,top_k,experts,align,cols", [(1, 8, 16, 128, 512), (3, 2, 4, 16, 128 * 4),
                                                             (67, 4, 16, 16, 1536), (33, 7, 9, 1, 7168),
                                                             (10, 11, 30, 2, 2048)])
@pytest.mark.parametrize("weighted", [True, False])
def test_backward(fmt, group, flags, tokens, top_k, experts, align, cols, weighted):
    plan, dest, source, offsets, _ = plan_of(tokens, top_k, experts, align, total=experts + 3, first=1)
    g = torch.Generator().manual_seed(tokens)
    rows = source.size
    y = torch.randn(rows, cols, generator=g).to(torch.bfloat16)
    y[torch.from_numpy(source < 0)] = float("nan")
    dout = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    w = torch.rand(tokens, top_k, generator=g) if weighted else None
    wd = None if w is None else w.to(DEV)
    out = filled(pq.code_shape(fmt, rows, cols),
                 {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}.get(fmt, torch.uint8))
    shape, dt = pq.sf_layout_shape(rows, cols, group, flags)
    out_sf = filled(shape, dt)
    dy = filled((rows, cols), torch.bfloat16)
    r = pq.qcast_combine_backward_per_token(dout.to(DEV), plan, y.to(DEV), wd, fmt, group, sf_flags=flags,
                                            want_dy=True, out=out, out_sf=out_sf, dy=dy)
    assert r.out is out and r.out_sf is out_sf and r.dy is dy
    held, live = source >= 0, int(offsets[-1])
    v = np.zeros((rows, cols), np.float32)
    v[held] = dout.float().numpy()[source[held] // top_k]
    if weighted:
        v[held] *= w.reshape(-1).numpy()[source[held], None]
    # the product is the fp32 one; its cast and its rounding are exact operations
    if flags & 5 and weighted:
        q1, s1 = pq.qcast_dispatch_per_token(dout.to(DEV), plan, wd, fmt, group, sf_flags=flags)
        assert np.array_equal(bytes_of(out)[:live], bytes_of(q1)[:live])
        assert np.array_equal(scale_rows(out_sf, rows, flags & 2)[:live], scale_rows(s1, rows, flags & 2)[:live])
    else:
        if flags & 5:
            sorted_x = torch.from_numpy(v).to(torch.bfloat16)
            q_ref, sf_ref = oracle.per_token_sf(workloads.bf16_bits(sorted_x), fmt, group, sf_flags=flags)
            sf_ref = sf_ref.view(np.int32)[:, :rows].T if flags & 2 else sf_ref.view(np.int32)
        else:
            q_ref, sf_ref = oracle.per_token_f32(v, fmt, group)
            sf_ref = sf_ref.view(np.int32)
        assert np.array_equal(bytes_of(out)[:live], q_ref.reshape(rows, -1)[:live])
        assert np.array_equal(scale_rows(out_sf, rows, flags & 2)[:live], sf_ref[:live])
    assert torch.equal(dy.cpu()[:live], torch.from_numpy(v[:live]).to(torch.bfloat16))
    assert (bytes_of(out)[live:] == FILL).all() and (bytes_of(dy)[live:] == FILL).all()
    assert (scale_rows(out_sf, rows, flags & 2)[live:] == -1515870811).all()
    _, dw, mag = moe_ref.combine_grad(dout, y, dest, w)
    bound = mag * ((cols / 64 + 24) * 2.0 ** -24) + 1e-40
    got = r.dw.cpu().double()
    assert ((got - dw).abs() <= bound).all() and (got[torch.from_numpy(dest < 0)] == 0).all()
    # each output by itself is the same
    r2 = pq.qcast_combine_backward_per_token(dout.to(DEV), plan, y.to(DEV), wd, want_codes=False)
    assert torch.equal(r2.dw, r.dw) and r2.out is None and r2.dy is None
    r3 = pq.qcast_combine_backward_per_token(dout.to(DEV), plan, None, wd, fmt, group, sf_flags=flags)
    assert np.array_equal(bytes_of(r3.out)[:live], bytes_of(out)[:live]) and r3.dw is None
    r4 = pq.qcast_combine_backward_per_token(dout.to(DEV), plan, None, wd, want_codes=False, want_dy=True)
    assert torch.equal(r4.dy[:live], dy[:live])


def test_gradient_against_differences():
    """dw is the slope of <combine(w), dout> in each weight: of a sum that is
    linear in the weights, from two fp32-exact settings (0 and 1)."""
    plan, dest, source, *_ = plan_of(6, 2, 4, 1)
    g = torch.Generator().manual_seed(1)
    y = torch.randint(-4, 5, (source.size, 128), generator=g).to(torch.bfloat16)
    dout = torch.randint(-4, 5, (6, 128), generator=g).to(torch.bfloat16)
    dw = pq.qcast_combine_backward_per_token(dout.to(DEV), plan, y.to(DEV), torch.ones(6, 2, device=DEV)).dw.cpu()
    for t in range(6):
        for k in range(2):
            w = torch.zeros(6, 2)
            w[t, k] = 1
            out = pq.qcast_combine(y.to(DEV), plan.dest, w.to(DEV)).cpu()
            assert dw[t, k] == (out.double() * dout.double()).sum()


def test_the_gradient_of_a_dispatch_is_the_unweighted_combine():
    plan, dest, source, *_ = plan_of(31, 3, 6, 16, total=8, first=1)
    g = torch.Generator().manual_seed(1)
    d_sorted = torch.randn(source.size, 256, generator=g).to(torch.bfloat16)
    x = torch.randn(31, 256, generator=g, dtype=torch.float64, requires_grad=True)
    held = torch.from_numpy(np.flatnonzero(source >= 0))
    sorted_x = x[torch.from_numpy(source).long()[held] // 3]
    (grad,) = torch.autograd.grad((sorted_x * d_sorted[held].double()).sum(), x)
    got = pq.qcast_combine(d_sorted.to(DEV), plan.dest)
    near(got, grad, moe_ref.combine(d_sorted, dest)[1], 3, "dispatch gradient")


def test_refusals():
    plan, *_ = plan_of(4, 2, 3, 16)
    rows = plan.source.numel()
    y = torch.zeros(rows, 256, dtype=torch.bfloat16, device=DEV)
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    for bad in (lambda: pq.qcast_combine(y), lambda: pq.qcast_combine(y, top_k=5),
                lambda: pq.qcast_combine(y, plan.dest, top_k=3), lambda: pq.qcast_combine(y, plan.dest.long()),
                lambda: pq.qcast_combine(y, plan.dest, torch.zeros(4, 3, device=DEV)),
                lambda: pq.qcast_combine(y, plan.dest, base=y), lambda: pq.qcast_combine(y.float(), plan.dest),
                lambda: pq.qcast_combine(y[:, :12].contiguous(), plan.dest),
                lambda: pq.qcast_combine(y, plan.dest, out=y),
                lambda: pq.qcast_combine_backward_per_token(x[:3], plan, y),
                lambda: pq.qcast_combine_backward_per_token(x, plan, y[1:]),
                lambda: pq.qcast_combine_backward_per_token(x, plan, want_codes=False),
                lambda: pq.qcast_combine_backward_per_token(x, plan, y, group=16),
                lambda: pq.qcast_combine_backward_per_token(x, plan, y, want_codes=False, out=y),
                lambda: pq.qcast_combine_backward_per_token(x, plan, y, dy=y)):
        with pytest.raises(pq.QcastError):
            bad()
