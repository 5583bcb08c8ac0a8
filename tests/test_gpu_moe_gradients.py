"""The gradient of a weighted dispatch, as the library's operators give it: the
weighted combine of the rows' gradient, and dw of the combine's gradient with x
in dout's place. Against autograd and central differences in 64 bits (the rows
are linear in x and in the weights, so differences have only their own rounding).
Bounds as in test_gpu_combine.py."""
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from test_gpu_combine import near

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("tokens,top_k,experts,align,cols", [(1, 1, 1, 1, 128), (37, 3, 6, 16, 256), (130, 8, 20, 128, 1920)])
@pytest.mark.parametrize("weighted", [True, False])
def test_gradient_of_a_dispatch(tokens, top_k, experts, align, cols, weighted):
    g = torch.Generator().manual_seed(tokens)
    ids = moe_ref.routing(tokens, top_k, experts, seed=tokens, total=experts + 2)
    plan = pq.qcast_expert_sort(ids.to(DEV), experts, align)
    dest = plan.dest.cpu()
    rows = plan.source.shape[0]
    x = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    w = torch.randn(tokens, top_k, generator=g) if weighted else None
    grad = torch.randn(rows, cols, generator=g).to(torch.bfloat16)     # of the dispatched rows
    grad[(plan.source < 0).cpu()] = float("nan")                      # no slot: not read
    here = (dest >= 0).double()
    at = dest.long().clamp_min(0)

    def loss(xv, wv):
        slots = grad.double().nan_to_num()[at] * xv.unsqueeze(1) * (wv * here).unsqueeze(2)
        return slots.sum()
    xv = x.double().requires_grad_()
    wv = (torch.ones(tokens, top_k) if w is None else w).double().requires_grad_()
    dx, dw = torch.autograd.grad(loss(xv, wv), (xv, wv))
    wd = None if w is None else w.to(DEV)
    got_dx = pq.qcast_combine(grad.to(DEV), plan.dest, wd)
    want, mag = moe_ref.combine(grad, dest.numpy(), w)
    assert torch.allclose(want, dx, rtol=1e-12, atol=1e-12)
    near(got_dx, dx, mag, top_k, "dx")
    got_dw = pq.qcast_combine_backward_per_token(x.to(DEV), plan, grad.to(DEV), wd, want_codes=False).dw.double().cpu()
    mag = (grad.double().nan_to_num()[at].abs() * x.double().abs().unsqueeze(1)).sum(2) * here
    bound = mag * (cols / 64 + 24) * 2.0 ** -24
    assert ((got_dw - dw).abs() <= bound).all() and not got_dw[dest < 0].any()
    for t, k in {(0, 0), (tokens - 1, top_k - 1), (tokens // 2, top_k // 2)}:
        step = torch.zeros(tokens, top_k, dtype=torch.float64)
        step[t, k] = 2.0 ** -10
        d = (loss(xv, wv + step) - loss(xv, wv - step)).item() * 2.0 ** 9
        # the losses' own sums: 2^-53 of their magnitudes for every addition, over the step
        own = ((mag * wv.abs()).sum().item() + mag[t, k].item()) * tokens * top_k * cols * 2.0 ** -53 * 2.0 ** 10
        assert abs(d - got_dw[t, k].item()) <= bound[t, k].item() + own
        step = torch.zeros(tokens, cols, dtype=torch.float64)
        step[t, 5 * k] = 2.0 ** -10
        d = (loss(xv + step, wv) - loss(xv - step, wv)).item() * 2.0 ** 9
        v, m = got_dx[t, 5 * k].item(), (grad.double().nan_to_num()[at[t], 5 * k] * (wv * here)[t]).abs().sum().item()
        assert abs(d - v) <= abs(d) * 2.0 ** -8 + m * (top_k * 2.0 ** -24 + 2.0 ** -30) * 1.01 + own
