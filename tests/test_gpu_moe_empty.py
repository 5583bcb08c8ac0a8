"""Plans without rows (no expert of this rank was chosen, and the buffers are as
short as that), in the same manner by every reader of a plan."""
import pytest
import torch

import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_a_plan_without_rows():
    tokens, top_k, cols, experts = 5, 3, 256, 4

    def i32(*shape, fill=0):
        return torch.full(shape, fill, dtype=torch.int32, device=DEV)
    plan = pq.ExpertPlan(i32(tokens, top_k, fill=-1), i32(0), i32(experts + 1), i32(experts), None, 16)
    x = torch.randn(tokens, cols, device=DEV).to(torch.bfloat16)
    y = x[:0]
    w = torch.rand(tokens, top_k, device=DEV)
    q, sf = pq.qcast_dispatch_per_token(x, plan, w)
    assert tuple(q.shape) == (0, cols) and tuple(sf.shape) == (0, 2)
    moved, _ = pq.qcast_dispatch_codes(x, plan)
    assert tuple(moved.shape) == (0, cols)
    assert torch.equal(pq.qcast_combine(y, plan.dest, w, x), x)
    assert not pq.qcast_combine(y, plan.dest, w).any()
    back = pq.qcast_combine_backward_per_token(x, plan, None, w, want_dy=True)
    assert tuple(back.out.shape) == tuple(back.dy.shape) == (0, cols) and back.dw is None
    back = pq.qcast_combine_backward_per_token(x, plan, y, w)
    assert tuple(back.dw.shape) == (tokens, top_k) and not back.dw.any()
    back = pq.qcast_combine_backward_per_token(x, plan, y, w, want_codes=False)
    assert not back.dw.any()


def test_no_expert_here():
    """The same from the sort: rows for slots that all go elsewhere."""
    ids = torch.full((5, 3), 9, device=DEV)
    plan = pq.qcast_expert_sort(ids, 4, 16)
    assert (plan.dest == -1).all() and (plan.source == -1).all() and not plan.offsets.any() and not plan.counts.any()
    x = torch.randn(5, 256, device=DEV).to(torch.bfloat16)
    rows = plan.source.shape[0]
    y = torch.full((rows, 256), float("nan"), dtype=torch.bfloat16, device=DEV)
    out = torch.full((rows, 256), 7, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    back = pq.qcast_combine_backward_per_token(x, plan, y, out=out)
    assert not back.dw.any() and (out.view(torch.uint8) == 7).all()
    pq.qcast_dispatch_per_token(x, plan, out=out)
    assert (out.view(torch.uint8) == 7).all() and torch.equal(pq.qcast_combine(y, plan.dest, None, x), x)


@pytest.mark.parametrize("tokens", [5, 20000])
def test_tokens_without_slots(tokens):
    """top_k 0: the base alone, or zeros."""
    x = torch.randn(tokens, 264, device=DEV).to(torch.bfloat16)
    dest = torch.zeros(tokens, 0, dtype=torch.int32, device=DEV)
    assert torch.equal(pq.qcast_combine(x[:3], dest, None, x), x)
    out = torch.full((tokens, 264), 7.0, dtype=torch.bfloat16, device=DEV)
    assert not pq.qcast_combine(x[:3], dest, out=out).any()
    plan = pq.qcast_expert_sort(torch.zeros(tokens, 0, dtype=torch.int64, device=DEV), 4, 16)
    assert tuple(plan.dest.shape) == (tokens, 0) and plan.source.shape[0] == 0
    assert not plan.offsets.any() and not plan.counts.any()


@pytest.mark.parametrize("experts,k", [(0, 256), (3, 0), (0, 0)])
def test_products_with_no_expert_or_no_k(experts, k):
    x = torch.ones(4, k, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros(experts, 40, k // 2, dtype=torch.uint8, device=DEV)
    sf = torch.ones(experts, 40, k // 32, device=DEV)
    ids = torch.arange(8, device=DEV) % 4
    out = torch.full((8, 40), 7.0, device=DEV)
    assert not pq.qcast_matvec_e2m1(x, w, sf, ids, out_dtype=torch.float32, out=out).any()
