"""qcast_expert_sort against the slot-by-slot reference: every output equal."""
import numpy as np
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(ids, experts, align=1, first=0, weight=None, **kw):
    p = pq.qcast_expert_sort(ids.to(DEV), experts, align, first,
                             weight=None if weight is None else weight.to(DEV), **kw)
    dest, source, offsets, counts, row_weight = moe_ref.sort(ids.numpy(), experts, align, first,
                                                             None if weight is None else weight.numpy())
    torch.cuda.synchronize()
    for name, want in (("offsets", offsets), ("counts", counts), ("dest", dest), ("source", source)):
        got = getattr(p, name)
        assert got.dtype == torch.int32 and np.array_equal(got.cpu().numpy(), want), name
    assert p.align == align
    if weight is None:
        assert p.row_weight is None
    else:
        assert np.array_equal(p.row_weight.cpu().numpy(), row_weight)
    return p


@pytest.mark.parametrize("tokens,top_k,experts,align,dtype", [
    (1, 1, 1, 1, torch.int64), (1, 8, 256, 128, torch.int64), (8, 8, 256, 16, torch.int32),
    (63, 1, 2, 4, torch.int64), (64, 1, 3, 1, torch.int32), (65, 3, 7, 2, torch.int64), (129, 5, 33, 128, torch.int64),
    (1023, 4, 4, 1, torch.int64), (1024, 4, 64, 16, torch.int64), (1025, 4, 1024, 1, torch.int64),
    (2049, 4, 257, 128, torch.int32), (5000, 7, 100, 64, torch.int64), (700, 64, 1000, 1024, torch.int64)])
def test_sizes(tokens, top_k, experts, align, dtype):
    ids = moe_ref.routing(tokens, top_k, experts, seed=tokens, dtype=dtype)
    check(ids, experts, align, weight=torch.rand(tokens, top_k, generator=torch.Generator().manual_seed(1)))
    check(ids, experts, align)


@pytest.mark.parametrize("tokens", [0, 5, 3000])
@pytest.mark.parametrize("experts", [1, 300])
def test_without_slots_or_experts(tokens, experts):
    check(torch.zeros(tokens, 0, dtype=torch.int64), experts, 16, weight=torch.zeros(tokens, 0))
    ids = torch.full((tokens, 3), experts)              # every expert is elsewhere
    check(ids, experts, 16, weight=torch.ones(tokens, 3))
    check(-1 - ids, experts, 16)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_a_share_of_the_experts(dtype):
    ids = moe_ref.routing(3000, 6, 128, seed=4, dtype=dtype)
    for first, experts in ((0, 32), (32, 32), (96, 32), (127, 1), (128, 4)):
        check(ids, experts, 128, first)
    if dtype == torch.int64:                             # differences that pass 32 and 64 bits
        ids = ids.clone()
        ids[::3, 0] = 2 ** 63 - 1
        ids[1::3, 1] = -2 ** 63
        ids[2::3, 2] = (1 << 32) + 40
        check(ids, 32, 16, 32)
        check(ids, 32, 16, -2 ** 63)
        check(ids, 1, 16, 2 ** 63 - 1)


def test_the_same_expert_again_and_again():
    check(torch.zeros(5000, 4, dtype=torch.int64) + 2, 4, 128)
    ids = moe_ref.routing(4500, 8, 5, seed=9, repeat=True)
    check(ids, 5, 8)
    check(torch.arange(9000).view(-1, 1) % 2, 2)


def test_many_parts():
    """More slots than 256 parts of 4096."""
    n = 1 << 21
    ids = moe_ref.routing(n // 2, 2, 16, seed=3, repeat=True)
    p = pq.qcast_expert_sort(ids.to(DEV), 16, 128)
    flat = ids.reshape(-1).numpy()
    order = np.argsort(flat, kind="stable")
    counts = np.bincount(flat, minlength=16)
    offsets = np.concatenate([[0], np.cumsum((counts + 127) // 128 * 128)])
    starts = np.concatenate([[0], np.cumsum(counts)])
    dest = np.empty(n, np.int64)
    dest[order] = offsets[flat[order]] + np.arange(n) - starts[flat[order]]
    assert np.array_equal(p.counts.cpu().numpy(), counts) and np.array_equal(p.offsets.cpu().numpy(), offsets)
    assert np.array_equal(p.dest.cpu().numpy().reshape(-1), dest)
    source = np.full(p.source.numel(), -1)
    source[dest] = np.arange(n)
    assert np.array_equal(p.source.cpu().numpy(), source)


def test_refusals():
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    for bad in (dict(experts=0), dict(experts=1025), dict(experts=4, align=0), dict(experts=4, align=12),
                dict(experts=-3)):
        with pytest.raises(pq.QcastError):
            pq.qcast_expert_sort(ids, **bad)
    for bad in (ids.to(torch.int16), ids.float(), ids[0], ids.t(), ids.unsqueeze(0)):
        with pytest.raises(pq.QcastError):
            pq.qcast_expert_sort(bad, 4)
    for w in (torch.zeros(4, 2, dtype=torch.float64, device=DEV), torch.zeros(4, 3, device=DEV), torch.zeros(4, 2)):
        with pytest.raises(pq.QcastError):
            pq.qcast_expert_sort(ids, 4, weight=w)
