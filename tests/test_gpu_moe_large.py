"""More workgroups than one grid holds (2^24 of 256 threads, 2^23 of 512): calls
that take several launches. Compared on the GPU with torch's indexing and with
the plain casts, where every value has to be the same; products within the bound
of test_gpu_matvec.py."""
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MANY = (1 << 26) + 1001            # four to a workgroup: 250 workgroups past a grid


@pytest.fixture(autouse=True)
def _memory():
    yield
    torch.cuda.empty_cache()


@pytest.fixture(scope="module")
def plan():
    """Every token to one of five experts, a few to none; long padding at the ends."""
    g = torch.Generator(device=DEV).manual_seed(1)
    ids = torch.randint(0, 6, (MANY, 1), generator=g, device=DEV, dtype=torch.int32)
    ids[-500:] = torch.arange(500, device=DEV, dtype=torch.int32).view(-1, 1) % 7
    plan = pq.qcast_expert_sort(ids, 5, 1024)
    # the sort itself, over 256 workgroups' parts
    want = torch.bincount(ids.view(-1), minlength=7)[:5]
    assert torch.equal(plan.counts.long(), want)
    runs = (want + 1023) // 1024 * 1024
    assert torch.equal(plan.offsets[1:].long(), runs.cumsum(0))
    here = ids.view(-1) < 5
    dest = plan.dest.view(-1).long()
    assert bool((dest[~here] == -1).all())
    for e in range(5):             # in the order of the slots
        mine = dest[ids.view(-1) == e]
        assert torch.equal(mine, torch.arange(mine.numel(), device=DEV) + plan.offsets[e].long())
    return plan


def places(plan):
    """(slots with a row, their rows, the padding rows)"""
    dest = plan.dest.view(-1).long()
    slots = (dest >= 0).nonzero()[:, 0]
    live = torch.arange(plan.source.shape[0], device=DEV) < plan.offsets[-1]
    return slots, dest[slots], (live & (plan.source < 0)).nonzero()[:, 0]


def test_dispatch_codes(plan):
    g = torch.Generator(device=DEV).manual_seed(2)
    x = torch.randint(0, 256, (MANY, 16), generator=g, device=DEV, dtype=torch.uint8)
    out = torch.full((plan.source.shape[0], 16), 7, dtype=torch.uint8, device=DEV)
    pq.qcast_dispatch_codes(x, plan, out=out)
    slots, rows, padding = places(plan)
    assert torch.equal(out[rows], x[slots]) and not out[padding].any()
    assert bool((out[int(plan.offsets[-1]):] == 7).all())


def test_dispatch_per_token(plan):
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(MANY, 32, generator=g, device=DEV, dtype=torch.bfloat16)
    out, out_sf = pq.qcast_dispatch_per_token(x, plan, group=32)
    q, sf = pq.qcast_per_token(x, group=32)
    slots, rows, padding = places(plan)
    out, q = out.view(torch.uint8), q.view(torch.uint8)
    assert torch.equal(out[rows], q[slots]) and torch.equal(out_sf[rows], sf[slots]) and not out[padding].any()


def test_combine():
    g = torch.Generator(device=DEV).manual_seed(4)
    y = torch.randn(1000, 8, generator=g, device=DEV, dtype=torch.bfloat16)
    dest = torch.randint(-1, 1000, (MANY, 3), generator=g, device=DEV, dtype=torch.int32)
    out = pq.qcast_combine(y, dest)
    padded = torch.cat([y.float(), torch.zeros(1, 8, device=DEV)])       # row -1
    want = (padded[dest[:, 0].long()] + padded[dest[:, 1].long()]) + padded[dest[:, 2].long()]
    assert torch.equal(out, want.to(torch.bfloat16))


def test_combine_backward():
    g = torch.Generator(device=DEV).manual_seed(5)
    tokens, top_k, cols = MANY // 8 + 1, 8, 32
    ids = torch.randint(0, 6, (tokens, top_k), generator=g, device=DEV, dtype=torch.int32)
    plan = pq.qcast_expert_sort(ids, 5, 128)
    rows = plan.source.shape[0]
    dout = torch.randint(-8, 9, (tokens, cols), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    y = torch.randint(-8, 9, (rows, cols), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    back = pq.qcast_combine_backward_per_token(dout, plan, y, group=32, want_dy=True)
    q, sf = pq.qcast_per_token(dout, group=32)
    slots, at, padding = places(plan)
    token = slots // top_k
    assert torch.equal(back.out.view(torch.uint8)[at], q.view(torch.uint8)[token])
    assert torch.equal(back.out_sf[at], sf[token]) and torch.equal(back.dy[at], dout[token])
    assert not back.out.view(torch.uint8)[padding].any() and not back.dy[padding].any()
    want = torch.zeros(tokens * top_k, device=DEV)       # whole numbers: sums are exact
    want[slots] = (dout[token].float() * y[at].float()).sum(1)
    assert torch.equal(back.dw.view(-1), want)


def test_matvec():
    n, k = 2 ** 31 - 1, 32                               # 2^23 workgroups of 16 column tiles
    g = torch.Generator(device=DEV).manual_seed(6)
    codes = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    sf = torch.empty(n, 1, device=DEV)
    part = 1 << 27
    for i in range(0, n, part):
        codes[i:i + part] = torch.randint(0, 256, (min(part, n - i), k // 2), generator=g, device=DEV, dtype=torch.uint8)
        sf[i:i + part] = torch.exp(torch.randn(min(part, n - i), 1, generator=g, device=DEV))
    x = torch.randn(1, k, generator=g, device=DEV, dtype=torch.bfloat16)
    out = pq.qcast_matvec_e2m1(x, codes, sf, out=torch.full((1, n), float("nan"), dtype=torch.bfloat16, device=DEV))
    value = torch.from_numpy(moe_ref.E2M1).to(DEV)
    for i in range(0, n, part):
        assert not out[0, i:i + part].isnan().any()
    for i in [0, 1 << 30, n - 5 * (1 << 20)] + [((1 << 23) - 8 * j) * 256 - (1 << 16) for j in (1, 2)]:
        c, s = codes[i:i + (5 << 20)].long(), sf[i:i + (5 << 20)].double()
        w = torch.stack([value[c & 15], value[c >> 4]], dim=2).flatten(1) * s
        want, mag = w @ x[0].double(), w.abs() @ x[0].double().abs()
        bound = mag * ((k / 32 + 66) * 2.0 ** -23) + 1e-38
        assert ((out[0, i:i + (5 << 20)].double() - want).abs() <= (want.abs() + bound) * 2.0 ** -8 + bound).all()
