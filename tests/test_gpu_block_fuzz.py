"""Seeded random shapes, types, gates and layouts of the checkpoint and norm
operators, each against the 64-bit formulas within the bounds of block_ref, with
zero rows, large channels and all-equal groups planted."""
import random

import pytest
import torch

import block_ref as br
import precision_quantization_amd as pq
import test_gpu_checkpoint as ck
import test_gpu_norm as nm

pytestmark = pytest.mark.gpu
LAYOUTS = [0, 0, pq.SF_ROUND_POW2, pq.SF_COL_MAJOR, pq.SF_PACKED_UE8M0, pq.SF_PACKED_UE8M0 | pq.SF_COL_MAJOR]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return torch.device("cuda:0")


def layout(rng, groups):
    f = rng.choice(LAYOUTS)
    return f if groups % 4 == 0 or not f & pq.SF_PACKED_UE8M0 else 0


@pytest.mark.parametrize("seed", range(12))
def test_norm(dev, seed):
    rng = random.Random(1000 + seed)
    group = rng.choice([32, 64, 128])
    cols = group * rng.randint(1, 2400 // group)
    rows = rng.choice([1, 2, 3, rng.randint(4, 300)])
    kind, post = rng.choice([None, "channel", "token", "full"]), rng.random() < 0.7
    fmt = rng.choice(["e4m3", "e5m2", "e2m1", "e5m6"])
    flags = layout(rng, cols // group)
    ckpt = rng.choice([None, "e4m3", "e5m2"]) if cols % 128 == 0 else None
    alpha, offset = rng.choice([1.0, 0.5, -1.25, 0.0]), rng.choice([0.0, 1.0])
    v, _ = nm.inputs(rows, cols, kind, post, seed)
    if rows > 2:
        v["h"][1] = 0
        v["y"][1] = 0
        v["y"][2] = 1.5
    nm.check_forward(dev, rows, cols, kind, post, fmt, group, flags, ckpt, alpha, offset, v=v, want_x=rng.random() < 0.5)
    nm.check_backward(dev, rows, cols, kind, post, ckpt or "bf16", fmt, group, flags, alpha, offset, residual=rng.random() < 0.7,
                      want_dy=rng.random() < 0.5, seed=seed)


@pytest.mark.parametrize("seed", range(12))
def test_swiglu_backward_and_recast(dev, seed):
    rng = random.Random(2000 + seed)
    cols = 128 * rng.randint(1, 9)
    rows = rng.choice([1, 127, 128, 129, rng.randint(2, 700)])
    ckpt, fmt = rng.choice(["e4m3", "e5m2"]), rng.choice(["e4m3", "e5m2"])
    tg = (rows + 127) // 128
    flags = layout(rng, cols // 128 if tg % 4 == 0 else 1)
    ck.check_backward(dev, rows, cols, ckpt, fmt, flags, rng.random() < 0.6, rng.choice([0.0, 1.0, 4.0]), seed=seed)
    group = rng.choice([32, 64, 128])
    c = group * rng.randint(1, 1200 // group)
    g = torch.Generator().manual_seed(seed)
    x = br.bf16(g, rows, c, std=rng.choice([1e-3, 1.0, 50.0]))
    x[:, 0] *= 100
    x[rows // 2] = 0
    ck.check_recast(dev, x, ckpt, group, fmt, layout(rng, tg), rng.choice([0.0, 0.25]))
