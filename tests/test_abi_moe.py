"""Refusals of the mixture-of-experts entry points, before any HIP call, and of
their binding."""
import types

import pytest
import torch

import precision_quantization_amd as pq
from conftest import gpu_available

(OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_FORMAT, ERR_GROUP, ERR_LAUNCH, ERR_DEVICE,
 ERR_VALUE) = range(9)
E4M3, E2M1, E5M2, E5M6 = 1, 2, 3, 4
A = 0x10000            # aligned, never dereferenced
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    from precision_quantization_amd import _lib
    return _lib.load()


def sort(lib, ids=A, width=8, tokens=4, top_k=2, experts=8, first=0, align=16, weight=A, dest=A, source=A,
         offsets=A, counts=A, row_weight=A, ws=A):
    return lib.qcast_expert_sort(ids, width, tokens, top_k, experts, first, align, weight, dest, source,
                                 offsets, counts, row_weight, ws, None)


def test_sort(lib):
    for bad in (dict(tokens=-1), dict(top_k=-1), dict(top_k=65), dict(experts=0), dict(experts=1025),
                dict(tokens=1 << 31), dict(tokens=1 << 62), dict(tokens=1 << 30, top_k=2),
                dict(tokens=(1 << 31) - 1, top_k=1, experts=1024, align=1024)):
        assert sort(lib, **bad) == ERR_SHAPE, bad
    for bad in (dict(width=2), dict(align=0), dict(align=3), dict(align=2048), dict(align=-16)):
        assert sort(lib, **bad) == ERR_VALUE, bad
    for k in ("ids", "dest", "source", "offsets", "counts", "weight", "row_weight"):
        assert sort(lib, **{k: None}) == ERR_NULL, k
    assert sort(lib, tokens=4096, ws=None) == ERR_NULL               # two parts
    for k in ("dest", "source", "offsets", "counts", "weight", "row_weight"):
        assert sort(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert sort(lib, ids=A + 4) == sort(lib, ws=A + 8) == sort(lib, ids=A + 2, width=4) == ERR_ALIGN
    assert sort(lib, tokens=0, offsets=None) == ERR_NULL             # written even without slots
    if not gpu_available():
        assert sort(lib, tokens=2048, ws=None) == sort(lib, ids=A + 4, width=4) == ERR_DEVICE
        assert sort(lib, tokens=0, ids=None, dest=None, source=None) == ERR_DEVICE


def codes(lib, q=A, tokens=4, row_bytes=256, sf=A, words=2, fin=0, top_k=2, dest=A, offsets=A, counts=A,
          experts=8, align=16, rows=128, out=A, out_sf=A, fout=0):
    return lib.qcast_dispatch_codes(q, tokens, row_bytes, sf, words, fin, top_k, dest, offsets, counts,
                                    experts, align, rows, out, out_sf, fout, None)


def test_dispatch_codes(lib):
    assert codes(lib, fin=8) == codes(lib, fout=-1) == ERR_FORMAT
    for bad in (dict(row_bytes=8), dict(row_bytes=-16), dict(row_bytes=1 << 31), dict(words=-1), dict(tokens=-1),
                dict(top_k=65), dict(rows=-1), dict(rows=1 << 31), dict(experts=0), dict(experts=1025),
                dict(tokens=1 << 30, words=2), dict(rows=1 << 30, words=2),
                dict(tokens=1 << 21, row_bytes=1 << 20)):
        assert codes(lib, **bad) == ERR_SHAPE, bad
    assert codes(lib, align=0) == codes(lib, align=24) == ERR_VALUE
    for k in ("q", "dest", "out", "sf", "out_sf", "offsets", "counts"):
        assert codes(lib, **{k: None}) == ERR_NULL, k
    for k in ("q", "out"):
        assert codes(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "out_sf", "dest", "offsets", "counts"):
        assert codes(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert codes(lib, tokens=0, q=None) == codes(lib, rows=0, out=None) == codes(lib, top_k=0, dest=None) == OK
    assert codes(lib, row_bytes=0, q=None) == OK
    if not gpu_available():
        assert codes(lib) == codes(lib, offsets=None, counts=None, align=0, experts=0) == ERR_DEVICE


def cast(lib, x=A, tokens=4, cols=256, top_k=2, dest=A, w=A, offsets=A, counts=A, experts=8, align=16, rows=128,
         fmt=E4M3, group=128, clamp_min=0.0, flags=0, q=A, sf=A):
    return lib.qcast_dispatch_per_token(x, tokens, cols, top_k, dest, w, offsets, counts, experts, align, rows,
                                        fmt, group, clamp_min, flags, q, sf, None)


def test_dispatch_per_token(lib):
    assert cast(lib, fmt=9) == cast(lib, flags=8) == ERR_FORMAT
    assert cast(lib, group=16) == ERR_GROUP
    for bad in (dict(cols=200), dict(cols=-128), dict(tokens=-1), dict(rows=-1), dict(top_k=65),
                dict(cols=384, flags=4), dict(rows=1 << 30, cols=512), dict(experts=0), dict(cols=1 << 31)):
        assert cast(lib, **bad) == ERR_SHAPE, bad
    assert cast(lib, clamp_min=NAN) == cast(lib, clamp_min=INF) == cast(lib, align=5) == ERR_VALUE
    for k in ("x", "dest", "q", "sf", "offsets", "counts"):
        assert cast(lib, **{k: None}) == ERR_NULL, k
    for k in ("x", "q"):
        assert cast(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "dest", "w", "offsets", "counts"):
        assert cast(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert cast(lib, tokens=0, x=None) == cast(lib, cols=0, x=None) == cast(lib, rows=0, q=None) == OK


def combine(lib, y=A, rows=128, tokens=4, top_k=2, cols=256, dest=A, w=A, base=A, out=A):
    return lib.qcast_combine(y, rows, tokens, top_k, cols, dest, w, base, out, None)


def test_combine(lib):
    for bad in (dict(cols=12), dict(cols=-8), dict(rows=-1), dict(rows=1 << 31), dict(tokens=-1), dict(top_k=65),
                dict(dest=None, rows=7), dict(tokens=1 << 31), dict(tokens=1 << 30, cols=1024)):
        assert combine(lib, **bad) == ERR_SHAPE, bad
    assert combine(lib, y=None) == combine(lib, out=None) == ERR_NULL
    for k in ("y", "base", "out"):
        assert combine(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("dest", "w"):
        assert combine(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert combine(lib, tokens=0, y=None, out=None) == combine(lib, cols=0, y=None, out=None) == OK
    if not gpu_available():
        assert combine(lib, dest=None, rows=8) == combine(lib, rows=0, y=None) == combine(lib, top_k=0, y=None) == ERR_DEVICE


def bwd(lib, dout=A, y=A, tokens=4, cols=256, top_k=2, dest=A, w=A, offsets=A, counts=A, experts=8, align=16,
        rows=128, fmt=E4M3, group=128, clamp_min=0.0, flags=0, q=A, sf=A, dy=A, dw=A):
    return lib.qcast_combine_backward_per_token(dout, y, tokens, cols, top_k, dest, w, offsets, counts, experts,
                                                align, rows, fmt, group, clamp_min, flags, q, sf, dy, dw, None)


def test_combine_backward(lib):
    assert bwd(lib, fmt=0) == bwd(lib, flags=16) == ERR_FORMAT
    assert bwd(lib, group=256) == ERR_GROUP
    for bad in (dict(cols=200), dict(tokens=-1), dict(rows=1 << 31), dict(top_k=65), dict(cols=384, flags=4),
                dict(cols=0)):
        assert bwd(lib, **bad) == ERR_SHAPE, bad
    assert bwd(lib, clamp_min=INF) == bwd(lib, align=6) == ERR_VALUE
    for k in ("dout", "y", "dest", "q", "sf", "offsets", "counts"):
        assert bwd(lib, **{k: None}) == ERR_NULL, k
    assert bwd(lib, q=None, sf=None, dy=None, dw=None) == ERR_NULL
    for k in ("dout", "y", "q", "dy"):
        assert bwd(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "dest", "w", "dw", "offsets", "counts"):
        assert bwd(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert bwd(lib, tokens=0, dout=None) == bwd(lib, cols=0, dw=None) == bwd(lib, top_k=0) == OK


def matvec(lib, x=A, x_fmt=0, x_sf=None, x_group=128, x_rows=2, w=A, w_sf=A, w_group=32, flags=0, experts=8, ids=A,
           width=8, rows=4, n=64, k=256, od=1, out=A):
    return lib.qcast_matvec_e2m1(x, x_fmt, x_sf, x_group, x_rows, w, w_sf, w_group, flags, experts, ids, width,
                                 rows, n, k, od, out, None)


def test_matvec(lib):
    for bad in (dict(x_fmt=E2M1), dict(x_fmt=9), dict(od=0), dict(od=3), dict(flags=2), dict(flags=8)):
        assert matvec(lib, **bad) == ERR_FORMAT, bad
    assert matvec(lib, w_group=16) == matvec(lib, x_fmt=E4M3, x_sf=A, x_group=256) == ERR_GROUP
    for bad in (dict(rows=-1), dict(rows=5), dict(x_rows=0), dict(x_rows=-1), dict(n=-1), dict(k=-32), dict(k=48),
                dict(k=1 << 24), dict(k=96, w_group=32, flags=4), dict(experts=-1), dict(ids=None),
                dict(k=96, x_fmt=E4M3, x_sf=A, x_group=64), dict(rows=1 << 31, x_rows=1),
                dict(rows=1 << 30, x_rows=1, n=1 << 30), dict(n=1 << 31), dict(experts=1 << 60)):
        assert matvec(lib, **bad) == ERR_SHAPE, bad
    assert matvec(lib, width=2) == ERR_VALUE
    for k in ("x", "w", "w_sf", "out"):
        assert matvec(lib, **{k: None}) == ERR_NULL, k
    assert matvec(lib, x_sf=A) == matvec(lib, x_fmt=E5M2) == ERR_NULL     # scales go with codes
    for k in ("x", "w", "out"):
        assert matvec(lib, **{k: A + 8}) == ERR_ALIGN, k
    assert matvec(lib, w_sf=A + 2) == matvec(lib, ids=A + 4) == matvec(lib, x_fmt=E4M3, x_sf=A + 2) == ERR_ALIGN
    assert matvec(lib, rows=0, x_rows=0, x=None) == matvec(lib, n=0, out=None) == OK
    if not gpu_available():
        assert matvec(lib) == matvec(lib, k=0, x=None, w=None, w_sf=None) == ERR_DEVICE
        assert matvec(lib, ids=None, experts=1) == matvec(lib, ids=A + 4, width=4) == ERR_DEVICE


def test_binding_refuses_what_is_not_on_the_gpu():
    """Every check of the binding that comes before a tensor's device."""
    t = torch.zeros(4, 2, dtype=torch.int64)
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    plan = pq.ExpertPlan(t.int(), torch.zeros(8, dtype=torch.int32), torch.zeros(3, dtype=torch.int32),
                         torch.zeros(2, dtype=torch.int32), None, 1)
    for call in (lambda: pq.qcast_expert_sort(t, 2), lambda: pq.qcast_dispatch_codes(x, plan),
                 lambda: pq.qcast_dispatch_per_token(x, plan), lambda: pq.qcast_combine(x, plan.dest),
                 lambda: pq.qcast_combine_backward_per_token(x, plan),
                 lambda: pq.qcast_matvec_e2m1(x, torch.zeros(8, 64, dtype=torch.uint8), torch.zeros(8, 1)),
                 lambda: pq.qcast_expert_sort(None, 2), lambda: pq.qcast_matvec_e2m1(None, None, None),
                 lambda: pq.qcast_dispatch_codes(types.SimpleNamespace(), plan)):
        with pytest.raises(pq.QcastError):
            call()
