"""Refusals of the checkpoint and norm entry points, before any HIP call."""
import ctypes

import pytest

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


def fwd(lib, h=A, rows=4, cols=256, w=None, fmt=E4M3, group=128, clamp_min=0.0, flags=0, clamp=0.0,
        q=A, sf=A, cf=E4M3, ckpt=A, ckpt_sf=A):
    return lib.qcast_swiglu_checkpoint(h, rows, cols, w, fmt, group, clamp_min, flags, clamp, q, sf,
                                       cf, ckpt, ckpt_sf, None)


def test_swiglu_checkpoint(lib):
    assert fwd(lib, fmt=9) == fwd(lib, cf=E2M1) == fwd(lib, cf=E5M6) == ERR_FORMAT
    assert fwd(lib, flags=8) == ERR_FORMAT
    assert fwd(lib, group=16) == ERR_GROUP
    assert fwd(lib, cols=200) == fwd(lib, rows=-1) == fwd(lib, cols=1 << 19) == ERR_SHAPE
    assert fwd(lib, cols=384, flags=4) == ERR_SHAPE
    # the checkpoint's scale groups pass 2^31 before those of v
    assert fwd(lib, rows=(1 << 30) // 16, cols=4096, group=128) == ERR_SHAPE
    assert fwd(lib, clamp=NAN) == fwd(lib, clamp_min=INF) == ERR_VALUE
    for k in ("h", "q", "sf", "ckpt", "ckpt_sf"):
        assert fwd(lib, **{k: None}) == ERR_NULL, k
    for k in ("h", "q", "ckpt"):
        assert fwd(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "ckpt_sf", "w"):
        assert fwd(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert fwd(lib, rows=0, h=None, q=None, sf=None, ckpt=None, ckpt_sf=None) == OK


def bwd(lib, ckpt=A, ckpt_sf=A, dv=A, rows=4, cols=256, w=None, cf=E4M3, fmt=E4M3, group=128,
        clamp_min=0.0, flags=0, clamp=0.0, q=A, sf=A, dhT=A, dhT_sf=A, vT=A, vT_sf=A, dw=A, ws=A):
    return lib.qcast_swiglu_backward_checkpoint(ckpt, ckpt_sf, dv, rows, cols, w, cf, fmt, group,
                                                clamp_min, flags, clamp, q, sf, dhT, dhT_sf, vT,
                                                vT_sf, dw, ws, None)


def test_swiglu_backward_checkpoint(lib):
    assert bwd(lib, fmt=E2M1) == bwd(lib, fmt=E5M6) == bwd(lib, cf=E2M1) == ERR_FORMAT
    assert bwd(lib, flags=16) == ERR_FORMAT
    assert bwd(lib, group=64) == ERR_GROUP
    assert bwd(lib, cols=192) == bwd(lib, rows=-1) == bwd(lib, cols=1 << 23) == ERR_SHAPE
    assert bwd(lib, rows=1 << 24) == ERR_SHAPE
    # packed words: four channel groups per half, and four token groups when transposed
    assert bwd(lib, cols=256, flags=4) == ERR_SHAPE
    assert bwd(lib, cols=512, flags=4, rows=257) == ERR_SHAPE
    assert bwd(lib, clamp=NAN) == bwd(lib, clamp_min=NAN) == ERR_VALUE
    for k in ("ckpt", "ckpt_sf", "dv", "q", "sf", "ws"):
        assert bwd(lib, **{k: None}) == ERR_NULL, k
    for k in ("dhT", "dhT_sf", "vT", "vT_sf"):          # codes and scales come together
        assert bwd(lib, **{k: None}) == ERR_NULL, k
    for k in ("ckpt", "dv", "q", "dhT", "vT", "ws"):
        assert bwd(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("ckpt_sf", "sf", "w", "dhT_sf", "vT_sf", "dw"):
        assert bwd(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert bwd(lib, rows=0, ckpt=None, dv=None, q=None, sf=None) == OK


def recast(lib, q=A, sf=A, rows=4, cols=256, in_fmt=E4M3, in_group=128, fmt=E4M3, group=128,
           clamp_min=0.0, flags=0, qT=A, out_sf=A):
    return lib.qcast_recast_per_channel_T(q, sf, rows, cols, in_fmt, in_group, fmt, group, clamp_min,
                                          flags, qT, out_sf, None)


def test_recast(lib):
    assert recast(lib, in_fmt=E2M1) == recast(lib, fmt=E5M6) == recast(lib, flags=8) == ERR_FORMAT
    assert recast(lib, in_group=16) == recast(lib, group=64) == ERR_GROUP
    assert recast(lib, cols=200) == recast(lib, rows=-1) == recast(lib, cols=1 << 24) == ERR_SHAPE
    assert recast(lib, rows=1 << 24) == recast(lib, flags=4, rows=100) == ERR_SHAPE
    assert recast(lib, clamp_min=INF) == ERR_VALUE
    for k in ("q", "sf", "qT", "out_sf"):
        assert recast(lib, **{k: None}) == ERR_NULL, k
    for k in ("q", "qT"):
        assert recast(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "out_sf"):
        assert recast(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert recast(lib, rows=0, q=None, qT=None) == OK


def norm(lib, y=A, h=A, rows=4, cols=256, w_post=A, w_pre=A, gate=A, kind=1, alpha=1.0, offset=0.0,
         eps=1e-6, fmt=E4M3, group=128, clamp_min=0.0, flags=0, h_out=A, q=A, sf=A, x_out=None,
         rstd_post=A, rstd_pre=A, cf=E4M3, y_ckpt=A, y_ckpt_sf=A, h_ckpt=A, h_ckpt_sf=A):
    return lib.qcast_norm_per_token(y, h, rows, cols, w_post, w_pre, gate, kind, alpha, offset, eps,
                                    fmt, group, clamp_min, flags, h_out, q, sf, x_out, rstd_post,
                                    rstd_pre, cf, y_ckpt, y_ckpt_sf, h_ckpt, h_ckpt_sf, None)


NO_Y = dict(y=None, w_post=None, gate=None, kind=0, h_out=None, rstd_post=None, y_ckpt=None,
            y_ckpt_sf=None)


def test_norm(lib):
    assert norm(lib, fmt=9) == norm(lib, cf=E2M1) == norm(lib, flags=8) == ERR_FORMAT
    assert norm(lib, group=16) == ERR_GROUP
    assert norm(lib, cols=200) == norm(lib, rows=-1) == norm(lib, cols=16384 + 128) == ERR_SHAPE
    assert norm(lib, cols=64, group=32) == ERR_SHAPE          # checkpoints take groups of 128
    assert norm(lib, rows=1 << 31, cols=128) == norm(lib, cols=384, flags=4) == ERR_SHAPE
    for bad in (dict(eps=NAN), dict(eps=-1.0), dict(eps=INF), dict(alpha=INF), dict(offset=NAN),
                dict(kind=4), dict(kind=-1), dict(clamp_min=NAN)):
        assert norm(lib, **bad) == ERR_VALUE, bad
    assert norm(lib, **{**NO_Y, "alpha": 2.0}) == ERR_VALUE
    for k in ("h", "w_pre", "h_out", "sf", "gate", "y_ckpt", "y_ckpt_sf", "h_ckpt", "h_ckpt_sf"):
        assert norm(lib, **{k: None}) == ERR_NULL, k
    assert norm(lib, q=None, sf=None) == ERR_NULL              # nothing to write x into
    assert norm(lib, kind=0) == ERR_NULL                       # a gate of no kind
    assert norm(lib, w_post=None) == ERR_NULL                  # rstd_post of no norm
    for k in ("w_post", "gate", "h_out", "y_ckpt"):            # what needs y
        kw = dict(NO_Y)
        kw[k] = A
        if k == "gate":
            kw["kind"] = 1
        assert norm(lib, **kw) == ERR_NULL, k
    for k in ("y", "h", "w_post", "w_pre", "gate", "h_out", "q", "x_out", "y_ckpt", "h_ckpt"):
        assert norm(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("sf", "rstd_post", "rstd_pre", "y_ckpt_sf", "h_ckpt_sf"):
        assert norm(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert norm(lib, rows=0, h=None) == norm(lib, cols=0, h=None) == OK
    if not gpu_available():
        assert norm(lib) == norm(lib, **NO_Y) == norm(lib, kind=2, gate=A + 4) == ERR_DEVICE


def nbwd(lib, dx=A, dh_in=A, rows=4, cols=256, saved=E4M3, h=A, h_sf=A, y=A, y_sf=A, r1=A, r2=A,
         w_post=A, w_pre=A, gate=A, kind=1, alpha=1.0, offset=0.0, fmt=E4M3, group=128,
         clamp_min=0.0, flags=0, dh_out=A, q=A, sf=A, dy=None, dw_post=A, dw_pre=A, dgate=A, ws=A):
    return lib.qcast_norm_backward_per_token(dx, dh_in, rows, cols, saved, h, h_sf, y, y_sf, r1, r2,
                                             w_post, w_pre, gate, kind, alpha, offset, fmt, group,
                                             clamp_min, flags, dh_out, q, sf, dy, dw_post, dw_pre,
                                             dgate, ws, None)


def test_norm_backward(lib):
    assert nbwd(lib, fmt=9) == nbwd(lib, saved=E2M1) == nbwd(lib, flags=8) == ERR_FORMAT
    assert nbwd(lib, group=16) == ERR_GROUP
    assert nbwd(lib, cols=200) == nbwd(lib, rows=-1) == nbwd(lib, cols=16384 + 128) == ERR_SHAPE
    assert nbwd(lib, cols=192, group=64) == ERR_SHAPE
    for bad in (dict(alpha=NAN), dict(offset=INF), dict(kind=7), dict(clamp_min=INF)):
        assert nbwd(lib, **bad) == ERR_VALUE, bad
    for k in ("dx", "h", "h_sf", "y_sf", "r1", "r2", "w_pre", "dh_out", "sf", "q", "gate", "ws"):
        assert nbwd(lib, **{k: None}) == ERR_NULL, k
    assert nbwd(lib, q=None, sf=None) == ERR_NULL              # nothing to write dy into
    assert nbwd(lib, w_post=None) == ERR_NULL                  # rstd_post without it
    assert nbwd(lib, y=None) == ERR_NULL                       # scales, weight and gate of nothing
    assert nbwd(lib, saved=0) == ERR_NULL                      # scales of bf16 values
    assert nbwd(lib, kind=0) == ERR_NULL
    for k in ("dx", "dh_in", "h", "y", "w_post", "w_pre", "gate", "dh_out", "q", "dy", "dw_post",
              "dw_pre", "dgate", "ws"):
        assert nbwd(lib, **{k: A + 8}) == ERR_ALIGN, k
    for k in ("h_sf", "y_sf", "r1", "r2", "sf"):
        assert nbwd(lib, **{k: A + 2}) == ERR_ALIGN, k
    assert nbwd(lib, rows=0, dx=None, dw_pre=None, dw_post=None, dgate=None) == OK
    assert nbwd(lib, cols=0) == OK
    if not gpu_available():
        # sums over no rows are zeros, which a kernel has to write
        assert nbwd(lib, rows=0, dx=None) == ERR_DEVICE
        assert nbwd(lib, rows=1) == ERR_DEVICE


def test_norm_checkpoints_of_no_format(lib):
    assert norm(lib, cf=0) == norm(lib, **{**NO_Y, "cf": 0}) == ERR_FORMAT
    assert norm(lib, cf=0, y_ckpt=None, y_ckpt_sf=None) == ERR_FORMAT
    if not gpu_available():       # without checkpoints the format says nothing
        none = dict(y_ckpt=None, y_ckpt_sf=None, h_ckpt=None, h_ckpt_sf=None)
        assert norm(lib, cf=0, **none) == norm(lib, cf=9, **none) == ERR_DEVICE


def test_norm_backward_channel_gate_without_rows(lib):
    # the sums over no rows are written by a kernel that reads the channel gate
    none = dict(rows=0, dx=None, gate=None, dgate=None)
    assert nbwd(lib, kind=1, **none) == ERR_NULL
    if not gpu_available():
        assert nbwd(lib, kind=2, **none) == nbwd(lib, kind=3, **none) == ERR_DEVICE


def test_binding_refuses_cpu_tensors():
    import torch

    import precision_quantization_amd as pq
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    w = torch.zeros(256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.uint8).view(torch.float8_e4m3fn)
    sf = torch.zeros(4, 2)
    for call in (lambda: pq.qcast_swiglu_checkpoint(x),
                 lambda: pq.qcast_swiglu_backward_checkpoint(q, sf, x),
                 lambda: pq.qcast_recast_per_channel_T(q, sf),
                 lambda: pq.qcast_norm_per_token(x, w),
                 lambda: pq.qcast_norm_backward_per_token(x, x, sf, w)):
        with pytest.raises(pq.QcastError):
            call()


def test_workspace_rows_of_header_and_binding(tmp_path):
    import os
    import subprocess

    import precision_quantization_amd as pq
    from conftest import ROOT
    sizes = [(r, c) for r in (0, 1, 255, 256, 257, 2047, 2048, 2056, 8192, 16384, 40000) for c in (32, 512, 544, 1024, 7168, 8192, 16384)]
    src = tmp_path / "ws.c"
    src.write_text('#include <stdio.h>\n#include "qcast.h"\nint main(void) {\n' +
                   "".join(f'  printf("%lld\\n", (long long)qcast_norm_ws_rows({r}, {c}));\n' for r, c in sizes) + "  return 0;\n}\n")
    exe = str(tmp_path / "ws")
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{os.path.join(ROOT, 'include')}", str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [pq.norm_ws_rows(r, c) for r, c in sizes]
    assert pq.norm_ws_rows(8192, 2048) == 1024 and pq.norm_ws_rows(4096, 7168) == 256 and pq.norm_ws_rows(3, 512) == 3
