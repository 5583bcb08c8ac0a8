"""MI355X (gfx950) quantization casts: a thin Python binding of libqcast.so.

Each ``qcast_*`` function has the name of the C entry point it calls and does
argument marshalling only: it checks that tensors are on one GPU and
contiguous, allocates outputs that were not given, and passes raw pointers
and torch's current stream. Every step of a cast runs in the HIP kernels; a
missing library raises ``QcastError``.

Outputs: E4M3 codes as ``torch.float8_e4m3fn`` and E5M2 codes as
``torch.float8_e5m2`` (one byte per code), E2M1 codes as ``torch.uint8`` with
two codes per byte (low nibble = even column), E5M6 codes as ``torch.uint8``
with two 12-bit codes per three bytes (a little-endian bit stream), scales as
``torch.float32``. Every cast takes every format; codes are packed along the
rows of its output (``code_shape``): columns for the per-token, SwiGLU,
per-block and per-channel casts, tokens for the transposed per-channel ones.

Around the products of a training step, the SwiGLU input and the norms' inputs
can be kept as 8-bit codes (``qcast_swiglu_checkpoint``, ``qcast_norm_per_token``)
and read by the backward pass (``qcast_swiglu_backward_checkpoint``,
``qcast_norm_backward_per_token``, ``qcast_recast_per_channel_T``). These calls
allocate what they return for the stream they run on.

Around the products of a mixture of experts: slots sorted by expert
(``qcast_expert_sort``, an ``ExpertPlan``), rows brought there and back
(``qcast_dispatch_codes``, ``qcast_dispatch_per_token``, ``qcast_combine``,
``qcast_combine_backward_per_token``), and for decoding products of a few rows
with E2M1 weights (``qcast_matvec_e2m1``).

``per_token_cast(x, fmt='e4m3', num_per_channels=128) -> (out, out_sf)``
mirrors the call shown in the quick start of the page
"DeepSeek开源TileKernels：用Python写的GPU算子逼近硬件性能上限".
"""
from collections import namedtuple
from contextlib import nullcontext

import torch

from ._lib import (FMT_E2M1, FMT_E4M3, FMT_E5M2, FMT_E5M6, GATE_CHANNEL, GATE_FULL, GATE_NONE,
                   GATE_TOKEN, OUT_BF16, OUT_F32, SF_COL_MAJOR, SF_PACKED_UE8M0,
                   SF_ROUND_POW2, QcastError, check, fmt_id, load)

__all__ = ["qcast_per_token", "qcast_e2m1", "qcast_swiglu_per_token", "qcast_per_block",
           "qcast_per_channel_T", "qcast_cast_back", "qcast_per_token_sf",
           "qcast_swiglu_per_token_sf", "qcast_swiglu_per_token_ex",
           "qcast_swiglu_backward_per_token", "qcast_swiglu_per_channel_T", "qcast_per_channel",
           "qcast_swiglu_per_token_noalloc", "qcast_per_block_sf", "qcast_per_channel_sf",
           "qcast_per_channel_T_sf", "qcast_swiglu_per_channel_T_sf",
           "qcast_swiglu_backward_per_token_sf", "qcast_swiglu_checkpoint",
           "qcast_swiglu_backward_checkpoint", "qcast_swiglu_backward_checkpoint_ex",
           "qcast_recast_per_channel_T",
           "qcast_norm_per_token", "qcast_norm_backward_per_token", "SwigluGrad", "NormOut",
           "NormGrad", "qcast_expert_sort", "qcast_dispatch_codes", "qcast_dispatch_per_token",
           "qcast_combine", "qcast_combine_backward_per_token", "qcast_matvec_e2m1", "ExpertPlan",
           "CombineGrad", "expert_rows", "sf_layout_shape", "SF_ROUND_POW2", "SF_COL_MAJOR",
           "SF_PACKED_UE8M0", "qcast_abi_version", "qcast_set_num_cus", "qcast_bench_copy",
           "qcast_bench_check_scale", "qcast_bench_time_next",
           "qcast_bench_per_channel_T_traffic",
           "per_token_cast",
           "QcastError", "FMT_E4M3", "FMT_E2M1", "FMT_E5M2", "FMT_E5M6", "code_shape"]


def _bf16_input(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise QcastError(1, f"{name} must be a CUDA (HIP) tensor")
    if x.dtype != torch.bfloat16:
        raise QcastError(2, f"{name} must be bfloat16, got {x.dtype}")
    if x.dim() != 2 or not x.is_contiguous():
        raise QcastError(2, f"{name} must be a contiguous 2-D tensor")
    return x


def _gate_up(h, name="h"):
    """A SwiGLU input ``[rows, 2*cols]`` (gate | up): (h, rows, cols). The
    width must be even, or the C ABI would walk h with a row stride one
    element short."""
    if isinstance(h, torch.Tensor) and h.dim() == 2 and h.shape[1] % 2:
        raise QcastError(2, f"{name} must have an even number of columns (gate | up), "
                            f"got {h.shape[1]}")
    h = _bf16_input(h, name)
    rows, two_n = h.shape
    return h, rows, two_n // 2


def _out(t, shape, dtype, device, name):
    if t is None:
        return torch.empty(*shape, dtype=dtype, device=device)     # 0.4 us less than a tuple
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or t.device != device or \
            not t.is_contiguous():
        raise QcastError(2, f"{name} must be a contiguous {dtype} tensor of shape {shape} "
                            f"on {device}")
    return t


def _stream(device, stream):
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.current_stream(device).cuda_stream


def _row_weight(row_weight, rows, device):
    if row_weight is None:
        return None
    if not isinstance(row_weight, torch.Tensor) or row_weight.dtype != torch.float32 or \
            tuple(row_weight.shape) != (rows,) or row_weight.device != device or \
            not row_weight.is_contiguous():
        raise QcastError(2, "row_weight must be a contiguous float32 [rows] tensor on h's device")
    return row_weight.data_ptr()


def _counter(clamp_count, device):
    """Device int64 [1] tensor the clamp count is added to (or None)."""
    if clamp_count is None:
        return None
    if not isinstance(clamp_count, torch.Tensor) or clamp_count.dtype != torch.int64 or \
            clamp_count.numel() != 1 or clamp_count.device != device:
        raise QcastError(2, "clamp_count must be a one-element int64 tensor on h's device")
    return clamp_count.data_ptr()


COUNT_WS_BYTES = 8192           # QCAST_COUNT_WS_BYTES
_count_ws_cache = {}


def _count_ws(count_workspace, clamp_count, device, stream_handle):
    """Device pointer of the clamp-count workspace (QCAST_COUNT_WS_BYTES,
    zero between calls): the caller's tensor; none when ``count_workspace``
    is False, when nothing is counted, or (for the default None) under graph
    capture, since a graph may be replayed on any stream; else, for None,
    one int64 tensor kept per device and stream (each call leaves it
    zeroed, and calls on one stream are ordered).

    The first counting call on a (device, stream) allocates that tensor
    (8 KB) and zeroes it with a fill kernel enqueued on the same stream,
    ahead of the cast: nothing waits on the host. Callers that must not
    allocate inside the call pass their own ``count_workspace``, or
    ``False`` (the capped grid, no workspace)."""
    if clamp_count is None or count_workspace is False:
        return None
    if count_workspace is None:
        if torch.cuda.is_current_stream_capturing():
            return None     # a graph may replay on any stream: no shared workspace
        key = (device, stream_handle)
        ws = _count_ws_cache.get(key)
        if ws is None:
            # allocated for, and zeroed on, the stream the cast runs on
            if torch.cuda.current_stream(device).cuda_stream == stream_handle:
                ws = torch.zeros(COUNT_WS_BYTES // 8, dtype=torch.int64, device=device)
            else:
                with torch.cuda.stream(torch.cuda.ExternalStream(stream_handle, device=device)):
                    ws = torch.zeros(COUNT_WS_BYTES // 8, dtype=torch.int64, device=device)
            _count_ws_cache[key] = ws
        return ws.data_ptr()
    if not isinstance(count_workspace, torch.Tensor) or count_workspace.device != device or \
            not count_workspace.is_contiguous() or \
            count_workspace.numel() * count_workspace.element_size() < COUNT_WS_BYTES:
        raise QcastError(2, f"count_workspace must be a contiguous tensor of at least "
                            f"{COUNT_WS_BYTES} bytes on h's device")
    return count_workspace.data_ptr()


def code_shape(fmt, rows, cols):
    """Shape of the uint8/float8 code tensor of a per-token cast."""
    f = fmt_id(fmt)
    if f == FMT_E2M1:
        return (rows, cols // 2)
    if f == FMT_E5M6:
        return (rows, cols // 2 * 3)
    return (rows, cols)


def _code_dtype(f):
    return {FMT_E4M3: torch.float8_e4m3fn, FMT_E5M2: torch.float8_e5m2}.get(f, torch.uint8)


def qcast_per_token(x, fmt="e4m3", group=128, clamp_min=0.0, out=None, out_sf=None,
                    stream=None):
    """Per-token cast of bf16 ``x [rows, cols]``; see include/qcast.h."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    qshape = code_shape(f, rows, cols)
    out = _out(out, qshape, _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (rows, cols // group if group > 0 else 0), torch.float32, x.device,
                  "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_token(x.data_ptr(), rows, cols, f, group, clamp_min,
                                     out.data_ptr(), out_sf.data_ptr(), _stream(x.device, stream)),
              "qcast_per_token")
    return out, out_sf


def sf_layout_shape(rows, cols, group, sf_flags):
    """(shape, dtype) of the scale tensor of a layout (include/qcast.h)."""
    groups = cols // group
    rows_pad = (rows + 3) // 4 * 4
    if sf_flags & SF_PACKED_UE8M0:
        shape = (groups // 4, rows_pad) if sf_flags & SF_COL_MAJOR else (rows, groups // 4)
        return shape, torch.int32
    shape = (groups, rows_pad) if sf_flags & SF_COL_MAJOR else (rows, groups)
    return shape, torch.float32


def qcast_per_token_sf(x, fmt="e4m3", group=128, clamp_min=0.0, sf_flags=0, out=None,
                       out_sf=None, stream=None):
    """qcast_per_token with a scale-factor layout; out_sf is float32 or int32
    (packed UE8M0 words) of ``sf_layout_shape``."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    qshape = code_shape(f, rows, cols)
    out = _out(out, qshape, _code_dtype(f), x.device, "out")
    shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, x.device, "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_token_sf(x.data_ptr(), rows, cols, f, group, clamp_min, sf_flags,
                                        out.data_ptr(), out_sf.data_ptr(),
                                        _stream(x.device, stream)), "qcast_per_token_sf")
    return out, out_sf


def qcast_swiglu_per_token_sf(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                              sf_flags=0, out=None, out_sf=None, stream=None):
    """qcast_swiglu_per_token with a scale-factor layout."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = None
    if row_weight is not None:
        if row_weight.dtype != torch.float32 or tuple(row_weight.shape) != (rows,) or \
                row_weight.device != h.device or not row_weight.is_contiguous():
            raise QcastError(2, "row_weight must be a contiguous float32 [rows] tensor on h's device")
        wptr = row_weight.data_ptr()
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), h.device, "out")
    shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, h.device, "out_sf")
    with torch.cuda.device(h.device):
        check(load().qcast_swiglu_per_token_sf(h.data_ptr(), rows, cols, wptr, f, group, clamp_min,
                                               sf_flags, out.data_ptr(), out_sf.data_ptr(),
                                               _stream(h.device, stream)),
              "qcast_swiglu_per_token_sf")
    return out, out_sf


def qcast_swiglu_per_token_ex(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                              sf_flags=0, swiglu_clamp=0.0, clamp_count=None, out=None,
                              out_sf=None, stream=None, count_workspace=None):
    """SwiGLU with the optional clamp (gate <= c, up in [-c, c]) fused with the
    per-token cast. ``clamp_count``: an int64 [1] device tensor to which the
    number of clamped values is added, or None. ``count_workspace``: see
    ``_count_ws`` (the default keeps one per device and stream)."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = _row_weight(row_weight, rows, h.device)
    cptr = _counter(clamp_count, h.device)
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), h.device, "out")
    shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, h.device, "out_sf")
    with torch.cuda.device(h.device):
        sh = _stream(h.device, stream)
        wsptr = _count_ws(count_workspace, clamp_count, h.device, sh)
        check(load().qcast_swiglu_per_token_ex(h.data_ptr(), rows, cols, wptr, f, group, clamp_min,
                                               sf_flags, swiglu_clamp, out.data_ptr(),
                                               out_sf.data_ptr(), cptr, wsptr, sh),
              "qcast_swiglu_per_token_ex")
    return out, out_sf


def qcast_swiglu_per_token_noalloc(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                                   sf_flags=0, swiglu_clamp=0.0, clamp_count=None, out=None,
                                   out_sf=None, stream=None):
    """qcast_swiglu_per_token_ex for callers that cannot allocate: the clamp
    count goes through the library's own device array (include/qcast.h), so
    with ``out`` and ``out_sf`` given nothing is allocated; calls that may
    overlap on one GPU race on that array."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = _row_weight(row_weight, rows, h.device)
    cptr = _counter(clamp_count, h.device)
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), h.device, "out")
    shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, h.device, "out_sf")
    with torch.cuda.device(h.device):
        check(load().qcast_swiglu_per_token_noalloc(h.data_ptr(), rows, cols, wptr, f, group,
                                                    clamp_min, sf_flags, swiglu_clamp,
                                                    out.data_ptr(), out_sf.data_ptr(), cptr,
                                                    _stream(h.device, stream)),
              "qcast_swiglu_per_token_noalloc")
    return out, out_sf


def qcast_swiglu_backward_per_token(h, dv, row_weight=None, fmt="e4m3", group=128,
                                    clamp_min=0.0, swiglu_clamp=0.0, out=None, out_sf=None,
                                    stream=None):
    """SwiGLU backward fused with the per-token cast of ``[dgate | dup]``:
    ``out [rows, 2*cols]``, ``out_sf [rows, 2*cols/group]``."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    two_n = 2 * cols
    dv = _bf16_input(dv, "dv")
    if tuple(dv.shape) != (rows, cols) or dv.device != h.device:
        raise QcastError(2, f"dv must be [{rows}, {cols}] on h's device")
    wptr = _row_weight(row_weight, rows, h.device)
    out = _out(out, code_shape(f, rows, two_n), _code_dtype(f), h.device, "out")
    out_sf = _out(out_sf, (rows, two_n // group if group > 0 else 0), torch.float32, h.device,
                  "out_sf")
    with torch.cuda.device(h.device):
        check(load().qcast_swiglu_backward_per_token(h.data_ptr(), dv.data_ptr(), rows, cols,
                                                     wptr, f, group, clamp_min, swiglu_clamp,
                                                     out.data_ptr(), out_sf.data_ptr(),
                                                     _stream(h.device, stream)),
              "qcast_swiglu_backward_per_token")
    return out, out_sf


def qcast_swiglu_backward_per_token_sf(h, dv, row_weight=None, fmt="e4m3", group=128,
                                       clamp_min=0.0, sf_flags=0, swiglu_clamp=0.0, out=None,
                                       out_sf=None, stream=None):
    """qcast_swiglu_backward_per_token with a scale-factor layout over the
    rows ``[dgate | dup]`` of 2*cols values (``sf_layout_shape(rows, 2*cols,
    group, sf_flags)``)."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    two_n = 2 * cols
    dv = _bf16_input(dv, "dv")
    if tuple(dv.shape) != (rows, cols) or dv.device != h.device:
        raise QcastError(2, f"dv must be [{rows}, {cols}] on h's device")
    wptr = _row_weight(row_weight, rows, h.device)
    out = _out(out, code_shape(f, rows, two_n), _code_dtype(f), h.device, "out")
    shape, dt = sf_layout_shape(rows, two_n, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, h.device, "out_sf")
    with torch.cuda.device(h.device):
        check(load().qcast_swiglu_backward_per_token_sf(h.data_ptr(), dv.data_ptr(), rows, cols,
                                                        wptr, f, group, clamp_min, sf_flags,
                                                        swiglu_clamp, out.data_ptr(),
                                                        out_sf.data_ptr(),
                                                        _stream(h.device, stream)),
              "qcast_swiglu_backward_per_token_sf")
    return out, out_sf


def qcast_swiglu_per_channel_T_sf(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                                  sf_flags=0, swiglu_clamp=0.0, clamp_count=None, out=None,
                                  out_sf=None, stream=None, count_workspace=None):
    """qcast_swiglu_per_channel_T with a scale-factor layout: the per-token
    layouts of the transposed values (``sf_layout_shape(cols, rows, group,
    sf_flags)``: rows are the channels)."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = _row_weight(row_weight, rows, h.device)
    cptr = _counter(clamp_count, h.device)
    out = _out(out, code_shape(f, cols, rows), _code_dtype(f), h.device, "out")
    shape, dt = sf_layout_shape(cols, rows, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, h.device, "out_sf")
    with torch.cuda.device(h.device):
        sh = _stream(h.device, stream)
        wsptr = _count_ws(count_workspace, clamp_count, h.device, sh)
        check(load().qcast_swiglu_per_channel_T_sf(h.data_ptr(), rows, cols, wptr, f, group,
                                                   clamp_min, sf_flags, swiglu_clamp,
                                                   out.data_ptr(), out_sf.data_ptr(), cptr,
                                                   wsptr, sh),
              "qcast_swiglu_per_channel_T_sf")
    return out, out_sf


def qcast_swiglu_per_channel_T(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                               swiglu_clamp=0.0, clamp_count=None, out=None, out_sf=None,
                               stream=None, count_workspace=None):
    """SwiGLU fused with the per-channel cast written transposed:
    ``out [cols, rows]``, ``out_sf [cols, rows/group]``; ``clamp_count`` and
    ``count_workspace`` as in qcast_swiglu_per_token_ex."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = _row_weight(row_weight, rows, h.device)
    cptr = _counter(clamp_count, h.device)
    out = _out(out, code_shape(f, cols, rows), _code_dtype(f), h.device, "out")
    out_sf = _out(out_sf, (cols, rows // group if group > 0 else 0), torch.float32, h.device,
                  "out_sf")
    with torch.cuda.device(h.device):
        sh = _stream(h.device, stream)
        wsptr = _count_ws(count_workspace, clamp_count, h.device, sh)
        check(load().qcast_swiglu_per_channel_T(h.data_ptr(), rows, cols, wptr, f, group,
                                                clamp_min, swiglu_clamp, out.data_ptr(),
                                                out_sf.data_ptr(), cptr, wsptr, sh),
              "qcast_swiglu_per_channel_T")
    return out, out_sf


def qcast_per_channel(x, fmt="e4m3", group=128, clamp_min=0.0, out=None, out_sf=None,
                      stream=None):
    """Per-channel cast in the input layout: ``out [tokens, channels]``,
    ``out_sf [tokens/group, channels]``."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (rows // group if group > 0 else 0, cols), torch.float32, x.device,
                  "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_channel(x.data_ptr(), rows, cols, f, group, clamp_min,
                                       out.data_ptr(), out_sf.data_ptr(),
                                       _stream(x.device, stream)), "qcast_per_channel")
    return out, out_sf


def qcast_e2m1(x, group=32, clamp_min=0.0, out=None, out_sf=None, stream=None):
    """Per-token cast to packed E2M1: ``out [rows, cols/2]`` uint8."""
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, (rows, cols // 2), torch.uint8, x.device, "out")
    out_sf = _out(out_sf, (rows, cols // group if group > 0 else 0), torch.float32, x.device,
                  "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_e2m1(x.data_ptr(), rows, cols, group, clamp_min, out.data_ptr(),
                                out_sf.data_ptr(), _stream(x.device, stream)), "qcast_e2m1")
    return out, out_sf


def qcast_swiglu_per_token(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0, out=None,
                           out_sf=None, stream=None):
    """SwiGLU of ``h [rows, 2N]`` (gate | up) times ``row_weight [rows]`` (fp32
    or None), cast per token: ``out [rows, N]``, ``out_sf [rows, N/group]``."""
    f = fmt_id(fmt)
    h, rows, cols = _gate_up(h)
    wptr = None
    if row_weight is not None:
        if row_weight.dtype != torch.float32 or tuple(row_weight.shape) != (rows,) or \
                row_weight.device != h.device or not row_weight.is_contiguous():
            raise QcastError(2, "row_weight must be a contiguous float32 [rows] tensor on h's device")
        wptr = row_weight.data_ptr()
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), h.device, "out")
    out_sf = _out(out_sf, (rows, cols // group if group > 0 else 0), torch.float32, h.device,
                  "out_sf")
    with torch.cuda.device(h.device):
        check(load().qcast_swiglu_per_token(h.data_ptr(), rows, cols, wptr, f, group, clamp_min,
                                            out.data_ptr(), out_sf.data_ptr(),
                                            _stream(h.device, stream)), "qcast_swiglu_per_token")
    return out, out_sf


def qcast_per_block(x, fmt="e4m3", block=128, clamp_min=0.0, out=None, out_sf=None,
                    stream=None):
    """One scale per ``block x block`` tile: ``out [rows, cols]``,
    ``out_sf [rows/block, cols/block]``."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (rows // block if block > 0 else 0, cols // block if block > 0 else 0),
                  torch.float32, x.device, "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_block(x.data_ptr(), rows, cols, f, block, clamp_min, out.data_ptr(),
                                     out_sf.data_ptr(), _stream(x.device, stream)),
              "qcast_per_block")
    return out, out_sf


def qcast_per_channel_T(x, fmt="e4m3", group=128, clamp_min=0.0, out=None, out_sf=None,
                        stream=None):
    """Per-channel cast of ``x [tokens, channels]`` written transposed:
    ``out [channels, tokens]``, ``out_sf [channels, tokens/group]``."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, cols, rows), _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (cols, rows // group if group > 0 else 0), torch.float32, x.device,
                  "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_channel_T(x.data_ptr(), rows, cols, f, group, clamp_min,
                                         out.data_ptr(), out_sf.data_ptr(),
                                         _stream(x.device, stream)), "qcast_per_channel_T")
    return out, out_sf


def qcast_per_block_sf(x, fmt="e4m3", block=128, clamp_min=0.0, sf_flags=0, out=None,
                       out_sf=None, stream=None):
    """qcast_per_block with round_sf (``sf_flags`` 0 or SF_ROUND_POW2);
    ``out_sf [rows/block, cols/block]`` float32."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (rows // block if block > 0 else 0, cols // block if block > 0 else 0),
                  torch.float32, x.device, "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_block_sf(x.data_ptr(), rows, cols, f, block, clamp_min, sf_flags,
                                        out.data_ptr(), out_sf.data_ptr(),
                                        _stream(x.device, stream)), "qcast_per_block_sf")
    return out, out_sf


def qcast_per_channel_sf(x, fmt="e4m3", group=128, clamp_min=0.0, sf_flags=0, out=None,
                         out_sf=None, stream=None):
    """qcast_per_channel with round_sf (``sf_flags`` 0 or SF_ROUND_POW2)."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, rows, cols), _code_dtype(f), x.device, "out")
    out_sf = _out(out_sf, (rows // group if group > 0 else 0, cols), torch.float32, x.device,
                  "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_channel_sf(x.data_ptr(), rows, cols, f, group, clamp_min, sf_flags,
                                          out.data_ptr(), out_sf.data_ptr(),
                                          _stream(x.device, stream)), "qcast_per_channel_sf")
    return out, out_sf


def qcast_per_channel_T_sf(x, fmt="e4m3", group=128, clamp_min=0.0, sf_flags=0, out=None,
                           out_sf=None, stream=None):
    """qcast_per_channel_T with a scale-factor layout: the per-token layouts
    of ``x^T`` (``sf_layout_shape(channels, tokens, group, sf_flags)``)."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, code_shape(f, cols, rows), _code_dtype(f), x.device, "out")
    shape, dt = sf_layout_shape(cols, rows, group if group > 0 else 1, sf_flags)
    out_sf = _out(out_sf, shape, dt, x.device, "out_sf")
    with torch.cuda.device(x.device):
        check(load().qcast_per_channel_T_sf(x.data_ptr(), rows, cols, f, group, clamp_min,
                                            sf_flags, out.data_ptr(), out_sf.data_ptr(),
                                            _stream(x.device, stream)), "qcast_per_channel_T_sf")
    return out, out_sf


def qcast_cast_back(q, sf, fmt="e4m3", group=128, out_dtype=torch.bfloat16, out=None,
                    stream=None):
    """Dequantize per-token codes ``q`` with scales ``sf [rows, cols/group]``
    to ``out [rows, cols]`` (bf16 or fp32): decode(q) * sf."""
    f = fmt_id(fmt)
    if isinstance(q, torch.Tensor) and q.dim() == 2 and f == FMT_E5M6 and q.shape[1] % 3:
        raise QcastError(2, f"E5M6 codes take three bytes per pair of columns: q's width "
                            f"{q.shape[1]} is not a multiple of 3")
    if not (isinstance(q, torch.Tensor) and q.is_cuda and q.dim() == 2 and q.is_contiguous()):
        raise QcastError(2, "q must be a contiguous 2-D CUDA tensor")
    if q.element_size() != 1:
        raise QcastError(2, "q must hold one byte per element")
    rows = q.shape[0]
    cols = {FMT_E2M1: q.shape[1] * 2, FMT_E5M6: q.shape[1] // 3 * 2}.get(f, q.shape[1])
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise QcastError(4, "out_dtype must be torch.bfloat16 or torch.float32")
    if sf.dtype != torch.float32 or tuple(sf.shape) != (rows, cols // group if group > 0 else 0) \
            or sf.device != q.device or not sf.is_contiguous():
        raise QcastError(2, "sf must be a contiguous float32 [rows, cols/group] tensor on q's device")
    out = _out(out, (rows, cols), out_dtype, q.device, "out")
    od = OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32
    with torch.cuda.device(q.device):
        check(load().qcast_cast_back(q.data_ptr(), sf.data_ptr(), rows, cols, f, group, od,
                                     out.data_ptr(), _stream(q.device, stream)), "qcast_cast_back")
    return out


# ---- around the products of a training step: checkpoints and norms ----------

SwigluGrad = namedtuple("SwigluGrad", "dh dh_sf dh_t dh_t_sf v_t v_t_sf dw")
NormOut = namedtuple("NormOut", "h out out_sf x rstd_post rstd_pre y_ckpt y_ckpt_sf h_ckpt "
                                "h_ckpt_sf")
NormGrad = namedtuple("NormGrad", "dh out out_sf dy dw_post dw_pre dgate")
_HERE = nullcontext()


def _torch_calls(c):
    """(allocate on the current device, index of the current device, handle of
    a device's current stream): what torch's generated code calls, from torch's
    C module ``c``, where it has them, else the public functions. A small
    call's time is mostly its 4 to 9 outputs: 0.7 us a tensor against 1.3 for
    torch.empty, and a stream's handle 2 us less than a Stream object."""
    try:
        strided = c._dynamo.guards._empty_strided_cuda
    except AttributeError:
        def strided(shape, strides, dtype):
            return torch.empty_strided(shape, strides, dtype=dtype, device="cuda")
    here = getattr(c, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(c, "_cuda_getCurrentRawStream",
                     lambda device: torch.cuda.current_stream(device).cuda_stream)
    return strided, here, stream


_strided, _current_device, _current_stream = _torch_calls(torch._C)


def _new(shape, dtype):
    """A contiguous tensor on the current device."""
    return _strided(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype)


def _new_out(t, shape, dtype, device, name):
    return _new(shape, dtype) if t is None else _out(t, shape, dtype, device, name)


def _placed(device, stream):
    """The handle of the stream a call runs on and the context in which it
    allocates: outputs and workspaces come from that stream's pool, so memory
    still in use on the current stream is never handed to another one."""
    here = _current_device()
    if device.index == here:
        current = _current_stream(here)
    else:
        current = torch.cuda.current_stream(device).cuda_stream
    handle = current if stream is None else _stream(device, stream)
    if handle != current:
        s = torch.cuda.default_stream(device) if handle == 0 else \
            torch.cuda.ExternalStream(handle, device=device)
        return handle, torch.cuda.stream(s)
    if device.index != here:
        return handle, torch.cuda.device(device)
    return handle, _HERE


def _ptr(t):
    return None if t is None else t.data_ptr()


def _codes(q, name):
    """Stored 8-bit codes ``[rows, cols]`` and their format, from the dtype."""
    f = {torch.float8_e4m3fn: FMT_E4M3, torch.float8_e5m2: FMT_E5M2}.get(
        getattr(q, "dtype", None))
    if f is None or not q.is_cuda:
        raise QcastError(4, f"{name} must be a float8_e4m3fn or float8_e5m2 CUDA (HIP) tensor")
    if q.dim() != 2 or not q.is_contiguous():
        raise QcastError(2, f"{name} must be a contiguous 2-D tensor")
    return f


def _like(t, shape, dtype, device, name):
    """An input that has to have this shape and type; returns its pointer."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.shape == shape and \
            t.device == device and t.is_contiguous():
        return t.data_ptr()
    raise QcastError(2, f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")


def _stored_scales(sf, rows, cols, device, name):
    """(group, pointer) of the scales ``[rows, cols/group]`` of stored codes."""
    if not isinstance(sf, torch.Tensor) or sf.dim() != 2 or sf.shape[0] != rows or \
            (sf.shape[1] == 0) != (cols == 0) or (cols and cols % sf.shape[1]):
        raise QcastError(2, f"{name} must be a [rows, columns/g] tensor of {rows} rows")
    return cols // sf.shape[1] if cols else 128, _like(sf, sf.shape, torch.float32, device, name)


def qcast_swiglu_checkpoint(h, row_weight=None, fmt="e4m3", group=128, clamp_min=0.0, sf_flags=0,
                            swiglu_clamp=0.0, ckpt_fmt="e4m3", out=None, out_sf=None, ckpt=None,
                            ckpt_sf=None, stream=None):
    """SwiGLU of ``h [rows, 2N]`` cast per token, and the 8-bit per-token cast
    of ``h`` itself, in the same groups, for qcast_swiglu_backward_checkpoint
    (which needs N to be a multiple of 128): ``(out [rows, N], out_sf, ckpt
    [rows, 2N], ckpt_sf [rows, 2N/group])``."""
    f, cf = fmt_id(fmt), fmt_id(ckpt_fmt)
    h, rows, cols = _gate_up(h)
    if cf not in (FMT_E4M3, FMT_E5M2):
        raise QcastError(4, "ckpt_fmt must be an 8-bit format (e4m3 or e5m2)")
    dev = h.device
    wptr = _row_weight(row_weight, rows, dev)
    g = group if group > 0 else 1
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, code_shape(f, rows, cols), _code_dtype(f), dev, "out")
        shape, dt = sf_layout_shape(rows, cols, g, sf_flags)
        out_sf = _new_out(out_sf, shape, dt, dev, "out_sf")
        ckpt = _new_out(ckpt, (rows, 2 * cols), _code_dtype(cf), dev, "ckpt")
        ckpt_sf = _new_out(ckpt_sf, (rows, 2 * cols // g), torch.float32, dev, "ckpt_sf")
        check(load().qcast_swiglu_checkpoint(
            h.data_ptr(), rows, cols, wptr, f, group, clamp_min, sf_flags, swiglu_clamp,
            out.data_ptr(), out_sf.data_ptr(), cf, ckpt.data_ptr(), ckpt_sf.data_ptr(), sh),
            "qcast_swiglu_checkpoint")
    return out, out_sf, ckpt, ckpt_sf


def qcast_swiglu_backward_checkpoint(ckpt, ckpt_sf, dv, row_weight=None, fmt="e4m3", group=128,
                                     clamp_min=0.0, sf_flags=0, swiglu_clamp=0.0,
                                     transposed=True, weight_grad=True, stream=None):
    """SwiGLU backward from the 8-bit checkpoint ``ckpt [rows, 2N]`` (its format
    is its dtype) with scales ``ckpt_sf [rows, 2N/g]`` (g = 32, 64 or 128): a
    ``SwigluGrad`` of ``dh [rows, 2N]`` codes of [dgate | dup] and ``dh_sf`` (in
    groups of 128, as all the outputs); with ``transposed``
    ``dh_t [2N, rows_T]``, ``v_t [N, rows_T]`` and their scales, the operands of
    the weight gradients, rows_T = rows up to a multiple of 128 and the codes
    behind the last row zero; with ``weight_grad`` ``dw [rows]``, the gradient
    of ``row_weight`` (of a weight of 1 without one; past 128 columns it takes a
    second launch). What is not asked for is None."""
    f = fmt_id(fmt)
    cf = _codes(ckpt, "ckpt")
    rows, two_n = ckpt.shape
    if two_n % 2:
        raise QcastError(2, f"ckpt must have an even number of columns (gate | up), got {two_n}")
    if f not in (FMT_E4M3, FMT_E5M2):
        raise QcastError(4, "fmt must be an 8-bit format (e4m3 or e5m2)")
    cols = two_n // 2
    dev = ckpt.device
    ckpt_group, sfptr = _stored_scales(ckpt_sf, rows, two_n, dev, "ckpt_sf")
    dvptr = _like(dv, (rows, cols), torch.bfloat16, dev, "dv")
    wptr = _row_weight(row_weight, rows, dev)
    rows_t = (rows + 127) // 128 * 128
    sh, ctx = _placed(dev, stream)
    with ctx:
        dt8 = _code_dtype(f)
        dh = _new((rows, two_n), dt8)
        shape, dt = sf_layout_shape(rows, two_n, 128, sf_flags)
        dh_sf = _new(shape, dt)
        dh_t = dh_t_sf = v_t = v_t_sf = dw = ws = None
        if transposed:
            dh_t = _new((two_n, rows_t), dt8)
            v_t = _new((cols, rows_t), dt8)
            dh_t_sf = _new(sf_layout_shape(two_n, rows_t, 128, sf_flags)[0], dt)
            v_t_sf = _new(sf_layout_shape(cols, rows_t, 128, sf_flags)[0], dt)
        if weight_grad:
            dw = _new((rows,), torch.float32)
            if cols > 128:
                ws = _new((rows * (cols // 128),), torch.float32)
        check(load().qcast_swiglu_backward_checkpoint_ex(
            ckpt.data_ptr(), sfptr, dvptr, rows, cols, wptr, cf, ckpt_group, f, group, clamp_min,
            sf_flags, swiglu_clamp, dh.data_ptr(), dh_sf.data_ptr(), _ptr(dh_t), _ptr(dh_t_sf),
            _ptr(v_t), _ptr(v_t_sf), _ptr(dw), _ptr(ws), sh), "qcast_swiglu_backward_checkpoint")
    return SwigluGrad(dh, dh_sf, dh_t, dh_t_sf, v_t, v_t_sf, dw)


# the checkpoint's group comes from the scales' shape, so one function serves
# both C entry points
qcast_swiglu_backward_checkpoint_ex = qcast_swiglu_backward_checkpoint


def qcast_recast_per_channel_T(q, sf, fmt="e4m3", group=128, clamp_min=0.0, sf_flags=0, out=None,
                               out_sf=None, stream=None):
    """Stored per-token codes ``q [rows, cols]`` (their format is their dtype)
    with scales ``sf [rows, cols/g]`` (g = 32, 64 or 128) cast again along the
    tokens and transposed: ``out [cols, rows_T]``, ``out_sf`` in the layouts of
    ``sf_layout_shape(cols, rows_T, 128, sf_flags)``, rows_T = rows up to a
    multiple of 128 and the codes behind the last row zero."""
    f = fmt_id(fmt)
    cf = _codes(q, "q")
    rows, cols = q.shape
    if f not in (FMT_E4M3, FMT_E5M2):
        raise QcastError(4, "fmt must be an 8-bit format (e4m3 or e5m2)")
    dev = q.device
    in_group, sfptr = _stored_scales(sf, rows, cols, dev, "sf")
    rows_t = (rows + 127) // 128 * 128
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, (cols, rows_t), _code_dtype(f), dev, "out")
        shape, dt = sf_layout_shape(cols, rows_t, 128, sf_flags)
        out_sf = _new_out(out_sf, shape, dt, dev, "out_sf")
        check(load().qcast_recast_per_channel_T(
            q.data_ptr(), sfptr, rows, cols, cf, in_group, f, group, clamp_min, sf_flags,
            out.data_ptr(), out_sf.data_ptr(), sh), "qcast_recast_per_channel_T")
    return out, out_sf


def _no_empty_rows(rows, cols):
    if rows and not cols:
        raise QcastError(2, "there is no norm of rows without columns")


def _gate_arg(gate, rows, cols, device):
    """(kind, pointer) of a gate: [cols] bf16, [rows] fp32 or [rows, cols] bf16."""
    if gate is None:
        return GATE_NONE, None
    if isinstance(gate, torch.Tensor) and gate.dtype == torch.float32:
        return GATE_TOKEN, _like(gate, (rows,), torch.float32, device, "gate")
    if isinstance(gate, torch.Tensor) and gate.dim() == 1:
        return GATE_CHANNEL, _like(gate, (cols,), torch.bfloat16, device, "gate")
    return GATE_FULL, _like(gate, (rows, cols), torch.bfloat16, device, "gate")


def qcast_norm_per_token(h, w_pre, y=None, w_post=None, gate=None, residual_scale=1.0,
                         weight_offset=0.0, eps=1e-6, fmt="e4m3", group=128, clamp_min=0.0,
                         sf_flags=0, ckpt_fmt=None, want_x=False, want_codes=True, stream=None):
    """Norm after a block (``y``, weight ``w_post``), its ``gate`` and the scaled
    residual ``h``, the norm before the next block (``w_pre``) and the per-token
    cast of that block's input (include/qcast.h). ``gate``: bf16 ``[cols]``,
    fp32 ``[rows]`` or bf16 ``[rows, cols]``.

    Returns a ``NormOut``: ``h`` the new residual stream (the given one without
    ``y``), ``out``/``out_sf`` the cast (with ``want_codes``), ``x`` the bf16
    input (with ``want_x``), ``rstd_post``/``rstd_pre``, and with ``ckpt_fmt``
    ('e4m3' or 'e5m2') the 8-bit checkpoints of ``y`` and of the new residual
    stream for qcast_norm_backward_per_token."""
    f = fmt_id(fmt)
    h = _bf16_input(h, "h")
    rows, cols = h.shape
    _no_empty_rows(rows, cols)
    dev = h.device
    bf16, f32 = torch.bfloat16, torch.float32
    wqptr = _like(w_pre, (cols,), bf16, dev, "w_pre")
    yptr = None if y is None else _like(y, (rows, cols), bf16, dev, "y")
    wpptr = None if w_post is None else _like(w_post, (cols,), bf16, dev, "w_post")
    kind, gptr = _gate_arg(gate, rows, cols, dev)
    if y is None and (w_post is not None or gate is not None):
        raise QcastError(1, "w_post and gate need y")
    cf = 0 if ckpt_fmt is None else fmt_id(ckpt_fmt)
    if cf not in (0, FMT_E4M3, FMT_E5M2):
        raise QcastError(4, "ckpt_fmt must be an 8-bit format (e4m3 or e5m2)")
    sh, ctx = _placed(dev, stream)
    with ctx:
        h_out = h if y is None else _new((rows, cols), bf16)
        out = out_sf = x = r1 = yc = yc_sf = hc = hc_sf = None
        if want_codes:
            out = _new(code_shape(f, rows, cols), _code_dtype(f))
            shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
            out_sf = _new(shape, dt)
        if want_x:
            x = _new((rows, cols), bf16)
        r2 = _new((rows,), f32)
        if w_post is not None:
            r1 = _new((rows,), f32)
        if cf:
            hc = _new((rows, cols), _code_dtype(cf))
            hc_sf = _new((rows, cols // 128), f32)
            if y is not None:
                yc, yc_sf = _new((rows, cols), _code_dtype(cf)), _new((rows, cols // 128), f32)
        check(load().qcast_norm_per_token(
            yptr, h.data_ptr(), rows, cols, wpptr, wqptr, gptr, kind, residual_scale,
            weight_offset, eps, f, group, clamp_min, sf_flags,
            None if y is None else h_out.data_ptr(), _ptr(out), _ptr(out_sf), _ptr(x), _ptr(r1),
            r2.data_ptr(), cf, _ptr(yc), _ptr(yc_sf), _ptr(hc), _ptr(hc_sf), sh),
            "qcast_norm_per_token")
    return NormOut(h_out, out, out_sf, x, r1, r2, yc, yc_sf, hc, hc_sf)


def norm_ws_rows(rows, cols):
    """Rows of partial sums of the norm backward's workspace
    (``qcast_norm_ws_rows`` of include/qcast.h)."""
    waves = (cols + 511) // 512
    most = 256 * (16 // waves) if 0 < waves < 16 else 256
    return min(rows, max(256, min(most, rows // 8)))


def qcast_norm_backward_per_token(dx, saved_h, rstd_pre, w_pre, dh=None, saved_h_sf=None,
                                  saved_y=None, saved_y_sf=None, rstd_post=None, w_post=None,
                                  gate=None, residual_scale=1.0, weight_offset=0.0, fmt="e4m3",
                                  group=128, clamp_min=0.0, sf_flags=0, want_dy=False,
                                  want_codes=True, stream=None):
    """Gradient of qcast_norm_per_token (include/qcast.h) from ``dx``, the
    gradient of its cast input, and ``dh``, the gradient of the residual stream
    (None: zero). ``saved_h``/``saved_y``: the bf16 residual stream and block
    output, or their 8-bit checkpoints with ``saved_h_sf``/``saved_y_sf``.

    Returns a ``NormGrad``: ``dh`` the gradient of the residual input,
    ``out``/``out_sf`` the per-token cast of the block output's gradient (with
    ``want_codes``), ``dy`` the same in bf16 (with ``want_dy``), ``dw_post`` and
    ``dw_pre`` fp32, and ``dgate`` in the gate's shape (fp32; bf16 for a
    ``[rows, cols]`` gate)."""
    f = fmt_id(fmt)
    dx = _bf16_input(dx, "dx")
    rows, cols = dx.shape
    _no_empty_rows(rows, cols)
    dev = dx.device
    bf16, f32 = torch.bfloat16, torch.float32
    dhptr = None if dh is None else _like(dh, (rows, cols), bf16, dev, "dh")
    sf = 0
    if saved_h_sf is None:
        shptr, shsf = _like(saved_h, (rows, cols), bf16, dev, "saved_h"), None
    else:
        sf = _codes(saved_h, "saved_h")
        shptr = _like(saved_h, (rows, cols), saved_h.dtype, dev, "saved_h")
        shsf = _like(saved_h_sf, (rows, cols // 128), f32, dev, "saved_h_sf")
    syptr = sysf = None
    if saved_y is not None:
        syptr = _like(saved_y, (rows, cols), saved_h.dtype, dev, "saved_y")
        if sf:
            sysf = _like(saved_y_sf, (rows, cols // 128), f32, dev, "saved_y_sf")
    elif w_post is not None or gate is not None:
        raise QcastError(1, "w_post and gate need saved_y")
    if saved_y_sf is not None and (not sf or saved_y is None):
        raise QcastError(1, "saved_y_sf needs saved_y and saved_h in 8 bits")
    r2ptr = _like(rstd_pre, (rows,), f32, dev, "rstd_pre")
    wqptr = _like(w_pre, (cols,), bf16, dev, "w_pre")
    if (w_post is None) != (rstd_post is None):
        raise QcastError(1, "w_post and rstd_post come together")
    wpptr = None if w_post is None else _like(w_post, (cols,), bf16, dev, "w_post")
    r1ptr = None if rstd_post is None else _like(rstd_post, (rows,), f32, dev, "rstd_post")
    kind, gptr = _gate_arg(gate, rows, cols, dev)
    stream_handle, ctx = _placed(dev, stream)
    with ctx:
        dh_out = _new((rows, cols), bf16)
        out = out_sf = dy = dw_post = dgate = ws = None
        if saved_y is not None:
            if want_codes:
                out = _new(code_shape(f, rows, cols), _code_dtype(f))
                shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
                out_sf = _new(shape, dt)
            if want_dy:
                dy = _new((rows, cols), bf16)
        dw_pre = _new((cols,), f32)
        if w_post is not None:
            dw_post = _new((cols,), f32)
        if kind:
            dgate = _new(tuple(gate.shape), bf16 if kind == GATE_FULL else f32)
        if rows:
            ws = _new((norm_ws_rows(rows, cols) * 2 * cols,), f32)
        check(load().qcast_norm_backward_per_token(
            dx.data_ptr(), dhptr, rows, cols, sf, shptr, shsf, syptr, sysf, r1ptr, r2ptr, wpptr,
            wqptr, gptr, kind, residual_scale, weight_offset, f, group, clamp_min, sf_flags,
            dh_out.data_ptr(), _ptr(out), _ptr(out_sf), _ptr(dy), _ptr(dw_post),
            dw_pre.data_ptr(), _ptr(dgate), _ptr(ws), stream_handle),
            "qcast_norm_backward_per_token")
    return NormGrad(dh_out, out, out_sf, dy, dw_post, dw_pre, dgate)


# ---- a mixture-of-experts layer around its products -------------------------

MAX_EXPERTS = 1024              # QCAST_MAX_EXPERTS
MAX_ALIGN = 1024                # QCAST_MAX_ALIGN
ExpertPlan = namedtuple("ExpertPlan", "dest source offsets counts row_weight align")
CombineGrad = namedtuple("CombineGrad", "out out_sf dy dw")


def expert_rows(tokens, top_k, experts, align):
    """Rows of the sorted buffers of a layer (``qcast_expert_rows`` of
    include/qcast.h)."""
    slots = tokens * top_k
    return (slots + min(experts, slots) * (align - 1)) // align * align


def _sort_parts(slots):
    """Workgroups of qcast_expert_sort, each of which has a row of its
    workspace (``qcast_expert_sort_ws_bytes`` of include/qcast.h)."""
    if slots <= 4096:
        return 0
    part = max(2048, ((slots + 255) // 256 + 1023) // 1024 * 1024)
    return (slots + part - 1) // part


def _ids(ids, name, dim):
    """An int32 or int64 index tensor: (pointer, bytes of an index)."""
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda:
        raise QcastError(1, f"{name} must be a CUDA (HIP) tensor")
    if ids.dtype not in (torch.int64, torch.int32) or ids.dim() != dim or not ids.is_contiguous():
        raise QcastError(2, f"{name} must be a contiguous {dim}-D int32 or int64 tensor")
    return ids.data_ptr(), 8 if ids.dtype == torch.int64 else 4


def qcast_expert_sort(ids, experts, align=1, first=0, weight=None, stream=None):
    """The slots of ``ids [tokens, top_k]`` (int32 or int64, as a router's
    top-k gives them) sorted by expert (include/qcast.h): an ``ExpertPlan`` of
    ``dest [tokens, top_k]``, ``source [rows]``, ``offsets [experts + 1]``,
    ``counts [experts]`` (int32) and, with ``weight [tokens, top_k]`` (fp32),
    ``row_weight [rows]``; rows = ``expert_rows(tokens, top_k, experts,
    align)``. The experts here are ``first`` to ``first + experts - 1``; each
    one's rows start at a multiple of ``align``."""
    ptr, width = _ids(ids, "ids", 2)
    tokens, top_k = ids.shape
    experts, align = int(experts), int(align)
    if not 1 <= experts <= MAX_EXPERTS:
        raise QcastError(2, f"experts must be 1 to {MAX_EXPERTS}, got {experts}")
    if not 1 <= align <= MAX_ALIGN:
        raise QcastError(8, f"align must be a power of two up to {MAX_ALIGN}, got {align}")
    dev = ids.device
    wptr = None if weight is None else _like(weight, (tokens, top_k), torch.float32, dev, "weight")
    rows = expert_rows(tokens, top_k, experts, align)
    parts = _sort_parts(tokens * top_k)
    i32 = torch.int32
    sh, ctx = _placed(dev, stream)
    with ctx:
        dest = _new((tokens, top_k), i32)
        source = _new((rows,), i32)
        offsets = _new((experts + 1,), i32)
        counts = _new((experts,), i32)
        row_weight = None if wptr is None else _new((rows,), torch.float32)
        ws = _new((parts * experts,), i32) if parts else None
        check(load().qcast_expert_sort(ptr, width, tokens, top_k, experts, first, align, wptr,
                                       dest.data_ptr(), source.data_ptr(), offsets.data_ptr(),
                                       counts.data_ptr(), _ptr(row_weight), _ptr(ws), sh),
              "qcast_expert_sort")
    return ExpertPlan(dest, source, offsets, counts, row_weight, align)


def _plan(plan, tokens, device):
    """(rows, top_k, experts, dest, offsets, counts) of a plan for `tokens`
    tokens; the last three are pointers."""
    i32 = torch.int32
    dest, source, offsets, counts = plan.dest, plan.source, plan.offsets, plan.counts
    if dest.dim() != 2 or source.dim() != 1 or counts.dim() != 1:
        raise QcastError(2, "plan must hold dest [tokens, top_k], source [rows] and counts [experts]")
    top_k, experts = dest.shape[1], counts.shape[0]
    return (source.shape[0], top_k, experts, _like(dest, (tokens, top_k), i32, device, "plan.dest"),
            _like(offsets, (experts + 1,), i32, device, "plan.offsets"),
            _like(counts, (experts,), i32, device, "plan.counts"))


def qcast_dispatch_codes(q, plan, sf=None, sf_flags=0, out_sf_flags=None, out=None, out_sf=None,
                         stream=None):
    """Rows of ``q [tokens, n]`` (codes of any format, or bf16; a row's bytes a
    multiple of 16) and their scales ``sf`` brought to the rows of ``plan``:
    ``(out [rows, n], out_sf)``. ``sf`` is float32 or int32 (packed UE8M0
    words): ``[tokens, words]``, or with SF_COL_MAJOR in ``sf_flags`` ``[words,
    tokens up to a multiple of 4]``; ``out_sf`` the same by ``out_sf_flags``
    (None: as ``sf_flags``). A run's padding rows are zeros; rows behind the
    last run are left as they were (new outputs: undefined)."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise QcastError(1, "q must be a CUDA (HIP) tensor")
    if q.dim() != 2 or not q.is_contiguous():
        raise QcastError(2, "q must be a contiguous 2-D tensor")
    tokens, n = q.shape
    dev = q.device
    rows, top_k, experts, dptr, optr, cptr = _plan(plan, tokens, dev)
    out_sf_flags = sf_flags if out_sf_flags is None else out_sf_flags
    words, sfptr, sf_shape = 0, None, None
    if sf is not None:
        if not isinstance(sf, torch.Tensor) or sf.dim() != 2 or \
                sf.dtype not in (torch.float32, torch.int32):
            raise QcastError(2, "sf must be a 2-D float32 or int32 tensor")
        words = sf.shape[0] if sf_flags & SF_COL_MAJOR else sf.shape[1]
        sfptr = _like(sf, (words, (tokens + 3) // 4 * 4) if sf_flags & SF_COL_MAJOR
                      else (tokens, words), sf.dtype, dev, "sf")
        sf_shape = (words, (rows + 3) // 4 * 4) if out_sf_flags & SF_COL_MAJOR else (rows, words)
    elif out_sf is not None:
        raise QcastError(1, "out_sf needs sf")
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, (rows, n), q.dtype, dev, "out")
        if sf is not None:
            out_sf = _new_out(out_sf, sf_shape, sf.dtype, dev, "out_sf")
        check(load().qcast_dispatch_codes(
            q.data_ptr(), tokens, n * q.element_size(), sfptr, words, sf_flags, top_k, dptr, optr,
            cptr, experts, plan.align, rows, out.data_ptr(), _ptr(out_sf), out_sf_flags, sh),
            "qcast_dispatch_codes")
    return out, out_sf


def qcast_dispatch_per_token(x, plan, weight=None, fmt="e4m3", group=128, clamp_min=0.0,
                             sf_flags=0, out=None, out_sf=None, stream=None):
    """The per-token cast of bf16 ``x [tokens, cols]`` (times ``weight [tokens,
    top_k]``, fp32) written to the rows of ``plan``: ``out [rows, cols]``,
    ``out_sf`` of ``sf_layout_shape(rows, cols, group, sf_flags)``. A run's
    padding rows are the cast of zeros; rows behind the last run are left as
    they were (new outputs: undefined)."""
    f = fmt_id(fmt)
    x = _bf16_input(x, "x")
    tokens, cols = x.shape
    dev = x.device
    rows, top_k, experts, dptr, optr, cptr = _plan(plan, tokens, dev)
    wptr = None if weight is None else _like(weight, (tokens, top_k), torch.float32, dev, "weight")
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, code_shape(f, rows, cols), _code_dtype(f), dev, "out")
        shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
        out_sf = _new_out(out_sf, shape, dt, dev, "out_sf")
        check(load().qcast_dispatch_per_token(
            x.data_ptr(), tokens, cols, top_k, dptr, wptr, optr, cptr, experts, plan.align, rows, f,
            group, clamp_min, sf_flags, out.data_ptr(), out_sf.data_ptr(), sh),
            "qcast_dispatch_per_token")
    return out, out_sf


def qcast_combine(y, dest=None, weight=None, base=None, top_k=None, out=None, stream=None):
    """``base + sum_k weight[:, k] * y[dest[:, k]]`` as bf16 ``[tokens, cols]``
    from the experts' outputs ``y [rows, cols]`` (bf16). ``dest [tokens,
    top_k]``: int32 (an ``ExpertPlan``'s), -1 where there is no row; None:
    ``y`` holds a token's ``top_k`` rows next to one another. ``weight
    [tokens, top_k]`` fp32 (None: ones); ``base [tokens, cols]`` bf16 (None:
    zeros). Without base, of the rows' gradient and with the weights that a
    dispatch had, it is that dispatch's gradient."""
    y = _bf16_input(y, "y")
    rows, cols = y.shape
    dev = y.device
    if dest is not None:
        if not isinstance(dest, torch.Tensor) or dest.dim() != 2:
            raise QcastError(2, "dest must be an int32 [tokens, top_k] tensor")
        if top_k is not None and dest.shape[1] != top_k:
            raise QcastError(2, f"dest has {dest.shape[1]} slots a token, not {top_k}")
        tokens, top_k = dest.shape
        dptr = _like(dest, (tokens, top_k), torch.int32, dev, "dest")
    else:
        if top_k is None or top_k < 1 or rows % top_k:
            raise QcastError(2, "without dest, top_k must be given and divide y's rows")
        tokens, dptr = rows // top_k, None
    wptr = None if weight is None else _like(weight, (tokens, top_k), torch.float32, dev, "weight")
    bptr = None if base is None else _like(base, (tokens, cols), torch.bfloat16, dev, "base")
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, (tokens, cols), torch.bfloat16, dev, "out")
        check(load().qcast_combine(y.data_ptr(), rows, tokens, top_k, cols, dptr, wptr, bptr,
                                   out.data_ptr(), sh), "qcast_combine")
    return out


def qcast_combine_backward_per_token(dout, plan, y=None, weight=None, fmt="e4m3", group=128,
                                     clamp_min=0.0, sf_flags=0, want_codes=True, want_dy=False,
                                     out=None, out_sf=None, dy=None, stream=None):
    """Gradient of qcast_combine over the rows of ``plan`` from ``dout [tokens,
    cols]`` (bf16), fused with the per-token cast of the experts' output
    gradient: a ``CombineGrad`` of ``out [rows, cols]``/``out_sf`` (with
    ``want_codes``), the same in bf16 ``dy`` (with ``want_dy``) and, where
    ``y`` (the forward's) is given, ``dw [tokens, top_k]`` fp32, the gradient
    of ``weight`` (of a dispatch's weights: with its ``x`` as ``dout`` and its
    rows' gradient as ``y``). Padding rows and rows behind the last run as
    qcast_dispatch_per_token leaves them."""
    f = fmt_id(fmt)
    dout = _bf16_input(dout, "dout")
    tokens, cols = dout.shape
    dev = dout.device
    rows, top_k, experts, dptr, optr, cptr = _plan(plan, tokens, dev)
    yptr = None if y is None else _like(y, (rows, cols), torch.bfloat16, dev, "y")
    wptr = None if weight is None else _like(weight, (tokens, top_k), torch.float32, dev, "weight")
    if (out is not None or out_sf is not None) and not want_codes:
        raise QcastError(1, "out and out_sf need want_codes")
    if dy is not None and not want_dy:
        raise QcastError(1, "dy needs want_dy")
    sh, ctx = _placed(dev, stream)
    with ctx:
        if want_codes:
            out = _new_out(out, code_shape(f, rows, cols), _code_dtype(f), dev, "out")
            shape, dt = sf_layout_shape(rows, cols, group if group > 0 else 1, sf_flags)
            out_sf = _new_out(out_sf, shape, dt, dev, "out_sf")
        if want_dy:
            dy = _new_out(dy, (rows, cols), torch.bfloat16, dev, "dy")
        dw = None if y is None else _new((tokens, top_k), torch.float32)
        check(load().qcast_combine_backward_per_token(
            dout.data_ptr(), yptr, tokens, cols, top_k, dptr, wptr, optr, cptr, experts,
            plan.align, rows, f, group, clamp_min, sf_flags, _ptr(out), _ptr(out_sf), _ptr(dy),
            _ptr(dw), sh), "qcast_combine_backward_per_token")
    return CombineGrad(out, out_sf, dy, dw)


def qcast_matvec_e2m1(x, w, w_sf, ids=None, x_sf=None, out_dtype=torch.bfloat16, out=None,
                      stream=None):
    """Products of a few rows with E2M1 weights: ``out [rows, n]`` (bf16 or
    fp32), row r being ``W[ids[r]] @ x[r // (rows / x_rows)]``. ``w [experts,
    n, k/2]`` (uint8, qcast_e2m1's codes of each weight) with scales ``w_sf
    [experts, n, k/g]`` float32, or int32 packed UE8M0 words ``[experts, n,
    k/g/4]``, g = 32, 64 or 128. ``ids``: int32 or int64, any shape, one row
    each (zeros where outside the experts); None: one weight ``w [n, k/2]``
    for every row of x. ``x [x_rows, k]``: bf16, or float8 codes with ``x_sf
    [x_rows, k/g]``."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise QcastError(1, "x must be a CUDA (HIP) tensor")
    if x.dim() != 2 or not x.is_contiguous():
        raise QcastError(2, "x must be a contiguous 2-D tensor")
    x_rows, k = x.shape
    dev = x.device
    xf, xg, xsptr = 0, 128, None
    if x_sf is not None:
        xf = _codes(x, "x")
        xg, xsptr = _stored_scales(x_sf, x_rows, k, dev, "x_sf")
    elif x.dtype != torch.bfloat16:
        raise QcastError(2, f"x must be bfloat16 (or float8 codes with x_sf), got {x.dtype}")
    dims = 2 if ids is None else 3
    if not isinstance(w, torch.Tensor) or w.dim() != dims or not isinstance(w_sf, torch.Tensor) or \
            w_sf.dim() != dims:
        raise QcastError(2, "w and w_sf must be [n, k/2] and [n, k/g] tensors, or with ids "
                            "[experts, n, k/2] and [experts, n, k/g]")
    experts, n = (1, w.shape[0]) if ids is None else w.shape[:2]
    lead = tuple(w.shape[:-1])
    wptr = _like(w, lead + (k // 2,), torch.uint8, dev, "w")
    packed = w_sf.dtype == torch.int32
    groups = w_sf.shape[-1] * (4 if packed else 1)
    if (groups == 0) != (k == 0) or (k and k % groups):
        raise QcastError(2, f"w_sf holds {groups} groups of a row of {k}")
    wsptr = _like(w_sf, lead + (w_sf.shape[-1],), torch.int32 if packed else torch.float32, dev,
                  "w_sf")
    rows, iptr, width = x_rows, None, 8
    if ids is not None:
        if not isinstance(ids, torch.Tensor):
            raise QcastError(1, "ids must be a CUDA (HIP) tensor")
        iptr, width = _ids(ids, "ids", ids.dim())
        rows = ids.numel()
        if ids.device != dev:
            raise QcastError(2, "ids must be on x's device")
    if out_dtype not in (torch.bfloat16, torch.float32):
        raise QcastError(4, "out_dtype must be torch.bfloat16 or torch.float32")
    sh, ctx = _placed(dev, stream)
    with ctx:
        out = _new_out(out, (rows, n), out_dtype, dev, "out")
        check(load().qcast_matvec_e2m1(
            x.data_ptr(), xf, xsptr, xg, x_rows, wptr, wsptr, k // groups if k else 128,
            SF_PACKED_UE8M0 if packed else 0, experts, iptr, width, rows, n, k,
            OUT_BF16 if out_dtype == torch.bfloat16 else OUT_F32, out.data_ptr(), sh),
            "qcast_matvec_e2m1")
    return out


def qcast_abi_version():
    return load().qcast_abi_version()


def qcast_set_num_cus(n):
    load().qcast_set_num_cus(int(n))


def qcast_bench_copy(src, dst, stream=None):
    """Measurement helper (include/qcast_bench.h): copy src's bytes to dst."""
    if not (src.is_cuda and dst.is_cuda and src.is_contiguous() and dst.is_contiguous()):
        raise QcastError(2, "src and dst must be contiguous CUDA tensors")
    n = src.numel() * src.element_size()
    if dst.numel() * dst.element_size() != n or src.device != dst.device:
        raise QcastError(2, "src and dst must have the same size on one device")
    with torch.cuda.device(src.device):
        check(load().qcast_bench_copy(src.data_ptr(), dst.data_ptr(), n, _stream(src.device, stream)),
              "qcast_bench_copy")


def qcast_bench_per_channel_T_traffic(x, out=None, stream=None):
    """Measurement helper (include/qcast_bench.h): the loads and qT stores of
    qcast_per_channel_T on bf16 ``x [tokens, channels]`` without its
    arithmetic; ``out [channels, tokens]`` bytes receives meaningless data."""
    x = _bf16_input(x, "x")
    rows, cols = x.shape
    out = _out(out, (cols, rows), torch.uint8, x.device, "out")
    with torch.cuda.device(x.device):
        check(load().qcast_bench_per_channel_T_traffic(x.data_ptr(), rows, cols, out.data_ptr(),
                                                       _stream(x.device, stream)),
              "qcast_bench_per_channel_T_traffic")
    return out


def qcast_bench_check_scale(fmt, first, last, device="cuda:0", stream=None):
    """Self-check helper (include/qcast_bench.h): mismatches of the kernels'
    scale routine against IEEE division over fp32 patterns [first, last];
    returns (sf mismatches, sf_inv mismatches)."""
    dev = torch.device(device)
    counts = torch.empty(2 * 2048, dtype=torch.int32, device=dev)
    with torch.cuda.device(dev):
        check(load().qcast_bench_check_scale(fmt_id(fmt), first, last, counts.data_ptr(),
                                             _stream(dev, stream)), "qcast_bench_check_scale")
        c = counts.view(2048, 2).sum(dim=0, dtype=torch.int64).cpu()
    return int(c[0]), int(c[1])


def qcast_bench_time_next(start_event, stop_event):
    """Measurement helper (include/qcast_bench.h): the next kernel this thread
    launches through the library records these HIP events (raw hipEvent_t
    handles) at its own start and end."""
    check(load().qcast_bench_time_next(start_event, stop_event), "qcast_bench_time_next")


def per_token_cast(x, fmt="e4m3", num_per_channels=128):
    """``(out, out_sf)`` as in the page's quick-start call."""
    if fmt_id(fmt) == FMT_E2M1:
        return qcast_e2m1(x, num_per_channels)
    return qcast_per_token(x, fmt, num_per_channels)
