"""The operators around a block's products in 64 bits, for the tests, and the
bound their casts are held to.

A cast of fp32 values that are off by at most ``slack`` (absolute, per element)
from the 64-bit values x may differ from x by half a step of the format at x
(relative 2^-(m+1) for m mantissa bits; half the smallest step, times the
scale, below the normal range), plus that slack, plus what the fp32 scale and
its inverse add (three roundings of 2^-24, counted as 2^-21 of the group's
abs-max). The scale itself may be off by the relative slack of the abs-max and
two roundings."""
import numpy as np
import torch

import oracle
from precision_quantization_amd import workloads
from swiglu_bar import element_codes, scale_values

MANTISSA = {"e4m3": 3, "e5m2": 2, "e2m1": 1, "e5m6": 6}
SMALLEST = {"e4m3": 2.0 ** -9, "e5m2": 2.0 ** -16, "e2m1": 0.5, "e5m6": 2.0 ** -20}


def decoded(q, fmt, cols):
    c = element_codes(q, fmt, cols)
    return oracle.decode(fmt, c.astype(np.uint16 if fmt == "e5m6" else np.uint8)).astype(
        np.float64).reshape(c.shape)


def raw(t):
    """A code or scale tensor as numpy bytes or words."""
    if t.dtype in (torch.float8_e4m3fn, torch.float8_e5m2):
        t = t.view(torch.uint8)
    return t.cpu().numpy()


def check_cast(q, sf, x, fmt, group, slack, sf_flags=0, clamp_min=0.0, what=""):
    """q, sf: stored codes and scales of [rows, cols] values in the layout
    sf_flags; x: the values in float64; slack: absolute error of the fp32
    values, [rows, cols] or a number times each group's abs-max."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    if x.size == 0:
        return
    s = scale_values(sf, rows, cols // group, sf_flags)[..., None]
    g = x.reshape(rows, cols // group, group)
    amax = np.abs(g).max(axis=2, keepdims=True)
    floor = clamp_min if clamp_min > 0 else oracle.default_floor(fmt)
    top = np.maximum(amax, floor)
    slack = slack.reshape(g.shape) if isinstance(slack, np.ndarray) else slack * amax
    ideal = top / oracle.format_max(fmt)
    off = slack.max(axis=2, keepdims=True) / oracle.format_max(fmt) + ideal * 2.0 ** -22
    if sf_flags & 5:                      # a power of two at or above the plain scale
        assert (np.exp2(np.round(np.log2(s))) == s).all(), what
        assert (s >= (ideal - off) * (1 - 2.0 ** -23)).all() and (s <= 2 * (ideal + off)).all(), what
    else:
        assert (np.abs(s - ideal) <= off).all(), f"{what}: scale off by {np.max(np.abs(s - ideal) / off):.3g} of its bound"
    deq = decoded(q, fmt, cols).reshape(g.shape) * s
    half = np.maximum(np.abs(g) * 2.0 ** -(MANTISSA[fmt] + 1), s * SMALLEST[fmt] / 2)
    bound = (half + slack) * (1 + 2.0 ** -10) + top * 2.0 ** -21
    worst = np.max(np.abs(deq - g) / bound)
    assert worst <= 1.0, f"{what}: values off by {worst:.3g} of their bound"


def f64(t):
    return t.detach().cpu().double()


# ---- formulas ---------------------------------------------------------------

def swiglu_grad(h, dv, w=None, clamp=0.0):
    """(d [rows, 2N], v [rows, N], dw [rows]) from float64 h = (gate | up)."""
    n = h.shape[1] // 2
    g, u = h[:, :n], h[:, n:]
    c = clamp if clamp > 0 else float("inf")
    pg, pu = g <= c, u.abs() <= c
    g, u = g.clamp(max=c), u.clamp(-c, c)
    s = torch.sigmoid(g)
    ww = torch.ones(h.shape[0], 1, dtype=h.dtype) if w is None else w[:, None]
    silu = g * s
    dg = dv * ww * u * (s + silu * (1 - s)) * pg
    du = dv * ww * silu * pu
    return torch.cat([dg, du], 1), silu * u * ww, (dv * silu * u).sum(1)


def norm_forward(h, w_pre, y=None, w_post=None, gate=None, alpha=1.0, offset=0.0, eps=1e-6):
    """float64 dict of h' ("h"), "x", "r1", "r2", and "mag": the sum of the
    magnitudes h' is formed from."""
    r1 = None
    mag = h.abs()
    if y is not None:
        t = y
        if w_post is not None:
            r1 = 1 / (y.square().mean(1) + eps).sqrt()
            t = y * r1[:, None] * (w_post + offset)
        if gate is not None:
            t = t * (gate[:, None] if gate.dim() == 1 and gate.shape[0] == h.shape[0]
                     and gate.shape[0] != h.shape[1] else gate)
        mag = (alpha * h).abs() + t.abs()
        h = alpha * h + t
    r2 = 1 / (h.square().mean(1) + eps).sqrt()
    return dict(h=h, x=h * r2[:, None] * (w_pre + offset), r1=r1, r2=r2, mag=mag)


def norm_backward(dx, dh_in, h, r2, w_pre, y=None, r1=None, w_post=None, gate=None, alpha=1.0,
                  offset=0.0, kind=None):
    """float64 dict of "dh", "dy", "dw_pre", "dw_post", "dgate"; kind: None,
    "channel", "token" or "full"."""
    n = h.shape[1]
    xh = h * r2[:, None]
    g = dx * (w_pre + offset)
    d = r2[:, None] * (g - xh * (g * xh).sum(1, keepdim=True) / n)
    if dh_in is not None:
        d = d + dh_in
    out = dict(dh=alpha * d, dw_pre=(dx * xh).sum(0), d=d, dy=None, dw_post=None, dgate=None)
    if y is None:
        return out
    a = y if r1 is None else y * r1[:, None]
    wp = torch.ones((), dtype=h.dtype) if w_post is None else w_post + offset
    gg = 1.0 if gate is None else gate[:, None] if kind == "token" else gate
    dz = d * gg
    full = d * a * wp
    out["dgate"] = {None: None, "channel": full.sum(0), "token": full.sum(1), "full": full}[kind]
    if w_post is None:
        out["dy"] = dz
    else:
        out["dw_post"] = (dz * a).sum(0)
        da = dz * wp
        out["dy"] = r1[:, None] * (da - a * (da * a).sum(1, keepdim=True) / n)
    return out


# ---- inputs -----------------------------------------------------------------

def bf16(gen, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=gen) * std + mean).to(torch.bfloat16)


def gate_of(kind, gen, rows, cols):
    if kind == "channel":
        return bf16(gen, cols, std=0.5, mean=0.5)
    if kind == "token":
        return torch.rand(rows, generator=gen)
    if kind == "full":
        return bf16(gen, rows, cols, std=0.5, mean=0.5)
    return None


def stored(t, fmt, group=128):
    """Per-token codes of a bf16 CPU tensor by the oracle: float8 codes, fp32
    scales, and the float64 values they stand for."""
    q, sf = oracle.per_token(workloads.bf16_bits(t), fmt, group)
    dt = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}[fmt]
    codes = torch.from_numpy(q.copy()).view(dt)
    scales = torch.from_numpy(sf.copy())
    # the fp32 product code * sf, as every reader of the codes forms it
    v = codes.float() * scales.repeat_interleave(group, 1)
    return codes, scales, v.double()


# ---- error bounds of the fp32 evaluation ------------------------------------
# U is one rounding. The counts below are the roundings on the longest path to
# a value: a sum over a row is at most 32 terms in a lane, 6 steps over the
# wave and 15 over the workgroup.

U = 2.0 ** -24
ROW_SUM = 32 + 6 + 15


def swiglu_grad_slack(h, dv, w=None, clamp=0.0):
    """(slack of d, of v, of dw) of the fp32 evaluation: the exponential of a
    rounded argument (|g| log2 e roundings of ln 2 each, 2 for the function),
    the reciprocal and at most 10 products and sums; dsilu is a sum of two
    terms of either sign."""
    n = h.shape[1] // 2
    c = clamp if clamp > 0 else float("inf")
    g, u = h[:, :n].clamp(max=c), h[:, n:].clamp(-c, c)
    s = torch.sigmoid(g)
    ww = torch.ones(h.shape[0], 1, dtype=h.dtype) if w is None else w[:, None]
    k = U * (2 * g.abs() + 16)
    silu = (g * s).abs()
    x = k * (dv * ww).abs()
    kv = k * silu * u.abs()
    sum_steps = U * (8 + 4 + n // 128)
    return (torch.cat([x * u.abs() * (s + silu * (1 - s)), x * silu], 1), kv * ww.abs(),
            (dv.abs() * (kv + sum_steps * silu * u.abs())).sum(1))


def norm_backward_slack(dx, dh_in, h, r2, w_pre, y=None, r1=None, w_post=None, gate=None,
                        alpha=1.0, offset=0.0, kind=None):
    rows, n = h.shape
    xh = (h * r2[:, None]).abs()
    g = (dx * (w_pre + offset)).abs()
    di = torch.zeros_like(h) if dh_in is None else dh_in.abs()
    mean1 = (g * xh).sum(1, keepdim=True) / n
    size_d = di + r2[:, None] * (g + xh * mean1)
    d = U * (10 * size_d + (ROW_SUM + 4) * r2[:, None] * xh * mean1)
    # a column sum: a workgroup's rows one after another (at least 256 workgroups
    # share them, or each row has its own), then a wave's 16th of at most 4096
    # workgroups, the 16 waves, and the products
    steps = U * (rows // 256 + 256 + 16 + 8)
    out = dict(dh=abs(alpha) * d, dw_pre=(steps * dx.abs() * xh).sum(0))
    if y is None:
        return out
    a = y.abs() if r1 is None else y.abs() * r1[:, None]
    wp = torch.ones((), dtype=h.dtype) if w_post is None else (w_post + offset).abs()
    gg = torch.ones((), dtype=h.dtype) if gate is None else \
        (gate[:, None] if kind == "token" else gate).abs()
    c = a * wp * (1.0 if kind == "token" else gg)
    sums = ((di + r2[:, None] * g) * c).sum(1, keepdim=True) + \
        r2[:, None] * mean1 * (xh * c).sum(1, keepdim=True)
    sums = sums * U * (2 * ROW_SUM + 16)
    full = (d + 4 * U * size_d) * a * wp
    out["dgate"] = {None: None, "full": full, "token": sums.squeeze(1),
                    "channel": (full + steps * size_d * a * wp).sum(0)}[kind]
    out["dy"] = d * gg + 4 * U * size_d * gg
    if w_post is not None:
        out["dw_post"] = ((d + (steps + 4 * U) * size_d) * gg * a).sum(0)
        m2 = (size_d * gg * wp * a).sum(1, keepdim=True) / n
        token = gg if kind == "token" else 1.0
        out["dy"] = r1[:, None] * (d * gg * wp + U * 10 * (size_d * gg * wp + a * m2) +
                                   a * sums * token / n)
    return out
