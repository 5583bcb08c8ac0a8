"""The training and serving operators around the casts: SwiGLU with an 8-bit checkpoint of its input,
its backward pass from that checkpoint, stored codes turned into a weight gradient's operand, and the
norms before and after a block with its gate and residual scale, forward and backward.

``run`` computes them from elementary torch operations in fp32, or, where ``own`` is true, with the
library. Sizes are those of the library's workloads (hidden 7168, expert intermediate 2048, 4096 to
16384 tokens), with odd and small ones beside them."""
import math

import torch

own = False

DEV = "cuda"
LARGEST = 16384 * 7168          # elements of the largest listed case
_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FLOOR = 1e-4


def listed():
    return [
        # one expert layer's forward pass in training: codes for the next product, checkpoint for the backward
        dict(name="swiglu_checkpoint_8192x2048", op="swiglu", rows=8192, cols=2048, weighted=True, clamp=0.0,
             fmt="e4m3", ckpt="e4m3", group=128),
        # a few tokens reach an expert; clamped, 32-element groups, an odd row count
        dict(name="swiglu_checkpoint_67x1920", op="swiglu", rows=67, cols=1920, weighted=True, clamp=6.0,
             fmt="e4m3", ckpt="e5m2", group=32),
        # the same layer's backward pass: operands of both products of the gradient, and the routing weight's gradient
        dict(name="swiglu_backward_8192x2048", op="swiglu_bwd", rows=8192, cols=2048, weighted=True, clamp=0.0,
             fmt="e4m3", ckpt="e4m3"),
        # tokens that do not fill the last group of 128, gradients in E5M2, a clamp
        dict(name="swiglu_backward_1000x1920", op="swiglu_bwd", rows=1000, cols=1920, weighted=True, clamp=6.0,
             fmt="e5m2", ckpt="e4m3"),
        # a layer's stored input becomes the operand of its weight gradient
        dict(name="recast_16384x7168", op="recast", rows=16384, cols=7168, fmt="e4m3", ckpt="e4m3", group=128),
        # the same for a short, ragged batch
        dict(name="recast_1000x2048", op="recast", rows=1000, cols=2048, fmt="e4m3", ckpt="e5m2", group=32),
        # between two blocks in training: both norms, gate, residual, cast, both checkpoints
        dict(name="norm_4096x7168", op="norm", rows=4096, cols=7168, gate="channel", post=True, save=True,
             fmt="e4m3", group=128),
        # the same between two blocks for one token in serving: nothing is kept
        dict(name="norm_1x7168", op="norm", rows=1, cols=7168, gate="none", post=True, save=False,
             fmt="e4m3", group=128),
        # no post-norm, one gate per token, 32-element groups
        dict(name="norm_257x2048", op="norm", rows=257, cols=2048, gate="token", post=False, save=False,
             fmt="e4m3", group=32),
        # its backward pass from the checkpoints: gradients of both weights and the channel gate
        dict(name="norm_backward_4096x7168", op="norm_bwd", rows=4096, cols=7168, gate="channel", post=True,
             ckpt="e4m3", fmt="e4m3", group=128),
        # from bf16 activations, elementwise gate
        dict(name="norm_backward_1000x2048", op="norm_bwd", rows=1000, cols=2048, gate="full", post=True,
             ckpt="bf16", fmt="e5m2", group=128),
        # a few tokens
        dict(name="norm_backward_67x1920", op="norm_bwd", rows=67, cols=1920, gate="token", post=True,
             ckpt="e4m3", fmt="e4m3", group=64),
    ]


def draw(rng):
    op = rng.choice(["swiglu", "swiglu_bwd", "recast", "norm", "norm_bwd"])
    units = max(1, min(56, int(round(math.exp(rng.uniform(0, math.log(56)))))))
    cols = 128 * units
    weight = {"swiglu": 3.5, "swiglu_bwd": 4.5, "recast": 1.0, "norm": 4.5, "norm_bwd": 4.5}[op]
    most = max(1, min(16384, int(LARGEST / (weight * cols))))
    rows = max(1, min(most, int(round(math.exp(rng.uniform(0, math.log(most + 0.5)))))))
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    group = rng.choice([32, 64, 128])
    if op == "swiglu":
        return dict(op=op, rows=rows, cols=cols + rng.choice([0, group]), weighted=rng.random() < 0.7,
                    clamp=rng.choice([0.0, 6.0]), fmt=fmt, ckpt=rng.choice(["e4m3", "e5m2"]), group=group)
    if op == "swiglu_bwd":
        return dict(op=op, rows=rows, cols=cols, weighted=rng.random() < 0.7, clamp=rng.choice([0.0, 6.0]),
                    fmt=fmt, ckpt=rng.choice(["e4m3", "e5m2"]))
    if op == "recast":
        return dict(op=op, rows=rows, cols=cols, fmt=fmt, ckpt=rng.choice(["e4m3", "e5m2"]), group=group)
    case = dict(op=op, rows=rows, cols=cols + rng.choice([0, group]),
                gate=rng.choice(["none", "channel", "token", "full"]), post=rng.random() < 0.75, fmt=fmt, group=group)
    if op == "norm":
        return dict(case, save=rng.random() < 0.5 and case["cols"] % 128 == 0)
    return dict(case, ckpt=rng.choice(["e4m3", "e5m2", "bf16"]) if case["cols"] % 128 == 0 else "bf16")


# ---- the plain forms -------------------------------------------------------

def _cast(x, group, fmt):
    """Codes and scales of fp32 x [rows, cols], one scale per `group` elements of a row."""
    rows, cols = x.shape
    g = x.view(rows, cols // group, group)
    sf = g.abs().amax(dim=2).clamp_min(_FLOOR) / _MAX[fmt]
    y = (g * (1.0 / sf).unsqueeze(2)).clamp(-_MAX[fmt], _MAX[fmt])
    return y.to(_F8[fmt]).view(rows, cols), sf


def _decode(q, sf):
    rows, cols = q.shape
    return (q.float().view(rows, sf.shape[1], -1) * sf.unsqueeze(2)).view(rows, cols)


def _cast_T(x, fmt):
    """The cast of x transposed, 128 tokens a group; a last partial group is filled up with zeros."""
    rows = x.shape[0]
    pad = -rows % 128
    if pad:
        x = torch.cat([x, x.new_zeros(pad, x.shape[1])])
    return _cast(x.t().contiguous(), 128, fmt)


def _swiglu_terms(h, clamp):
    g, u = h.chunk(2, dim=1)
    if clamp > 0:
        passes = (g <= clamp).float(), (u.abs() <= clamp).float()
        g, u = g.clamp(max=clamp), u.clamp(-clamp, clamp)
    else:
        passes = None
    s = 1.0 / (1.0 + torch.exp(-g))
    return g, u, s, passes


def _swiglu(st):
    h = st["h"].float()
    g, u, s, _ = _swiglu_terms(h, st["clamp"])
    v = g * s * u
    if st["w"] is not None:
        v = v * st["w"].unsqueeze(1)
    q, sf = _cast(v, st["group"], st["fmt"])
    ckpt, ckpt_sf = _cast(h, st["group"], st["ckpt"])
    return dict(q=q, sf=sf, ckpt=ckpt, ckpt_sf=ckpt_sf)


def _swiglu_bwd(st):
    h, dv = _decode(st["ckpt"], st["ckpt_sf"]), st["dv"].float()
    g, u, s, passes = _swiglu_terms(h, st["clamp"])
    silu = g * s
    x = silu * u
    dw = (dv * x).sum(dim=1)
    if st["w"] is not None:
        w = st["w"].unsqueeze(1)
        dv, x = dv * w, x * w
    dg, du = dv * u * (s + silu * (1.0 - s)), dv * silu
    if passes is not None:
        dg, du = dg * passes[0], du * passes[1]
    d = torch.cat([dg, du], dim=1)
    q, sf = _cast(d, 128, st["fmt"])
    qt, sft = _cast_T(d, st["fmt"])
    vt, vsft = _cast_T(x, st["fmt"])
    return dict(dh=q, dh_sf=sf, dh_t=qt, dh_t_sf=sft, v_t=vt, v_t_sf=vsft, dw=dw)


def _recast(st):
    q, sf = _cast_T(_decode(st["ckpt"], st["ckpt_sf"]), st["fmt"])
    return dict(q=q, sf=sf)


def _gate(st):
    g = st["gate"]
    return None if g is None else g.float().unsqueeze(1) if st["gate_kind"] == "token" else g.float()


def _norm(st):
    y, h = st["y"].float(), st["h"].float()
    out = {}
    if st["w_post"] is not None:
        r1 = 1.0 / torch.sqrt((y * y).mean(dim=1) + st["eps"])
        a = y * r1.unsqueeze(1)
        z = a * st["w_post"].float()
        out["rstd_post"] = r1
    else:
        a = z = y
    gate = _gate(st)
    if gate is not None:
        z = z * gate
    x = st["alpha"] * h + z
    r2 = 1.0 / torch.sqrt((x * x).mean(dim=1) + st["eps"])
    xh = x * r2.unsqueeze(1)
    q, sf = _cast(xh * st["w_pre"].float(), st["group"], st["fmt"])
    out.update(h=x.to(torch.bfloat16), q=q, sf=sf, rstd_pre=r2)
    if st["save"]:
        out["y_ckpt"], out["y_ckpt_sf"] = _cast(y, 128, "e4m3")
        out["h_ckpt"], out["h_ckpt_sf"] = _cast(x, 128, "e4m3")
    return out


def _norm_bwd(st):
    dx, dhn = st["dx"].float(), st["dhn"].float()
    r2 = st["rstd_pre"].unsqueeze(1)
    r1 = None if st["rstd_post"] is None else st["rstd_post"].unsqueeze(1)
    x, y = (st["x"].float(), st["y"].float()) if st["x_sf"] is None else (_decode(st["x"], st["x_sf"]), _decode(st["y"], st["y_sf"]))
    xh = x * r2
    a = y if r1 is None else y * r1
    g = dx * st["w_pre"].float()
    d = dhn + r2 * (g - xh * (g * xh).mean(dim=1, keepdim=True))
    w_post = None if st["w_post"] is None else st["w_post"].float()
    z = a if w_post is None else a * w_post
    gate = _gate(st)
    dz = d if gate is None else d * gate
    out = dict(dh=(st["alpha"] * d).to(torch.bfloat16), dw_pre=(dx * xh).sum(dim=0))
    if w_post is None:
        dy = dz
    else:
        da = dz * w_post
        dy = r1 * (da - a * (da * a).mean(dim=1, keepdim=True))
        out["dw_post"] = (dz * a).sum(dim=0)
    if st["gate_kind"] == "channel":
        out["dgate"] = (d * z).sum(dim=0)
    elif st["gate_kind"] == "token":
        out["dgate"] = (d * z).sum(dim=1)
    elif st["gate_kind"] == "full":
        out["dgate"] = (d * z).to(torch.bfloat16)
    out["dy"], out["dy_sf"] = _cast(dy, st["group"], st["fmt"])
    return out


_PLAIN = dict(swiglu=_swiglu, swiglu_bwd=_swiglu_bwd, recast=_recast, norm=_norm, norm_bwd=_norm_bwd)


# ---- the library's calls ---------------------------------------------------

def _own(st):
    import precision_quantization_amd as pq
    op = st["op"]
    if op == "swiglu":
        q, sf, ckpt, ckpt_sf = pq.qcast_swiglu_checkpoint(st["h"], st["w"], st["fmt"], st["group"], swiglu_clamp=st["clamp"],
                                                          ckpt_fmt=st["ckpt"])
        return dict(q=q, sf=sf, ckpt=ckpt, ckpt_sf=ckpt_sf)
    if op == "swiglu_bwd":
        r = pq.qcast_swiglu_backward_checkpoint(st["ckpt"], st["ckpt_sf"], st["dv"], st["w"], st["fmt"],
                                                swiglu_clamp=st["clamp"])
        return dict(dh=r.dh, dh_sf=r.dh_sf, dh_t=r.dh_t, dh_t_sf=r.dh_t_sf, v_t=r.v_t, v_t_sf=r.v_t_sf, dw=r.dw)
    if op == "recast":
        q, sf = pq.qcast_recast_per_channel_T(st["ckpt"], st["ckpt_sf"], st["fmt"])
        return dict(q=q, sf=sf)
    if op == "norm":
        r = pq.qcast_norm_per_token(st["h"], st["w_pre"], st["y"], st["w_post"], st["gate"], residual_scale=st["alpha"],
                                    eps=st["eps"], fmt=st["fmt"], group=st["group"],
                                    ckpt_fmt="e4m3" if st["save"] else None)
        out = dict(h=r.h, q=r.out, sf=r.out_sf, rstd_pre=r.rstd_pre)
        if st["w_post"] is not None:
            out["rstd_post"] = r.rstd_post
        if st["save"]:
            out.update(y_ckpt=r.y_ckpt, y_ckpt_sf=r.y_ckpt_sf, h_ckpt=r.h_ckpt, h_ckpt_sf=r.h_ckpt_sf)
        return out
    r = pq.qcast_norm_backward_per_token(st["dx"], st["x"], st["rstd_pre"], st["w_pre"], dh=st["dhn"], saved_h_sf=st["x_sf"],
                                         saved_y=st["y"], saved_y_sf=st["y_sf"], rstd_post=st["rstd_post"],
                                         w_post=st["w_post"], gate=st["gate"], residual_scale=st["alpha"], fmt=st["fmt"],
                                         group=st["group"])
    out = dict(dh=r.dh, dw_pre=r.dw_pre, dy=r.out, dy_sf=r.out_sf)
    if st["w_post"] is not None:
        out["dw_post"] = r.dw_post
    if st["gate"] is not None:
        out["dgate"] = r.dgate
    return out


# ---- states ----------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(std).add_(mean)

    def bf16(*shape, std=1.0, mean=0.0):
        return normal(*shape, std=std, mean=mean).to(torch.bfloat16)

    rows, cols, op = case["rows"], case["cols"], case["op"]
    st = dict(op=op, fmt=case["fmt"], group=case.get("group", 128), ckpt=case.get("ckpt"), clamp=case.get("clamp", 0.0))
    if op in ("swiglu", "swiglu_bwd"):
        h = bf16(rows, 2 * cols, std=2.0)
        st["w"] = torch.rand(rows, generator=gen, device=DEV) if case["weighted"] else None
        if op == "swiglu":
            return dict(st, h=h)
        st["ckpt"], st["ckpt_sf"] = _cast(h.float(), 128, case["ckpt"])
        return dict(st, dv=bf16(rows, cols))
    if op == "recast":
        # the layer's input: a normal one with a few large channels
        x = normal(rows, cols)
        x *= 1.0 + 20.0 * (torch.rand(cols, generator=gen, device=DEV) < 0.01)
        st["ckpt"], st["ckpt_sf"] = _cast(x, st["group"], case["ckpt"])
        return st
    st.update(alpha=1.0 if case["gate"] == "none" else 0.75, eps=1e-6, save=case.get("save", False), gate_kind=case["gate"],
              w_pre=bf16(cols, std=0.2, mean=1.0), w_post=bf16(cols, std=0.2, mean=1.0) if case["post"] else None)
    st["gate"] = {"none": lambda: None, "channel": lambda: bf16(cols, std=0.5, mean=0.5),
                  "token": lambda: torch.rand(rows, generator=gen, device=DEV),
                  "full": lambda: bf16(rows, cols, std=0.5, mean=0.5)}[case["gate"]]()
    # the block's output, and a residual stream with a few large channels
    y = bf16(rows, cols, std=0.7)
    h = normal(rows, cols, std=2.0)
    h *= 1.0 + 10.0 * (torch.rand(cols, generator=gen, device=DEV) < 0.005)
    st.update(y=y, h=h.to(torch.bfloat16))
    if op == "norm":
        return st
    fwd = _norm(st)
    st.update(rstd_pre=fwd["rstd_pre"], rstd_post=fwd.get("rstd_post"), x=fwd["h"], x_sf=None, y_sf=None)
    if case["ckpt"] != "bf16":
        st["y"], st["y_sf"] = _cast(y.float(), 128, case["ckpt"])
        st["x"], st["x_sf"] = _cast(fwd["h"].float(), 128, case["ckpt"])
    st.update(h=None, dx=bf16(rows, cols), dhn=bf16(rows, cols))
    return st


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    r, c, op = case["rows"], case["cols"], case["op"]
    g = case.get("group", 128)
    pad = -(-r // 128) * 128
    if op == "swiglu":
        n = 4 * r * c + 3 * r * c + 3 * r * c // g * 4 + (4 * r if case["weighted"] else 0)
        return dict(bytes=n, flops=12 * r * c)
    if op == "swiglu_bwd":
        n = 2 * r * c + 2 * r * c + 2 * r * c + 3 * pad * c + 4 * (4 * r * c // 128 + 3 * pad * c // 128) + 8 * r
        return dict(bytes=n, flops=30 * r * c)
    if op == "recast":
        return dict(bytes=r * c + pad * c + 4 * (r * c // g + pad * c // 128), flops=4 * r * c)
    gate = {"none": 0, "channel": 2 * c, "token": 4 * r, "full": 2 * r * c}[case["gate"]]
    weights = 2 * c + (2 * c if case["post"] else 0)
    if op == "norm":
        n = 4 * r * c + gate + weights + 3 * r * c + 4 * r * c // g + 4 * r * (2 if case["post"] else 1)
        if case["save"]:
            n += 2 * (r * c + 4 * r * c // 128)
        return dict(bytes=n, flops=16 * r * c)
    saved = 2 * r * c * 2 if case["ckpt"] == "bf16" else 2 * (r * c + 4 * r * c // 128)
    dgate = {"none": 0, "channel": 4 * c, "token": 4 * r, "full": 2 * r * c}[case["gate"]]
    n = 4 * r * c + saved + gate + dgate + weights + 2 * weights + 4 * r * (2 if case["post"] else 1)
    return dict(bytes=n + 2 * r * c + r * c + 4 * r * c // g, flops=30 * r * c)


# ---- the definitions in 64 bits --------------------------------------------

_BITS = {"e4m3": (3, -6), "e5m2": (2, -14)}     # mantissa bits, smallest normal exponent


def _to_f8(v, fmt):
    """The values of the nearest codes (ties to the even one) of fp64 v, at most the format's largest."""
    bits, low = _BITS[fmt]
    exponent = torch.frexp(v)[1].clamp_min(low + 1) - 1 - bits
    step = torch.ldexp(torch.ones_like(v), exponent)
    return (torch.round(v / step) * step).clamp(-_MAX[fmt], _MAX[fmt])


def _groups64(v, group, fmt):
    parts = v.unflatten(1, (-1, group))
    top = torch.maximum(parts.abs().amax(dim=2, keepdim=True), torch.tensor(_FLOOR, dtype=torch.float64, device=v.device))
    scale = top / _MAX[fmt]
    return _to_f8(parts / scale, fmt).flatten(1), scale.squeeze(2)


def _tokens64(v, fmt):
    full = torch.zeros(-(-v.shape[0] // 128) * 128, v.shape[1], dtype=torch.float64, device=v.device)
    full[: v.shape[0]] = v
    return _groups64(full.T.contiguous(), 128, fmt)


def _stored64(codes, scales):
    per = codes.shape[1] // scales.shape[1]
    return codes.float().double() * scales.double().repeat_interleave(per, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op, fmt, group = st["op"], st["fmt"], st["group"]
    if op == "recast":
        q, sf = _tokens64(_stored64(st["ckpt"], st["ckpt_sf"]), fmt)
        return dict(q=q, sf=sf)
    if op in ("swiglu", "swiglu_bwd"):
        h = st["h"].double() if op == "swiglu" else _stored64(st["ckpt"], st["ckpt_sf"])
        c = st["clamp"] if st["clamp"] > 0 else math.inf
        half = h.shape[1] // 2
        gate, up = h[:, :half], h[:, half:]
        free_g, free_u = gate <= c, up.abs() <= c
        gate, up = torch.where(free_g, gate, torch.full_like(gate, c)), torch.where(free_u, up, torch.sign(up) * c)
        sig = torch.sigmoid(gate)
        w = torch.ones(h.shape[0], 1, dtype=torch.float64, device=h.device) if st["w"] is None else st["w"].double()[:, None]
        prod = gate * sig * up
        if op == "swiglu":
            q, sf = _groups64(prod * w, group, fmt)
            ckpt, ckpt_sf = _groups64(h, group, st["ckpt"])
            return dict(q=q, sf=sf, ckpt=ckpt, ckpt_sf=ckpt_sf)
        dv = st["dv"].double()
        zero = torch.zeros_like(dv)
        d_gate = torch.where(free_g, dv * w * up * sig * (1 + gate * (1 - sig)), zero)
        d_up = torch.where(free_u, dv * w * gate * sig, zero)
        d = torch.cat([d_gate, d_up], dim=1)
        q, sf = _groups64(d, 128, fmt)
        qt, sft = _tokens64(d, fmt)
        vt, vsft = _tokens64(prod * w, fmt)
        return dict(dh=q, dh_sf=sf, dh_t=qt, dh_t_sf=sft, v_t=vt, v_t_sf=vsft, dw=(dv * prod).sum(1))
    rows, cols = case["rows"], case["cols"]
    one = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    w_pre = st["w_pre"].double()
    w_post = one if st["w_post"] is None else st["w_post"].double()
    gate = one if st["gate"] is None else st["gate"].double()
    gate = gate[:, None] if st["gate_kind"] == "token" else gate
    if op == "norm":
        y = st["y"].double()
        r1 = None if st["w_post"] is None else (y.square().sum(1) / cols + st["eps"]).rsqrt()
        a = y if r1 is None else y * r1[:, None]
        x = st["alpha"] * st["h"].double() + gate * w_post * a
        r2 = (x.square().sum(1) / cols + st["eps"]).rsqrt()
        q, sf = _groups64(x * r2[:, None] * w_pre, group, fmt)
        out = dict(h=x, q=q, sf=sf, rstd_pre=r2)
        if r1 is not None:
            out["rstd_post"] = r1
        if st["save"]:
            out["y_ckpt"], out["y_ckpt_sf"] = _groups64(y, 128, "e4m3")
            out["h_ckpt"], out["h_ckpt_sf"] = _groups64(x, 128, "e4m3")
        return out
    r2 = st["rstd_pre"].double()[:, None]
    r1 = one if st["rstd_post"] is None else st["rstd_post"].double()[:, None]
    x, y = (st["x"].double(), st["y"].double()) if st["x_sf"] is None else (_stored64(st["x"], st["x_sf"]), _stored64(st["y"], st["y_sf"]))
    xh, a = x * r2, y * r1
    dx = st["dx"].double()
    along = dx * w_pre
    total = st["dhn"].double() + r2 * (along - xh * ((along * xh).sum(1, keepdim=True) / cols))
    out = dict(dh=st["alpha"] * total, dw_pre=(dx * xh).sum(0))
    da = total * gate * w_post
    dy = da
    if st["w_post"] is not None:
        dy = r1 * (da - a * ((da * a).sum(1, keepdim=True) / cols))
        out["dw_post"] = (total * gate * a).sum(0)
    if st["gate"] is not None:
        dgate = total * a * w_post
        out["dgate"] = {"channel": lambda: dgate.sum(0), "token": lambda: dgate.sum(1), "full": lambda: dgate}[st["gate_kind"]]()
    out["dy"], out["dy_sf"] = _groups64(dy, group, fmt)
    return out
