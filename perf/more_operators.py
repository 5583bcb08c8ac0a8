"""A mixture-of-experts layer around its products: tokens sorted by expert, rows brought to their
experts (moved as codes with their scales, or cast on the way), the experts' outputs weighted and
summed, the gradient of that, and the products themselves with 4-bit weights for the few tokens of a
serving step.

``run`` computes them from elementary torch operations in fp32, or, where ``own`` is true, with the
library. Sizes are those of the library's workloads (hidden 7168, expert intermediate 2048, weights of
18432 columns, up to 16384 tokens), with odd and small ones beside them."""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LARGEST = 4096 * 8 * 7168       # row elements of the largest listed case
_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
_F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_FLOOR = 1e-4
_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _routed(tokens, top_k, experts, total=None, first=0, align=128):
    """The routing of a case: `experts` of `total` experts, from `first` on, are here; the others' rows are not."""
    return dict(tokens=tokens, top_k=top_k, experts=experts, total=total or experts, first=first, align=align)


def listed():
    return [
        # a serving step of eight tokens: where does each token's row go
        dict(name="sort_8x8_of_256", op="sort", **_routed(8, 8, 256, align=16), ids="int64", weighted=True),
        # a training step's tokens over all the experts of a layer, runs that fill groups of 128 tokens
        dict(name="sort_16384x8_of_256", op="sort", **_routed(16384, 8, 256), ids="int64", weighted=True),
        # the norm's codes and scales go to 64 experts, scales as the products read them
        dict(name="dispatch_codes_4096x7168", op="dispatch", **_routed(4096, 8, 64), cols=7168, moved="e4m3", group=128,
             col_major=True),
        # bf16 rows of a short batch are cast on the way; a quarter of the experts are on this GPU
        dict(name="dispatch_cast_1000x2048", op="dispatch_cast", **_routed(1000, 6, 32, 128, 32), cols=2048, fmt="e4m3",
             group=32, col_major=False, weighted=False),
        # a few tokens' bf16 rows, moved as they are
        dict(name="dispatch_bf16_67x1920", op="dispatch", **_routed(67, 4, 16, align=16), cols=1920, moved="bf16", group=128,
             col_major=False),
        # the experts' outputs, weighted, on top of the shared expert's
        dict(name="combine_4096x7168", op="combine", **_routed(4096, 8, 64), cols=7168, weighted=True, base=True, sorted=True),
        # the same for one token whose rows were never sorted
        dict(name="combine_1x7168", op="combine", **_routed(1, 8, 64), cols=7168, weighted=True, base=True, sorted=False),
        # its gradient in training: the operand of the experts' backward products, and the routing weights' gradient
        dict(name="combine_backward_4096x7168", op="combine_bwd", **_routed(4096, 8, 64), cols=7168, weighted=True, fmt="e4m3",
             group=128, col_major=False, bf16=False),
        # the same for a few tokens, gradients in E5M2
        dict(name="combine_backward_257x2048", op="combine_bwd", **_routed(257, 6, 32, align=16), cols=2048, weighted=True,
             fmt="e5m2", group=64, col_major=False, bf16=False),
        # one token through a dense layer's down projection
        dict(name="matvec_1x18432", op="matvec", **_routed(1, 0, 1), n=7168, k=18432, group=32, packed=False, x="bf16",
             x_group=128, out="bf16"),
        # one token through the gate and up projections of its eight experts
        dict(name="matvec_1x8_7168", op="matvec", **_routed(1, 8, 32), n=4096, k=7168, group=128, packed=False, x="bf16",
             x_group=128, out="bf16"),
        # sixteen tokens through the down projections of their experts, from the SwiGLU's codes
        dict(name="matvec_16x8_2048", op="matvec", **_routed(16, 8, 32), n=7168, k=2048, group=32, packed=True, x="e4m3",
             x_group=128, out="bf16"),
    ]


def _spread(rng, low, high):
    """A whole number from low to high, spread over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.5)))))))


def draw(rng):
    op = rng.choice(["sort", "dispatch", "dispatch_cast", "combine", "combine_bwd", "matvec", "matvec"])
    top_k = rng.randint(1, 8)
    total = max(top_k, _spread(rng, 8, 256))
    experts = total if rng.random() < 0.6 else max(1, total // 4)
    first = 0 if experts == total else rng.randint(0, total - experts)
    align = rng.choice([1, 16, 128])
    if op == "sort":
        return dict(op=op, **_routed(_spread(rng, 1, 16384), top_k, experts, total, first, align),
                    ids=rng.choice(["int64", "int32"]), weighted=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    if op == "matvec":
        packed = rng.random() < 0.4
        unit = 4 * group if packed else group
        k = unit * max(1, int(round(_spread(rng, 128, 18432) / unit)))
        dense = rng.random() < 0.4
        most = 18432 * 7168 // k
        n = _spread(rng, 16, min(18432, most))
        here = 1 if dense else max(1, min(experts, 64, most * 8 // n))
        tokens = _spread(rng, 1, 64 if dense else 16)
        x = rng.choice(["bf16", "bf16", "e4m3", "e5m2"])
        route = _routed(tokens, 0, 1) if dense else _routed(tokens, top_k, here, max(here, top_k, min(total, 2 * here)), 0)
        return dict(op=op, **route, n=n, k=k, group=group, packed=packed, x=x,
                    x_group=group if k % 128 else rng.choice([32, 64, 128]), out=rng.choice(["bf16", "bf16", "f32"]))
    cols = 128 * _spread(rng, 1, 56) + rng.choice([0, group])
    # padding rows count too
    most = max(1, (LARGEST // cols - (align - 1) * min(experts, 64)) // (2 * top_k))
    route = _routed(_spread(rng, 1, min(16384, most)), top_k, min(experts, 64), max(top_k, min(total, 4 * min(experts, 64))),
                    0, align)
    fmt = rng.choice(["e4m3", "e4m3", "e5m2"])
    col_major = rng.random() < 0.3
    if op == "dispatch":
        return dict(op=op, **route, cols=cols, moved=rng.choice(["e4m3", "e5m2", "bf16"]), group=group, col_major=col_major)
    if op == "dispatch_cast":
        return dict(op=op, **route, cols=cols, fmt=fmt, group=group, col_major=col_major, weighted=rng.random() < 0.4)
    if op == "combine":
        return dict(op=op, **route, cols=cols, weighted=rng.random() < 0.7, base=rng.random() < 0.5,
                    sorted=rng.random() < 0.8)
    return dict(op=op, **route, cols=cols, weighted=rng.random() < 0.7, fmt=fmt, group=group, col_major=col_major,
                bf16=rng.random() < 0.3)


# ---- the plain forms -------------------------------------------------------

def _most_rows(case):
    """Rows of the sorted buffers: every slot, and a run's rounding up for as many experts as can have one."""
    slots = case["tokens"] * case["top_k"]
    return (slots + min(case["experts"], slots) * (case["align"] - 1)) // case["align"] * case["align"]


def _sort_plain(ids, experts, first, align, rows, weight):
    slots = ids.numel()
    key = ids.reshape(-1).long() - first
    key = torch.where((key >= 0) & (key < experts), key, experts)
    order = torch.argsort(key, stable=True)
    sizes = torch.zeros(experts + 1, dtype=torch.long, device=ids.device).index_add_(0, key, torch.ones_like(key))
    counts = sizes[:experts]
    zero = counts.new_zeros(1)
    offsets = torch.cat([zero, torch.cumsum((counts + align - 1) // align * align, 0)])
    starts = torch.cat([zero, torch.cumsum(counts, 0)])
    expert = key[order]
    row = offsets[expert] + torch.arange(slots, device=ids.device) - starts[expert]
    here = expert < experts
    dest = torch.empty_like(key)
    dest[order] = torch.where(here, row, -1)
    source = key.new_full((rows + 1,), -1)
    source[torch.where(here, row, rows)] = order
    source = source[:rows]
    out = dict(dest=dest.view(ids.shape).int(), source=source.int(), offsets=offsets.int(), counts=counts.int())
    if weight is not None:
        w = weight.reshape(-1)[source.clamp_min(0)]
        out["row_weight"] = torch.where(source >= 0, w, torch.zeros_like(w))
    return out


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


def _put(out, new, live):
    """new into the rows of out that belong to a run; the rows behind the last run stay as they were."""
    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[out.element_size()]
    o = out.view(kind)
    o.copy_(torch.where(live.unsqueeze(1), new.contiguous().view(kind), o))


def _places(st):
    """Of every sorted row: the slot it holds (0 where none), whether it holds one, whether it belongs to a run."""
    source = st["plan"]["source"].long()
    live = torch.arange(source.numel(), device=source.device) < st["plan"]["offsets"][-1]
    return source.clamp_min(0), source >= 0, live


def _put_scales(st, sf, live):
    if st["col_major"]:
        rows = st["out_sf"][:, :live.numel()]
        rows.copy_(torch.where(live, sf.t(), rows))
    else:
        _put(st["out_sf"], sf, live)


def _dispatch(st):
    slot, real, live = _places(st)
    token = slot // st["top_k"]
    rows = st["q"].view(torch.int16 if st["moved"] == "bf16" else torch.uint8)[token]
    _put(st["out"], torch.where(real.unsqueeze(1), rows, torch.zeros_like(rows)), live)
    if st["sf"] is None:
        return dict(q=st["out"])
    sf = (st["sf"][:, :st["q"].shape[0]].t() if st["col_major"] else st["sf"])[token]
    _put_scales(st, torch.where(real.unsqueeze(1), sf, torch.zeros_like(sf)), live)
    return dict(q=st["out"], sf=st["out_sf"])


def _cast_rows(st, x):
    """Every sorted row's values: its token's row of x, times its routing weight."""
    slot, real, live = _places(st)
    v = x.float()[slot // st["top_k"]]
    if st["w"] is not None:
        v = v * st["w"].reshape(-1)[slot].unsqueeze(1)
    return torch.where(real.unsqueeze(1), v, torch.zeros_like(v)), live


def _dispatch_cast(st):
    v, live = _cast_rows(st, st["x"])
    q, sf = _cast(v, st["group"], st["fmt"])
    _put(st["out"], q, live)
    _put_scales(st, sf, live)
    return dict(q=st["out"], sf=st["out_sf"])


def _combine(st):
    tokens, top_k = st["tokens"], st["top_k"]
    dest = torch.arange(tokens * top_k, device=DEV).view(tokens, top_k) if st["dest"] is None else st["dest"].long()
    acc = torch.zeros(tokens, st["y"].shape[1], device=DEV) if st["base"] is None else st["base"].float()
    for k in range(top_k):
        d = dest[:, k]
        v = st["y"][d.clamp_min(0)].float()
        if st["w"] is not None:
            v = v * st["w"][:, k].unsqueeze(1)
        acc = acc + torch.where((d >= 0).unsqueeze(1), v, torch.zeros_like(v))
    return dict(out=acc.to(torch.bfloat16))


def _combine_bwd(st):
    v, live = _cast_rows(st, st["dout"])
    out = {}
    if st["bf16"]:
        _put(st["dy"], v.to(torch.bfloat16), live)
        out["dy"] = st["dy"]
    else:
        q, sf = _cast(v, st["group"], st["fmt"])
        _put(st["out"], q, live)
        _put_scales(st, sf, live)
        out.update(q=st["out"], sf=st["out_sf"])
    dest, dout = st["plan"]["dest"].long(), st["dout"].float()
    dots = [(dout * st["y"][dest[:, k].clamp_min(0)].float()).sum(1) for k in range(st["top_k"])]
    dw = torch.stack(dots, dim=1)
    out["dw"] = torch.where(dest >= 0, dw, torch.zeros_like(dw))
    return out


def _weights(codes, scales, table):
    """fp32 weights [n, k] of E2M1 codes [n, k/2], two in a byte, with fp32 or packed power-of-two scales."""
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], dim=2).flatten(1)
    if scales.dtype == torch.int32:
        shifts = torch.arange(0, 32, 8, device=scales.device)
        scales = torch.exp2((((scales.unsqueeze(2) >> shifts) & 255) - 127).float()).flatten(1)
    n, groups = scales.shape
    return (v.view(n, groups, -1) * scales.unsqueeze(2)).view(n, -1)


def _matvec(st):
    x = st["x"].float() if st["x_sf"] is None else _decode(st["x"], st["x_sf"])
    if st["ids"] is None:
        out = x @ _weights(st["wq"][0], st["w_sf"][0], st["table"]).t()
        return dict(out=out.to(st["out_dtype"]))
    ids = st["ids"].reshape(-1)
    x = x[torch.arange(ids.numel(), device=DEV) // (ids.numel() // x.shape[0])]
    out = torch.zeros(ids.numel(), st["wq"].shape[1], device=DEV)
    for e in range(st["wq"].shape[0]):
        y = x @ _weights(st["wq"][e], st["w_sf"][e], st["table"]).t()
        out = torch.where((ids == e).unsqueeze(1), y, out)
    return dict(out=out.to(st["out_dtype"]))


def _sort(st):
    return _sort_plain(st["ids"], st["experts"], st["first"], st["align"], st["rows"], st["w"])


_PLAIN = dict(sort=_sort, dispatch=_dispatch, dispatch_cast=_dispatch_cast, combine=_combine, combine_bwd=_combine_bwd,
              matvec=_matvec)


# ---- the library's calls ---------------------------------------------------

def _own(st):
    import precision_quantization_amd as pq
    op = st["op"]
    if op == "sort":
        p = pq.qcast_expert_sort(st["ids"], st["experts"], st["align"], st["first"], weight=st["w"])
        out = dict(dest=p.dest, source=p.source, offsets=p.offsets, counts=p.counts)
        if st["w"] is not None:
            out["row_weight"] = p.row_weight
        return out
    if op == "matvec":
        if st["ids"] is None:
            return dict(out=pq.qcast_matvec_e2m1(st["x"], st["wq"][0], st["w_sf"][0], x_sf=st["x_sf"], out_dtype=st["out_dtype"]))
        return dict(out=pq.qcast_matvec_e2m1(st["x"], st["wq"], st["w_sf"], st["ids"], x_sf=st["x_sf"], out_dtype=st["out_dtype"]))
    if op == "combine":
        return dict(out=pq.qcast_combine(st["y"], st["dest"], st["w"], st["base"], top_k=st["top_k"]))
    p = st["plan"]
    plan = pq.ExpertPlan(p["dest"], p["source"], p["offsets"], p["counts"], None, st["align"])
    flags = pq.SF_COL_MAJOR if st["col_major"] else 0
    if op == "dispatch":
        q, sf = pq.qcast_dispatch_codes(st["q"], plan, st["sf"], sf_flags=flags, out_sf_flags=flags, out=st["out"],
                                        out_sf=st["out_sf"])
        return dict(q=q) if sf is None else dict(q=q, sf=sf)
    if op == "dispatch_cast":
        q, sf = pq.qcast_dispatch_per_token(st["x"], plan, st["w"], st["fmt"], st["group"], sf_flags=flags, out=st["out"],
                                            out_sf=st["out_sf"])
        return dict(q=q, sf=sf)
    r = pq.qcast_combine_backward_per_token(st["dout"], plan, st["y"], st["w"], st["fmt"], st["group"], sf_flags=flags,
                                            want_codes=not st["bf16"], want_dy=st["bf16"], out=st["out"],
                                            out_sf=st["out_sf"], dy=st["dy"])
    return dict(dy=r.dy, dw=r.dw) if st["bf16"] else dict(q=r.out, sf=r.out_sf, dw=r.dw)


# ---- states ----------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=gen, device=DEV).mul_(std)

    def bf16(*shape, std=1.0):
        return normal(*shape, std=std).to(torch.bfloat16)

    op, tokens, top_k = case["op"], case["tokens"], case["top_k"]
    st = dict(op=op, tokens=tokens, top_k=top_k, experts=case["experts"], first=case["first"], align=case["align"])
    ids = None
    if top_k:
        # a router's choice: some experts are chosen far more often than others
        score = normal(tokens, case["total"]) + normal(case["total"], std=0.7)
        top, ids = torch.topk(score, top_k, dim=1)
        weight = torch.softmax(top, dim=1)
        st["w"] = weight if case.get("weighted") else None
        st["rows"] = rows = _most_rows(case)
    if op == "sort":
        return dict(st, ids=ids.to(getattr(torch, case["ids"])))
    if op == "matvec":
        n, k, group, experts = case["n"], case["k"], case["group"], case["experts"]
        st.update(ids=ids, x_sf=None, table=torch.tensor(_E2M1 + [-v for v in _E2M1], device=DEV),
                  out_dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        st["wq"] = torch.randint(0, 256, (experts, n, k // 2), generator=gen, device=DEV, dtype=torch.uint8)
        if case["packed"]:
            st["w_sf"] = sum(torch.randint(114, 122, (experts, n, k // group // 4), generator=gen, device=DEV,
                                           dtype=torch.int32) << (8 * i) for i in range(4))
        else:
            st["w_sf"] = torch.exp(normal(experts, n, k // group, std=0.4)).mul_(0.01)
        # tokens come once each; a down projection has a row of its own for every chosen expert
        x = normal(tokens * top_k if top_k and case["x"] != "bf16" else tokens, k)
        if case["x"] == "bf16":
            st["x"] = x.to(torch.bfloat16)
        else:
            st["x"], st["x_sf"] = _cast(x, case["x_group"], case["x"])
        return st
    cols = case["cols"]
    st["plan"] = plan = _sort_plain(ids, case["experts"], case["first"], case["align"], rows, None)
    if op == "combine":
        st["dest"] = plan["dest"] if case["sorted"] else None
        st["y"] = bf16(rows if case["sorted"] else tokens * top_k, cols)
        st["base"] = bf16(tokens, cols) if case["base"] else None
        return st
    group = case["group"]
    st.update(group=group, col_major=case["col_major"], fmt=case.get("fmt"), out=None, out_sf=None, dy=None)
    # the sorted buffers, which a program keeps from step to step
    padded = -(-rows // 4) * 4
    if case.get("bf16"):
        st["dy"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    else:
        kind = case.get("fmt") or case["moved"]
        st["out"] = torch.zeros(rows, cols, dtype=_F8.get(kind, torch.bfloat16), device=DEV)
        if kind != "bf16":
            st["out_sf"] = torch.zeros(*((cols // group, padded) if case["col_major"] else (rows, cols // group)), device=DEV)
    # a normal activation with a few large channels
    x = normal(tokens, cols)
    x *= 1.0 + 20.0 * (torch.rand(cols, generator=gen, device=DEV) < 0.01)
    if op == "dispatch_cast":
        return dict(st, x=x.to(torch.bfloat16))
    if op == "combine_bwd":
        return dict(st, bf16=case["bf16"], dout=x.to(torch.bfloat16), y=bf16(rows, cols))
    st.update(moved=case["moved"], q=x.to(torch.bfloat16), sf=None)
    if case["moved"] != "bf16":
        st["q"], sf = _cast(x, group, case["moved"])
        st["sf"] = sf
        if case["col_major"]:
            st["sf"] = torch.zeros(cols // group, -(-tokens // 4) * 4, device=DEV)
            st["sf"][:, :tokens] = sf.t()
    return st


def run(state):
    return _own(state) if own else _PLAIN[state["op"]](state)


def work(case):
    tokens, op = case["tokens"], case["op"]
    slots = tokens * case["top_k"]
    here = slots * case["experts"] // case["total"]     # slots whose expert is here, on average
    if op == "sort":
        n = slots * (12 if case["ids"] == "int64" else 8) + 8 * case["experts"] + 4 + 4 * _most_rows(case)
        return dict(bytes=n + (4 * slots + 4 * _most_rows(case) if case["weighted"] else 0), flops=slots)
    if op == "matvec":
        n, k, e = case["n"], case["k"], case["experts"]
        rows = slots or tokens
        # experts that any of the tokens chose, were the choice even
        used = e * (1 - (1 - case["top_k"] / case["total"]) ** tokens) if case["top_k"] else 1
        scales = n * k // case["group"] * (1 if case["packed"] else 4)
        x = 2 * tokens * k if case["x"] == "bf16" else rows * (k + 4 * k // case["x_group"])
        y = rows * n * (2 if case["out"] == "bf16" else 4)
        return dict(bytes=int(used * (n * k // 2 + scales)) + x + y, flops=2 * (here or tokens) * n * k)
    cols = case["cols"]
    weights = 4 * slots if case.get("weighted") else 0
    if op == "combine":
        n = 2 * here * cols + 2 * tokens * cols * (2 if case["base"] else 1) + weights
        return dict(bytes=n + (4 * slots if case["sorted"] else 0), flops=2 * here * cols)
    scales = 4 * cols // case["group"]
    if op == "dispatch":
        row = 2 * cols if case["moved"] == "bf16" else cols + scales
        return dict(bytes=(tokens + here) * row + 4 * slots, flops=0)
    row = 2 * cols if case.get("bf16") else cols + scales
    n = 2 * tokens * cols + here * row + 4 * slots + weights
    if op == "dispatch_cast":
        return dict(bytes=n, flops=4 * (here if case["weighted"] else tokens) * cols)
    return dict(bytes=n + 2 * here * cols + 4 * slots, flops=6 * here * cols)


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


def _runs(case, ids):
    """dest, source, offsets and counts on the host, expert by expert."""
    flat = ids.reshape(-1).cpu().numpy().astype(np.int64) - case["first"]
    dest = np.full(flat.size, -1, np.int64)
    source = np.full(_most_rows(case), -1, np.int64)
    offsets, counts = [0], []
    for e in range(case["experts"]):
        slots = np.flatnonzero(flat == e)
        dest[slots] = offsets[-1] + np.arange(slots.size)
        source[dest[slots]] = slots
        counts.append(slots.size)
        offsets.append(offsets[-1] + -(-slots.size // case["align"]) * case["align"])
    return dest.reshape(tuple(ids.shape)), source, np.array(offsets), np.array(counts)


def exact(case, seed):
    st = prepare(case, seed)
    op, tokens, top_k = st["op"], st["tokens"], st["top_k"]
    if op == "sort":
        dest, source, offsets, counts = _runs(case, st["ids"])
        out = dict(dest=torch.from_numpy(dest).int(), source=torch.from_numpy(source).int(),
                   offsets=torch.from_numpy(offsets).int(), counts=torch.from_numpy(counts).int())
        if st["w"] is not None:
            flat = st["w"].cpu().double().numpy().reshape(-1)
            out["row_weight"] = torch.from_numpy(np.where(source >= 0, flat[source], 0.0))
        return {k: v.to(DEV) for k, v in out.items()}
    if op == "matvec":
        x = st["x"].float().double()
        if st["x_sf"] is not None:
            x = x * st["x_sf"].double().repeat_interleave(case["x_group"], dim=1)
        chosen = [0] * tokens if st["ids"] is None else st["ids"].reshape(-1).tolist()
        per = len(chosen) // x.shape[0]
        out = torch.zeros(len(chosen), case["n"], dtype=torch.float64, device=DEV)
        value = torch.tensor([s * v for s in (1.0, -1.0) for v in _E2M1], dtype=torch.float64, device=DEV)
        for e in sorted({c for c in chosen if 0 <= c < case["experts"]}):
            codes = st["wq"][e].int()
            w = torch.empty(case["n"], case["k"], dtype=torch.float64, device=DEV)
            w[:, 0::2], w[:, 1::2] = value[codes % 16], value[codes // 16]
            scale = st["w_sf"][e]
            if case["packed"]:
                raw = scale.view(torch.uint8).double()     # the bytes of a word, lowest first
                scale = torch.pow(torch.full_like(raw, 2.0), raw - 127)
            w *= scale.double().repeat_interleave(case["group"], dim=1)
            for r, c in enumerate(chosen):
                if c == e:
                    out[r] = w @ x[r // per]
        return dict(out=out)
    if op == "combine":
        dest = st["dest"].tolist() if st["dest"] is not None else [list(range(t * top_k, (t + 1) * top_k)) for t in range(tokens)]
        index = torch.tensor(dest, device=DEV)
        w = torch.ones(tokens, top_k, dtype=torch.float64, device=DEV) if st["w"] is None else st["w"].double()
        w = w * (index >= 0)
        total = torch.zeros(tokens, case["cols"], dtype=torch.float64, device=DEV)
        for k in range(top_k):
            total += w[:, k:k + 1] * st["y"].double()[index[:, k].clamp(min=0)]
        return dict(out=total if st["base"] is None else total + st["base"].double())
    # the sorted rows: [slot] rows of values at their places, zeros in the runs' gaps, and the buffers' zeros behind
    source = st["plan"]["source"].long()
    end = int(st["plan"]["offsets"][-1])
    held = torch.nonzero(source >= 0).flatten()
    slots = source[held]

    def scales(sf):
        return _columns(sf) if case["col_major"] else sf

    def _columns(sf):
        out = torch.zeros(sf.shape[1], -(-sf.shape[0] // 4) * 4, dtype=torch.float64, device=DEV)
        out[:, :sf.shape[0]] = sf.t()
        return out

    cols = case["cols"]
    v = torch.zeros(source.numel(), cols, dtype=torch.float64, device=DEV)
    if op == "dispatch":
        v[held] = st["q"][slots // top_k].float().double() if case["moved"] == "bf16" else \
            st["q"].float().double()[slots // top_k]
        if st["sf"] is None:
            return dict(q=v)
        sf = torch.zeros(source.numel(), cols // case["group"], dtype=torch.float64, device=DEV)
        sf[held] = (st["sf"].t()[:tokens] if case["col_major"] else st["sf"]).double()[slots // top_k]
        return dict(q=v, sf=scales(sf))
    x = (st["x"] if op == "dispatch_cast" else st["dout"]).double()
    v[held] = x[slots // top_k]
    if st["w"] is not None:
        v[held] *= st["w"].double().reshape(-1)[slots].unsqueeze(1)
    out = {}
    if case.get("bf16"):
        out["dy"] = v
    else:
        q, sf = _groups64(v, case["group"], case["fmt"])
        sf[end:] = 0
        out.update(q=q, sf=scales(sf))
    if op == "combine_bwd":
        dw = torch.zeros(tokens * top_k, dtype=torch.float64, device=DEV)
        for part in torch.split(torch.arange(held.numel(), device=DEV), 8192):
            dw[slots[part]] = (x[slots[part] // top_k] * st["y"][held[part]].double()).sum(1)
        out["dw"] = dw.view(tokens, top_k)
    return out
