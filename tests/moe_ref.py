"""A mixture-of-experts layer's routing, dispatch, combine and products in plain
numpy/torch in 64 bits, slot by slot, for the tests."""
import numpy as np
import torch

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def routing(tokens, top_k, experts, seed=0, total=None, first=0, repeat=False, dtype=torch.int64):
    """Ids as a router gives them (distinct within a token unless `repeat`),
    some experts far more often than others."""
    g = torch.Generator().manual_seed(seed)
    total = total or experts
    if repeat or top_k > total:
        ids = torch.randint(0, total, (tokens, top_k), generator=g)
    else:
        score = torch.randn(tokens, total, generator=g) + torch.randn(total, generator=g)
        ids = torch.topk(score, top_k, dim=1).indices if top_k else torch.zeros(tokens, 0, dtype=torch.int64)
    return ids.to(dtype)


def bound_rows(tokens, top_k, experts, align):
    """The most rows any routing can need, by filling runs one at a time."""
    slots = tokens * top_k
    runs = min(slots, experts)
    if slots == 0:
        return 0
    return (slots + runs * (align - 1)) // align * align


def sort(ids, experts, align=1, first=0, weight=None):
    """dest, source, offsets, counts and row_weight, slot by slot."""
    ids = np.asarray(ids, dtype=object)
    tokens, top_k = ids.shape
    rows = bound_rows(tokens, top_k, experts, align)
    flat = [int(v) - first for v in ids.reshape(-1)]
    counts = np.zeros(experts, np.int32)
    for e in flat:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = np.zeros(experts + 1, np.int32)
    for e in range(experts):
        offsets[e + 1] = offsets[e] + -(-int(counts[e]) // align) * align
    dest = np.full(tokens * top_k, -1, np.int32)
    source = np.full(rows, -1, np.int32)
    row_weight = np.zeros(rows, np.float32)
    seen = np.zeros(experts, np.int64)
    for s, e in enumerate(flat):
        if 0 <= e < experts:
            r = int(offsets[e] + seen[e])
            seen[e] += 1
            dest[s], source[r] = r, s
            if weight is not None:
                row_weight[r] = np.asarray(weight).reshape(-1)[s]
    return dest.reshape(tokens, top_k), source, offsets, counts, row_weight


def combine(y, dest, weight=None, base=None):
    """(out, sum of the magnitudes) in float64."""
    tokens, top_k = dest.shape
    out = torch.zeros(tokens, y.shape[1], dtype=torch.float64) if base is None else base.double().clone()
    mag = out.abs()
    for t in range(tokens):
        for k in range(top_k):
            r = int(dest[t, k])
            if 0 <= r < y.shape[0]:
                v = y[r].double() * (1.0 if weight is None else weight[t, k].double())
                out[t] += v
                mag[t] += v.abs()
    return out, mag


def combine_grad(dout, y, dest, weight=None):
    """(dy [rows, cols], dw [tokens, top_k], sum of |products| of dw)."""
    tokens, top_k = dest.shape
    dy = torch.zeros(y.shape, dtype=torch.float64)
    dw = torch.zeros(tokens, top_k, dtype=torch.float64)
    mag = torch.zeros_like(dw)
    for t in range(tokens):
        for k in range(top_k):
            r = int(dest[t, k])
            if 0 <= r < y.shape[0]:
                dy[r] += dout[t].double() * (1.0 if weight is None else weight[t, k].double())
                p = dout[t].double() * y[r].double()
                dw[t, k] = p.sum()
                mag[t, k] = p.abs().sum()
    return dy, dw, mag


def e2m1_weights(codes, sf, group):
    """float64 weights [..., n, k] of packed codes [..., n, k/2] and scales
    [..., n, k/group] (fp32, or int32 words of four exponent bytes)."""
    c = codes.cpu().numpy()
    v = np.stack([E2M1[c & 15], E2M1[c >> 4]], axis=-1).reshape(*c.shape[:-1], -1)
    s = sf.cpu().numpy()
    if s.dtype == np.int32:
        e = np.ascontiguousarray(s).view(np.uint8).astype(np.float64)
        s = np.exp2(e - 127)
    return torch.from_numpy(v * np.repeat(s.astype(np.float64), group, axis=-1))


def matvec(x, w, ids=None):
    """(out [rows, n], sum of |products|) from float64 x and w."""
    rows = x.shape[0] if ids is None else ids.numel()
    per = rows // x.shape[0] if x.shape[0] else 1
    n = w.shape[-2]
    out = torch.zeros(rows, n, dtype=torch.float64)
    mag = torch.zeros_like(out)
    for r in range(rows):
        e = None if ids is None else int(ids.reshape(-1)[r])
        if e is not None and not 0 <= e < w.shape[0]:
            continue
        m = w if e is None else w[e]
        out[r] = m @ x[r // per]
        mag[r] = m.abs() @ x[r // per].abs()
    return out, mag
