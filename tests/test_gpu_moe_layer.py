"""The operators of a mixture-of-experts layer one after the other, as a
training step and a decoding step use them; in captured graphs, on streams of
their own and from two threads; and what they leave alone.

Rows of experts are independent, so the sorted layer has to give exactly what
the same casts and products give slot by slot, unsorted. Products of the
experts are done in float64 here and rounded once, which no order of adding
64-bit products changes; weights of slots are powers of two where a product
with them has to be exact in bf16."""
import threading

import numpy as np
import pytest
import torch

import moe_ref
import precision_quantization_amd as pq
from test_gpu_combine import near
from test_gpu_dispatch import bytes_of, filled
from test_gpu_guard import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def values(q, sf):
    """float64 values, on the CPU, of a cast's codes and row-major scales."""
    return q.float().double().cpu() * sf.double().cpu().repeat_interleave(q.shape[1] // sf.shape[1], 1)


def grouped(a, w, experts):
    """bf16 rows a[r] @ w[experts[r]].T; rows without an expert are zeros."""
    out = torch.zeros(a.shape[0], w.shape[1], dtype=torch.float64)
    for e in range(w.shape[0]):
        r = (experts == e).nonzero()[:, 0]
        out[r] = a[r] @ w[e].double().t()
    return out.to(torch.bfloat16)


@pytest.mark.parametrize("tokens,top_k,experts,align", [(1, 2, 4, 128), (37, 2, 6, 16), (130, 4, 9, 1)])
def test_a_training_step(tokens, top_k, experts, align):
    hidden, wide = 256, 128
    g = torch.Generator().manual_seed(tokens)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    w1 = (torch.randn(experts, 2 * wide, hidden, generator=g) / 16).to(torch.bfloat16)
    w2 = (torch.randn(experts, hidden, wide, generator=g) / 11).to(torch.bfloat16)
    ids = moe_ref.routing(tokens, top_k, experts + 1, seed=tokens)      # the last expert is elsewhere
    weight = torch.exp2(-torch.randint(0, 4, (tokens, top_k), generator=g).float())
    dout = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    xd, wd, dd = x.to(DEV), weight.to(DEV), dout.to(DEV)
    slot_e = ids.reshape(-1)
    here = slot_e < experts
    dest_ref, source_ref, offsets_ref, counts_ref, rw_ref = moe_ref.sort(ids.numpy(), experts, align, 0, weight.numpy())
    rows = source_ref.size
    row_e = torch.full((rows,), -1)
    row_e[torch.from_numpy(dest_ref.reshape(-1)[here.numpy()]).long()] = slot_e[here]
    slot_of = torch.from_numpy(dest_ref.reshape(-1)).long()

    # forward: codes sorted, the first product, SwiGLU and its cast with the
    # slot's weight or without, the second product, and the sum
    plan = pq.qcast_expert_sort(ids.to(DEV), experts, align, weight=wd)
    q, sf = pq.qcast_per_token(xd)
    xe, xe_sf = pq.qcast_dispatch_codes(q, plan, sf)
    live = int(offsets_ref[-1])
    assert np.array_equal(plan.dest.cpu().numpy(), dest_ref) and torch.equal(plan.row_weight.cpu()[:live],
                                                                             torch.from_numpy(rw_ref[:live]))
    once, once_sf = pq.qcast_dispatch_per_token(xd, plan)
    got = torch.from_numpy(np.flatnonzero(source_ref >= 0))
    assert np.array_equal(bytes_of(once)[got], bytes_of(xe)[got]) and torch.equal(once_sf.cpu()[got], xe_sf.cpu()[got])
    xv = values(q, sf)
    h_slots = grouped(xv.repeat_interleave(top_k, 0), w1, torch.where(here, slot_e, -1))
    h = torch.zeros(rows, 2 * wide, dtype=torch.bfloat16)
    held = row_e >= 0
    h[held] = grouped(values(xe, xe_sf)[held], w1, row_e[held])
    assert torch.equal(h[slot_of[here]], h_slots[here])
    for late in (True, False):                       # the weight at the sum, or in the activation
        rw = None if late else plan.row_weight
        a, a_sf = pq.qcast_swiglu_per_token(h.to(DEV), rw)
        a_slots, a_slots_sf = pq.qcast_swiglu_per_token(h_slots.to(DEV), None if late else wd.reshape(-1))
        assert np.array_equal(bytes_of(a)[slot_of[here]], bytes_of(a_slots)[here.numpy()])
        y = torch.full((rows, hidden), float("nan"), dtype=torch.bfloat16)
        y[held] = grouped(values(a, a_sf)[held], w2, row_e[held])
        y_slots = grouped(values(a_slots, a_slots_sf), w2, torch.where(here, slot_e, -1))
        out = pq.qcast_combine(y.to(DEV), plan.dest, wd if late else None, xd)
        k_of = torch.where(here.reshape(tokens, top_k), torch.arange(tokens * top_k).reshape(tokens, top_k), -1)
        want, mag = moe_ref.combine(y_slots, k_of.numpy(), weight if late else None, x)
        near(out, want, mag, top_k, "the layer's output")
        # unsorted, the very same bits
        flat = pq.qcast_combine(y_slots.to(DEV), k_of.to(torch.int32).to(DEV), wd if late else None, xd)
        assert torch.equal(out, flat)

    # backward, the weight at the sum: the experts' output gradient cast, the
    # weights' gradient, SwiGLU's gradient, and the tokens' own
    a, a_sf = pq.qcast_swiglu_per_token(h.to(DEV))
    y[held] = grouped(values(a, a_sf)[held], w2, row_e[held])
    back = pq.qcast_combine_backward_per_token(dd, plan, y.to(DEV), wd, want_dy=True)
    scaled = (dout.repeat_interleave(top_k, 0).float() * weight.reshape(-1, 1)).to(torch.bfloat16)   # exact
    q_slots, q_slots_sf = pq.qcast_per_token(scaled.to(DEV))
    assert np.array_equal(bytes_of(back.out)[slot_of[here]], bytes_of(q_slots)[here.numpy()])
    assert torch.equal(back.out_sf.cpu()[slot_of[here]], q_slots_sf.cpu()[here])
    assert torch.equal(back.dy.cpu()[slot_of[here]], scaled[here])
    _, dw, mag = moe_ref.combine_grad(dout, y, dest_ref, weight)
    assert ((back.dw.double().cpu() - dw).abs() <= mag * (hidden / 64 + 24) * 2.0 ** -24).all()
    da = torch.zeros(rows, wide, dtype=torch.bfloat16)
    da[held] = grouped(values(back.out, back.out_sf)[held], w2.transpose(1, 2), row_e[held])
    dh = pq.qcast_swiglu_backward_per_token(h.to(DEV), da.to(DEV))
    dh_q, dh_sf = dh[0], dh[1]
    dx_rows = torch.full((rows, hidden), float("nan"), dtype=torch.bfloat16)
    dx_rows[held] = grouped(values(dh_q, dh_sf)[held], w1.transpose(1, 2), row_e[held])
    dx = pq.qcast_combine(dx_rows.to(DEV), plan.dest, None, dd)      # the residual's gradient as base
    want, mag = moe_ref.combine(dx_rows, dest_ref, None, dout)
    near(dx, want, mag, top_k, "the tokens' gradient")


def decode_weights(g, experts, n, k, group):
    return (torch.randint(0, 256, (experts, n, k // 2), generator=g, dtype=torch.uint8),
            torch.exp(torch.randn(experts, n, k // group, generator=g)) / 40)


def decode(x, ids, weight, w1, s1, w2, s2, shared, shared_sf):
    """A decoding step of a layer with a shared part; every stage's output."""
    tokens, top_k = ids.shape
    up = pq.qcast_matvec_e2m1(x, w1, s1, ids)
    act, act_sf = pq.qcast_swiglu_per_token(up)
    y = pq.qcast_matvec_e2m1(act, w2, s2, ids, x_sf=act_sf)
    base = pq.qcast_matvec_e2m1(x, shared, shared_sf)
    return up, act, act_sf, y, base, pq.qcast_combine(y, None, weight, base, top_k=top_k)


@pytest.mark.parametrize("tokens,top_k,experts", [(1, 8, 32), (1, 1, 1), (5, 2, 3), (24, 4, 6)])
def test_a_decoding_step(tokens, top_k, experts):
    hidden, wide = 512, 256
    g = torch.Generator().manual_seed(tokens)
    w1, s1 = decode_weights(g, experts, 2 * wide, hidden, 32)
    w2, s2 = decode_weights(g, experts, hidden, wide, 64)
    sw, ss = decode_weights(g, 1, hidden, hidden, 128)
    x = torch.randn(tokens, hidden, generator=g).to(torch.bfloat16)
    weight = torch.rand(tokens, top_k, generator=g)
    ids = moe_ref.routing(tokens, top_k, experts, seed=3)
    up, act, act_sf, y, base, out = decode(*(t.to(DEV) for t in (x, ids, weight, w1, s1, w2, s2, sw[0], ss[0])))

    def product(got, xv, w, sf, group, ids):
        want, mag = moe_ref.matvec(xv, moe_ref.e2m1_weights(w, sf, group), ids)
        bound = mag * (xv.shape[1] / 32 + 66) * 2.0 ** -23
        assert ((got.double().cpu() - want).abs() <= (want.abs() + bound) * 2.0 ** -8 + bound).all()
    product(up, x.double(), w1, s1, 32, ids)
    product(y, values(act, act_sf), w2, s2, 64, ids)
    product(base, x.double(), sw[0], ss[0], 128, None)
    want, mag = moe_ref.combine(y.cpu(), np.arange(tokens * top_k).reshape(tokens, top_k), weight, base.cpu())
    near(out, want, mag, top_k, "the layer's output")


def training(x, ids, weight, dout, y, experts, align):
    plan = pq.qcast_expert_sort(ids, experts, align, weight=weight)
    xe, xe_sf = pq.qcast_dispatch_per_token(x, plan)
    q, sf = pq.qcast_per_token(x)
    moved, moved_sf = pq.qcast_dispatch_codes(q, plan, sf)
    out = pq.qcast_combine(y, plan.dest, weight, x)
    back = pq.qcast_combine_backward_per_token(dout, plan, y, weight, want_dy=True)
    return plan, xe, xe_sf, moved, moved_sf, out, back


def same_training(a, b):
    """Equal where the plan says that there is something."""
    live = int(b[0].offsets[-1])
    held = (b[0].source >= 0).nonzero()[:, 0]
    for name in ("dest", "source", "offsets", "counts"):
        assert torch.equal(getattr(a[0], name), getattr(b[0], name)), name
    for i in (1, 3):
        assert np.array_equal(bytes_of(a[i])[:live], bytes_of(b[i])[:live]), i
    for i in (2, 4):
        assert torch.equal(a[i][:live], b[i][:live]), i
    assert torch.equal(a[5], b[5])
    assert np.array_equal(bytes_of(a[6].out)[:live], bytes_of(b[6].out)[:live])
    assert torch.equal(a[6].out_sf[:live], b[6].out_sf[:live]) and torch.equal(a[6].dy[:live], b[6].dy[:live])
    assert torch.equal(a[6].dw, b[6].dw)
    assert torch.equal(a[0].row_weight[held], b[0].row_weight[held])


def training_inputs(seed, tokens, top_k, experts, align, cols):
    g = torch.Generator().manual_seed(seed)
    rows = pq.expert_rows(tokens, top_k, experts, align)
    return (torch.randn(tokens, cols, generator=g).to(torch.bfloat16).to(DEV),
            moe_ref.routing(tokens, top_k, experts + 2, seed=seed).to(DEV),
            torch.rand(tokens, top_k, generator=g).to(DEV),
            torch.randn(tokens, cols, generator=g).to(torch.bfloat16).to(DEV),
            torch.randn(rows, cols, generator=g).to(torch.bfloat16).to(DEV))


# the second: more slots than one workgroup sorts
@pytest.mark.parametrize("tokens,top_k,experts,align,cols", [(67, 4, 16, 16, 512), (2500, 2, 30, 128, 128)])
def test_training_in_two_graphs(tokens, top_k, experts, align, cols):
    """Two captured steps with buffers of their own, replayed in turn with new
    inputs and eager work between: every replay equals the eager step."""
    graphs = []
    for i in range(2):
        static = training_inputs(i, tokens, top_k, experts, align, cols)
        training(*static, experts, align)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = training(*static, experts, align)
        graphs.append((static, graph, out))
    for turn in range(6):
        static, graph, out = graphs[turn % 2]
        fresh = training_inputs(10 + turn, tokens, top_k, experts, align, cols)
        for s, f in zip(static, fresh):
            s.copy_(f)
        graph.replay()
        eager = training(*fresh, experts, align)
        torch.cuda.synchronize()
        same_training(out, eager)


def test_decoding_in_a_graph():
    g = torch.Generator().manual_seed(4)
    experts, tokens, top_k = 12, 3, 4
    w = [t.to(DEV) for t in (*decode_weights(g, experts, 512, 768, 32), *decode_weights(g, experts, 768, 256, 128))]
    sw, ss = decode_weights(g, 1, 768, 768, 128)
    w += [sw[0].to(DEV), ss[0].to(DEV)]
    x = torch.randn(tokens, 768, generator=g).to(torch.bfloat16).to(DEV)
    ids = moe_ref.routing(tokens, top_k, experts).to(DEV)
    weight = torch.rand(tokens, top_k, generator=g).to(DEV)
    decode(x, ids, weight, *w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = decode(x, ids, weight, *w)
    for turn in range(5):
        x.copy_(torch.randn(tokens, 768, generator=g).to(torch.bfloat16))
        ids.copy_(moe_ref.routing(tokens, top_k, experts, seed=turn, repeat=turn % 2 == 1))
        graph.replay()
        eager = decode(x.clone(), ids.clone(), weight, *w)
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert np.array_equal(bytes_of(a), bytes_of(b))


def test_two_threads_on_their_own_streams():
    sizes = [(67, 4, 16, 16, 512), (2500, 2, 30, 128, 128)]
    inputs = [training_inputs(i, *sizes[i]) for i in range(2)]
    alone = [training(*inputs[i], sizes[i][2], sizes[i][3]) for i in range(2)]
    g = torch.Generator().manual_seed(1)
    wts = [t.to(DEV) for t in decode_weights(g, 16, 48, 512, 32)]
    mv = [pq.qcast_matvec_e2m1(i[0][:, :128].repeat(1, 4).contiguous(), *wts, i[1]) for i in inputs]
    torch.cuda.synchronize()
    results, errors = [[], []], []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(8):
                    t = training(*inputs[i], sizes[i][2], sizes[i][3])
                    x = inputs[i][0][:, :128].repeat(1, 4).contiguous()
                    results[i].append((t, pq.qcast_matvec_e2m1(x, *wts, inputs[i][1])))
            s.synchronize()
        except Exception as e:               # reported below, on the main thread
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(timeout=60)
    assert not errors and not any(t.is_alive() for t in threads)
    for i in range(2):
        for t, m in results[i]:
            same_training(t, alone[i])
            assert torch.equal(m, mv[i])


def test_a_stream_that_is_given():
    """stream= alone: outputs and workspaces come from its pool."""
    tokens, top_k, experts, align, cols = 2500, 2, 30, 128, 128
    x, ids, weight, dout, y = training_inputs(5, tokens, top_k, experts, align, cols)
    alone = training(x, ids, weight, dout, y, experts, align)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    plan = pq.qcast_expert_sort(ids, experts, align, weight=weight, stream=s)
    xe, xe_sf = pq.qcast_dispatch_per_token(x, plan, stream=s)
    q, sf = pq.qcast_per_token(x, stream=s)
    moved, moved_sf = pq.qcast_dispatch_codes(q, plan, sf, stream=s)
    out = pq.qcast_combine(y, plan.dest, weight, x, stream=s.cuda_stream)
    back = pq.qcast_combine_backward_per_token(dout, plan, y, weight, want_dy=True, stream=s)
    s.synchronize()
    same_training((plan, xe, xe_sf, moved, moved_sf, out, back), alone)


@pytest.mark.parametrize("tokens,top_k,experts,align,cols", [(1, 1, 1, 1, 128), (67, 4, 16, 16, 640), (130, 3, 7, 128, 2048)])
@pytest.mark.parametrize("flags", [0, 6])
def test_nothing_outside_the_outputs(tokens, top_k, experts, align, cols, flags):
    x, ids, weight, dout, y = training_inputs(6, tokens, top_k, experts, align, cols)
    plan = pq.qcast_expert_sort(ids, experts, align, weight=weight)
    rows = plan.source.shape[0]
    group = 32                                  # packed words need 4 groups
    guard = Guarded(torch.device(DEV))
    shape, dt = pq.sf_layout_shape(rows, cols, group, flags)
    q, sf = pq.qcast_per_token_sf(x, group=group, sf_flags=flags)
    e4 = torch.float8_e4m3fn
    pq.qcast_dispatch_codes(q, plan, sf, flags, out=guard.make((rows, cols), e4), out_sf=guard.make(shape, dt))
    pq.qcast_dispatch_per_token(x, plan, weight, group=group, sf_flags=flags, out=guard.make((rows, cols), e4),
                                out_sf=guard.make(shape, dt))
    pq.qcast_combine_backward_per_token(dout, plan, y, weight, group=group, sf_flags=flags, want_dy=True,
                                        out=guard.make((rows, cols), e4), out_sf=guard.make(shape, dt),
                                        dy=guard.make((rows, cols), torch.bfloat16))
    pq.qcast_combine(y, plan.dest, weight, x, out=guard.make((tokens, cols), torch.bfloat16))
    g = torch.Generator().manual_seed(1)
    w, s = (t.to(DEV) for t in decode_weights(g, experts, 37, cols, 32))
    pq.qcast_matvec_e2m1(x, w, s, ids, out=guard.make((tokens * top_k, 37), torch.bfloat16))
    pq.qcast_matvec_e2m1(x, w[0], s[0], out=guard.make((tokens, 37), torch.bfloat16))
    # the sort's own outputs and workspace, through the C entry point
    i32 = torch.int32
    outs = [guard.make((tokens, top_k), i32), guard.make((rows,), i32), guard.make((experts + 1,), i32),
            guard.make((experts,), i32), guard.make((rows,), torch.float32)]
    rc = pq.load().qcast_expert_sort(ids.data_ptr(), 8, tokens, top_k, experts, 0, align, weight.data_ptr(),
                                     *(t.data_ptr() for t in outs), None,
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    guard.check("experts' operators")
    assert torch.equal(outs[0], plan.dest) and torch.equal(outs[1], plan.source)


def test_the_same_bits_again():
    """Sums in a fixed order, also with another count of compute units."""
    x, ids, weight, dout, y = training_inputs(8, 300, 6, 20, 16, 2048)
    g = torch.Generator().manual_seed(1)
    w, s = (t.to(DEV) for t in decode_weights(g, 20, 200, 2048, 64))

    def run():
        t = training(x, ids, weight, dout, y, 20, 16)
        return t, pq.qcast_matvec_e2m1(x[:9], w, s, ids[:9]), pq.qcast_matvec_e2m1(x[:3], w[0], s[0])
    first = run()
    try:
        for cus in (0, 1, 7, 0):
            pq.qcast_set_num_cus(cus)
            t, a, b = run()
            same_training(t, first[0])
            assert torch.equal(a, first[1]) and torch.equal(b, first[2])
    finally:
        pq.qcast_set_num_cus(0)


def test_rows_past_four_gigabytes():
    """Offsets that do not fit 32 bits: the last rows of a buffer of 4.5 GB, and
    the last of experts whose codes take 4.3."""
    cols, rows, tokens, top_k = 8192, 280000, 4, 2
    y = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    dest = torch.tensor([[rows - 1, 5], [rows - 7, 262144], [262143, -1], [rows, 131072]], dtype=torch.int32)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    for v in dest[(dest >= 0) & (dest < rows)].tolist():
        y[v] = torch.randn(cols, generator=g).to(torch.bfloat16).to(DEV)
    weight = torch.rand(tokens, top_k, generator=g)
    d = dest.to(DEV)
    kept = {int(v): y[int(v)].cpu() for v in dest.reshape(-1) if 0 <= v < rows}
    small = torch.stack(list(kept.values()))
    place = {v: i for i, v in enumerate(kept)}
    d_small = np.array([[place.get(int(v), -1) for v in r] for r in dest], np.int32)
    want, mag = moe_ref.combine(small, d_small, weight, x)
    near(pq.qcast_combine(y, d, weight.to(DEV), x.to(DEV)), want, mag, top_k, "combine")
    # a plan over the same rows: one expert, its run without padding
    source = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    plan = pq.ExpertPlan(d, source, torch.tensor([0, rows], dtype=torch.int32, device=DEV),
                         torch.tensor([rows], dtype=torch.int32, device=DEV), None, 1)
    grad = torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV)
    back = pq.qcast_combine_backward_per_token(x.to(DEV), plan, y, weight.to(DEV), dy=grad, want_dy=True,
                                               want_codes=False)
    dy, dw, mag = moe_ref.combine_grad(x, small, d_small, weight)
    assert ((back.dw.double().cpu() - dw).abs() <= mag * (cols / 64 + 24) * 2.0 ** -24).all()
    for v, i in place.items():
        # one fp32 product, rounded to bf16
        assert ((grad[v].cpu().double() - dy[i]).abs() <= dy[i].abs() * (2.0 ** -8 + 2.0 ** -24) * (1 + 2.0 ** -7)).all()
    q, sf = pq.qcast_per_token(x.to(DEV))
    wide = torch.empty(rows, cols * 2, dtype=torch.uint8, device=DEV).view(torch.bfloat16)
    moved, _ = pq.qcast_dispatch_codes(x.to(DEV), plan, out=wide)
    cast, cast_sf = pq.qcast_dispatch_per_token(x.to(DEV), plan, out=torch.empty(rows, cols, dtype=q.dtype, device=DEV))
    for t in range(tokens):
        for k in range(top_k):
            v = int(dest[t, k])
            if 0 <= v < rows:
                assert torch.equal(moved[v].cpu(), x[t]) and np.array_equal(bytes_of(cast[v]), bytes_of(q[t]))
                assert torch.equal(cast_sf[v], sf[t])
    del y, grad, back, wide, moved, cast
    experts, n, k = 70, 8192, 15104                    # 4.3e9 bytes of codes
    w = torch.zeros(experts, n, k // 2, dtype=torch.uint8, device=DEV)
    ws = torch.zeros(experts, n, k // 32, dtype=torch.float32, device=DEV)
    codes, s = decode_weights(g, 1, n, k, 32)
    w[experts - 1], ws[experts - 1] = codes[0].to(DEV), s[0].to(DEV)
    x = torch.randn(1, k, generator=g).to(torch.bfloat16).to(DEV)
    out = pq.qcast_matvec_e2m1(x, w, ws, torch.tensor([experts - 1, 3], device=DEV))
    want, mag = moe_ref.matvec(x.cpu().double(), moe_ref.e2m1_weights(codes[0], s[0], 32))
    bound = mag * (k / 32 + 66) * 2.0 ** -23
    assert ((out[:1].double().cpu() - want).abs() <= (want.abs() + bound) * 2.0 ** -8 + bound).all()
    assert not out[1].any()


@pytest.mark.parametrize("seed", range(24))
def test_drawn_sizes(seed):
    """Everything at drawn sizes, against the formulas and the oracle's casts
    (which the plain casts are held to elsewhere)."""
    r = np.random.default_rng(seed)
    tokens, top_k = int(r.integers(1, 90)), int(r.integers(1, 10))
    experts, align = int(r.integers(1, 40)), int(2 ** r.integers(0, 8))
    first, total = int(r.integers(0, 5)), experts + int(r.integers(0, 9)) + 5
    fmt = ["e4m3", "e5m2"][r.integers(0, 2)]
    group = int([32, 64, 128][r.integers(0, 3)])
    cols = group * int(r.integers(1, 24))
    g = torch.Generator().manual_seed(seed)
    ids = moe_ref.routing(tokens, top_k, experts, seed=seed, total=total, repeat=bool(r.integers(0, 2)),
                          dtype=[torch.int32, torch.int64][r.integers(0, 2)])
    weight = torch.randn(tokens, top_k, generator=g)
    plan = pq.qcast_expert_sort(ids.to(DEV), experts, align, first, weight.to(DEV))
    dest, source, offsets, counts, rw = moe_ref.sort(ids.numpy(), experts, align, first, weight.numpy())
    for got, want in zip(plan, (dest, source, offsets, counts)):
        assert np.array_equal(got.cpu().numpy(), want)
    live, rows = int(offsets[-1]), source.size
    assert np.array_equal(plan.row_weight.cpu().numpy(), rw)
    x = torch.randn(tokens, cols, generator=g).to(torch.bfloat16)
    q, sf = pq.qcast_per_token(x.to(DEV), fmt, group)
    xe, xe_sf = pq.qcast_dispatch_codes(q, plan, sf)
    xc, xc_sf = pq.qcast_dispatch_per_token(x.to(DEV), plan, None, fmt, group)
    held = (source >= 0)[:live]
    token = source[:live][held] // top_k
    for a, a_sf in ((xe, xe_sf), (xc, xc_sf)):
        assert np.array_equal(bytes_of(a)[:live][held], bytes_of(q)[token]) and not bytes_of(a)[:live][~held].any()
        assert np.array_equal(a_sf.cpu().numpy()[:live][held], sf.cpu().numpy()[token])
    y = torch.randn(rows, cols, generator=g).to(torch.bfloat16)
    want, mag = moe_ref.combine(y, dest, weight, x)
    near(pq.qcast_combine(y.to(DEV), plan.dest, weight.to(DEV), x.to(DEV)), want, mag, top_k, "combine")
    back = pq.qcast_combine_backward_per_token(x.to(DEV), plan, y.to(DEV), weight.to(DEV), fmt, group)
    _, dw, mag = moe_ref.combine_grad(x, y, dest, weight)
    assert ((back.dw.double().cpu() - dw).abs() <= mag * (cols / 64 + 24) * 2.0 ** -24).all()
    n = int(r.integers(1, 70))
    codes, s = decode_weights(g, experts, n, cols, group)
    near_ids = ids if first == 0 else ids - first
    for xin, xsf, xv in ((x, None, x.double()), (q, sf, values(q, sf))):
        got = pq.qcast_matvec_e2m1(xin.to(DEV), codes.to(DEV), s.to(DEV), near_ids.to(DEV), x_sf=xsf,
                                   out_dtype=torch.float32)
        want, mag = moe_ref.matvec(xv, moe_ref.e2m1_weights(codes, s, group), near_ids)
        assert ((got.double().cpu() - want).abs() <= mag * (cols / 32 + 66) * 2.0 ** -23).all()
