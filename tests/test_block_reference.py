"""The 64-bit formulas that the GPU tests of the checkpoint and norm operators
compare with, against autograd and against central differences."""
import pytest
import torch

import block_ref as br


@pytest.mark.parametrize("clamp", [0.0, 1.5])
def test_swiglu_gradient_against_autograd(clamp):
    g = torch.Generator().manual_seed(1)
    h = torch.randn(5, 24, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(5, generator=g, dtype=torch.float64, requires_grad=True)
    dv = torch.randn(5, 12, generator=g, dtype=torch.float64)
    c = clamp if clamp else float("inf")
    gate, up = h[:, :12].clamp(max=c), h[:, 12:].clamp(-c, c)
    v = torch.nn.functional.silu(gate) * up * w[:, None]
    (v * dv).sum().backward()
    d, v2, dw = br.swiglu_grad(h.detach(), dv, w.detach(), clamp)
    assert torch.allclose(d, h.grad, atol=1e-12) and torch.allclose(v2, v.detach(), atol=1e-12)
    assert torch.allclose(dw, w.grad, atol=1e-12)


@pytest.mark.parametrize("kind", [None, "channel", "token", "full"])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gradient_against_autograd_and_differences(kind, post):
    g = torch.Generator().manual_seed(2)
    rows, cols, alpha, offset = 3, 10, 0.7, 1.0

    def rand(*s):
        return torch.randn(*s, generator=g, dtype=torch.float64)

    v = dict(h=rand(rows, cols), y=rand(rows, cols), w_pre=rand(cols) * 0.1,
             w_post=rand(cols) * 0.1 if post else None,
             gate={None: None, "channel": rand(cols), "token": rand(rows),
                   "full": rand(rows, cols)}[kind])
    dx, dh_in = rand(rows, cols), rand(rows, cols)

    def loss(v):
        f = br.norm_forward(v["h"], v["w_pre"], v["y"], v["w_post"], v["gate"], alpha, offset)
        return (f["x"] * dx).sum() + (f["h"] * dh_in).sum()

    leaves = {k: t.clone().requires_grad_() for k, t in v.items() if t is not None}
    loss({k: leaves.get(k) for k in v}).backward()
    f = br.norm_forward(v["h"], v["w_pre"], v["y"], v["w_post"], v["gate"], alpha, offset)
    b = br.norm_backward(dx, dh_in, f["h"], f["r2"], v["w_pre"], v["y"], f["r1"], v["w_post"],
                         v["gate"], alpha, offset, kind)
    pairs = dict(h="dh", y="dy", w_pre="dw_pre", w_post="dw_post", gate="dgate")
    for k, leaf in leaves.items():
        assert torch.allclose(leaf.grad, b[pairs[k]], atol=1e-7), k
    # central differences in a random direction of each input
    for k, leaf in leaves.items():
        step = rand(*leaf.shape)
        e = 1e-5
        hi = loss({**v, k: v[k] + e * step})
        lo = loss({**v, k: v[k] - e * step})
        assert abs((hi - lo) / (2 * e) - (b[pairs[k]] * step).sum()) < 1e-5, k
