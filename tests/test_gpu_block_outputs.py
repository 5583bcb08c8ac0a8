"""The SwiGLU backward's optional outputs one by one through the C ABI: each
has the bits that the call with all of them gives."""
import pytest
import torch

import block_ref as br
import precision_quantization_amd as pq
from precision_quantization_amd import _lib, workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("want", ["dh_t", "v_t", "dw"])
@pytest.mark.parametrize("cols", [128, 384])
def test_one_optional_output(want, cols):
    dev, rows = torch.device("cuda:0"), 200
    h, dv, w = workloads.swiglu_grad(seed=5, rows=rows, cols=cols)
    codes, scales, _ = br.stored(h, "e4m3")
    codes, scales, dv, w = (t.to(dev) for t in (codes, scales, dv, w))
    full = pq.qcast_swiglu_backward_checkpoint(codes, scales, dv, w)
    out = {k: torch.zeros_like(v) for k, v in full._asdict().items()}
    ws = torch.zeros(rows * (cols // 128), device=dev)

    def p(name):
        return out[name].data_ptr() if name in ("dh", "dh_sf", want, want + "_sf") else None

    assert _lib.load().qcast_swiglu_backward_checkpoint(
        codes.data_ptr(), scales.data_ptr(), dv.data_ptr(), rows, cols, w.data_ptr(), 1, 1, 128, 0.0, 0, 0.0, p("dh"),
        p("dh_sf"), p("dh_t"), p("dh_t_sf"), p("v_t"), p("v_t_sf"), p("dw"), ws.data_ptr(),
        torch.cuda.current_stream(dev).cuda_stream) == 0
    torch.cuda.synchronize()
    for k in ("dh", "dh_sf", want) + (() if want == "dw" else (want + "_sf",)):
        assert torch.equal(out[k].view(torch.uint8), getattr(full, k).view(torch.uint8)), k
