"""Arguments that the binding turns away before it allocates for them or hands
them to a C int that does not hold them."""
import pytest
import torch

import precision_quantization_amd as pq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("bad", [dict(experts=4, align=(1 << 32) + 16), dict(experts=4, align=-(1 << 32) + 16),
                                 dict(experts=4, align=2048), dict(experts=1 << 40), dict(experts=(1 << 64) + 4)])
def test_sort(bad):
    ids = torch.zeros(4, 2, dtype=torch.int64, device=DEV)
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.max_memory_allocated()
    with pytest.raises(pq.QcastError):
        pq.qcast_expert_sort(ids, **bad)
    assert torch.cuda.max_memory_allocated() == before
