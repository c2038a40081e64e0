"""Offsets tensors that are not int32 are refused before anything is enqueued."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

pytestmark = pytest.mark.gpu


def test_offsets_of_another_type_are_refused():
    x, w = torch.ones((6, 8), device="cuda").bfloat16(), torch.ones((2, 8, 8), device="cuda").bfloat16()
    y = torch.full((6, 8), 7.0, device="cuda").bfloat16()
    off = torch.tensor([0, 2, 6], device="cuda")          # int64
    s = torch.cuda.current_stream()
    with F.GroupedPlan(6, 8, 8, 2, F.GROUPED_NN) as plan:
        for bad in (off, off.float(), off.int()[:2], off.int().cpu(), torch.zeros(6, dtype=torch.int32, device="cuda")[::2]):
            with pytest.raises(G.GemmRsError):
                plan.run(x, w, bad, y, stream=s)
        torch.cuda.synchronize()
        assert bool((y == 7.0).all())
        plan.run(x, w, off.int(), y, stream=s)
        assert plan.status(s)[0] == G.OK and bool((y == 8.0).all())
