"""Adding to weight gradients of experts without rows leaves every bit."""
import pytest
import torch

import ffn_cases as C
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [F.BF16, F.F32])
@pytest.mark.parametrize("large,split,sizes,N,K", [c for c in C.TN if 0 in c[2]] + [(False, False, [3, 0, 140], 33, 7)],
                         ids=lambda v: str(v) if not isinstance(v, list) else "E%d_%d" % (len(v), sum(v)))
def test_experts_without_rows(large, split, sizes, N, K, out):
    say("accumulate, no rows", large, split, len(sizes), N, K)
    g = torch.Generator(device="cuda").manual_seed(N)
    M, E = sum(sizes), len(sizes)
    x, dy = (torch.randn((M, c), generator=g, device="cuda").bfloat16() for c in (K, N))
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    c = torch.full((E, K, N), -0.0, dtype=torch.float32 if out == F.F32 else torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream()
    with F.GroupedPlan(M, N, K, E, F.GROUPED_TN, out, accumulate=1) as plan:
        plan.run(x, dy, off, c, stream=s)
        assert plan.status(s)[0] == G.OK
    empty = torch.tensor([n == 0 for n in sizes], device="cuda")
    assert not c[empty].any() and bool(torch.signbit(c[empty]).all())
    assert bool(c[~empty].any())
