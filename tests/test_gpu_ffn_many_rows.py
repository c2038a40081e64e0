"""More rows than fit one launch (2^32 threads): the 8-bit product takes several,
the products grouped by expert refuse them; and so many channels that one row does
not fit."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say
from test_gpu_dense_many_rows import PERIOD, memory_given_back, repeated, repeats, ternary  # noqa: F401

pytestmark = pytest.mark.gpu

M = 2 ** 30 + 1000


@pytest.mark.parametrize("out", [F.BF16, F.F32])
def test_q8(out):
    """Sums below 2^8 and scales of 1 and 2: exact."""
    N, K, s = 8, 16, torch.cuda.current_stream()
    say("many rows, q8", M, N, K)
    ra, w, rs = ternary(1, PERIOD, K).to(torch.int8), ternary(2, N, K).to(torch.int8), ternary(3, PERIOD, 1).float().abs() + 1
    a, scale = repeated(ra, M), repeated(rs, M)
    ws = torch.tensor([1.0, 2.0] * (N // 2), device="cuda")
    D = torch.empty((M, N), dtype=torch.float32 if out == F.F32 else torch.bfloat16, device="cuda")
    with F.Q8Plan(M, N, K, out_dtype=out) as plan:
        plan.run(a, scale, w, ws, None, D, stream=s)
        torch.cuda.synchronize()
    assert repeats(D, (ra.float() @ w.float().t() * rs * ws).to(D.dtype))


@pytest.mark.parametrize("op", [F.GROUPED_NN, F.GROUPED_NT])
def test_grouped(op):
    """Rows of 7: the kernel for any size, 64 rows to a workgroup of 256."""
    N, K, s = 7, 7, torch.cuda.current_stream()
    say("many rows, grouped", M, N, K)
    A, B = torch.ones((M, K), dtype=torch.bfloat16, device="cuda"), torch.ones((1, K, N), dtype=torch.bfloat16, device="cuda")
    C = torch.full((M, N), 5.0, dtype=torch.bfloat16, device="cuda")
    offsets = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    with F.GroupedPlan(M, N, K, 1, op) as plan:
        with pytest.raises(G.GemmRsError) as e:
            plan.run(A, B, offsets, C, stream=s)
        torch.cuda.synchronize()
        assert e.value.code == G.ERR_HIP and bool((C[0] == 5.0).all()) and bool((C[-1] == 5.0).all())
        rows = 2 ** 30 - 4096
        offsets[1] = rows
        plan.run(A, B, offsets, C, rows=rows, stream=s)
        assert plan.status(s)[0] == G.OK
    assert repeats(C[:rows], torch.full((1 << 20, N), 7.0, dtype=torch.bfloat16, device="cuda")) and bool((C[rows:] == 5.0).all())


@pytest.mark.parametrize("N,fit", [(2 ** 27 + 64, True), (2 ** 28 + 64, False)])
def test_q8_of_many_channels(N, fit):
    """32 channels to a workgroup of 512."""
    K, s = 16, torch.cuda.current_stream()
    say("many channels, q8", N)
    a, w = torch.ones((1, K), dtype=torch.int8, device="cuda"), torch.ones((N, K), dtype=torch.int8, device="cuda")
    scale, D = torch.ones(N, device="cuda"), torch.full((1, N), 7.0, device="cuda")
    with F.Q8Plan(1, N, K, out_dtype=F.F32) as plan:
        if fit:
            plan.run(a, scale, w, scale, None, D, stream=s)
        else:
            with pytest.raises(G.GemmRsError) as e:
                plan.run(a, scale, w, scale, None, D, stream=s)
            assert e.value.code == G.ERR_HIP
        torch.cuda.synchronize()
    assert bool((D == (16.0 if fit else 7.0)).all())
