"""Every kernel of the FFN operators' rules at small sizes that reach it
(ffn_cases.py), against the same oracles and bounds as the operators' own tests;
and the block norm's shapes for long rows and many of them."""
import numpy as np
import pytest
import torch

import ffn_cases as C
import test_gpu_ffn_grouped as grouped
import test_gpu_ffn_norm as norm
import test_gpu_ffn_q8 as q8
from tensor_gemm_reduce_lds_amd import ffn as F

from gpu_util import say

pytestmark = pytest.mark.gpu

_id = lambda v: str(v) if not isinstance(v, list) else "E%d_%d" % (len(v), sum(v))  # noqa: E731


@pytest.mark.parametrize("choice,M,N,K", C.Q8, ids=_id)
def test_q8(choice, M, N, K):
    say("q8", choice, M, N, K)
    q8._product(M, N, K, F.BF16, seed=M)
    q8._product(M, N, K, F.F32, bias=True, ldd=N + 3, seed=N)


@pytest.mark.parametrize("dtype", [F.BF16, F.F32])
@pytest.mark.parametrize("choice,rows,cols", C.QUANT, ids=_id)
def test_quantize(choice, rows, cols, dtype):
    say("quantize", choice, rows, cols)
    q8.test_quantize_equals_the_stated_float_steps(dtype, rows, cols, 0, 0)
    q8.test_quantize_equals_the_stated_float_steps(dtype, rows, cols, cols + 3, (cols + 15) // 16 * 16 + 1)


@pytest.mark.parametrize("op", ["NN", "NT"])
@pytest.mark.parametrize("choice,sizes,N,K", C.ROWS, ids=_id)
def test_grouped_rows(choice, sizes, N, K, op):
    say("grouped", op, choice, len(sizes), N, K)
    grouped._run(op, sizes, N, K, seed=N)
    grouped._run(op, sizes, N, K, out=F.F32, ternary=True, seed=K)


@pytest.mark.parametrize("out", [F.BF16, F.F32])
@pytest.mark.parametrize("accumulate", [0, 1])
@pytest.mark.parametrize("large,split,sizes,N,K", C.TN, ids=_id)
def test_weight_gradients(large, split, sizes, N, K, accumulate, out):
    say("grouped TN", large, split, len(sizes), N, K, accumulate, out)
    grouped._run("TN", sizes, N, K, out=out, accumulate=accumulate, seed=N)


@pytest.mark.parametrize("types", [norm.TYPES[0], norm.TYPES[3]], ids=["bb", "ff"])
@pytest.mark.parametrize("rpg", [0, 3, 100])
@pytest.mark.parametrize("cols", [16384, 9001])
def test_norm_backward_of_many_long_rows(cols, rpg, types):
    """Sums in LDS, over several rows of a workgroup and changes of gate row."""
    say("norm backward long", cols, rpg, types)
    norm._backward(norm.Case(600, cols, *types, rpg=rpg, backward=1, seed=cols + rpg))


@pytest.mark.parametrize("rows,cols", [(300, 8192), (300, 8191), (257, 16384), (600, 1001), (300, 72)])
def test_int8_norm_of_many_rows(rows, cols):
    """As the operator's own test of few rows: every integer the nearest of the
    64-bit u/u_scale up to the float error."""
    say("norm int8", rows, cols)
    c = norm.Case(rows, cols, quant=1, rpg=7, seed=cols)
    x_out = torch.empty_like(c.x)
    q = torch.full((rows, cols), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((rows,), -1.0, device="cuda")
    c.plan.run(c.x, c.y, c.w_post, c.gate, c.w_pre, x_out, q, scale, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    _, want = c.oracle()
    amax = np.abs(want).max(1)
    assert (np.abs(scale.cpu().numpy() - amax / 127) <= 4 * norm.FLOAT * amax / 127).all()
    q = q.cpu().numpy().astype(np.float64)
    assert np.abs(q - want / (amax / 127)[:, None]).max() <= 0.5 + 127 * 4 * norm.FLOAT
    assert (np.abs(q).max(1) == 127).all()

