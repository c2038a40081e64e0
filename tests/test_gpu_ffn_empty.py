"""Calls without rows, with tensors that have none (torch gives those no
address): a rank or an expert layer that received no token makes them."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu

BF, NAN = torch.bfloat16, float("nan")


def _empty(cols, dtype=BF):
    t = torch.empty((0, cols), dtype=dtype, device="cuda")
    assert t.data_ptr() == 0
    return t


@pytest.mark.parametrize("quant", [0, 1])
@pytest.mark.parametrize("rpg", [0, 4])
def test_norm_forward(quant, rpg):
    say("norm without rows", quant, rpg)
    w = torch.ones(64, device="cuda")
    e, gate = _empty(64), _empty(64, torch.float32) if rpg else None
    u, us = (_empty(64, torch.int8), torch.empty(0, device="cuda")) if quant else (e, None)
    s = torch.cuda.current_stream()
    with F.BlockNormPlan(8, 64, rows_per_gate=rpg, quant=quant) as plan:
        plan.run(e, e, w, gate, w, e, u, us, rows=0, stream=s)
        # what has elements is still wanted, what the plan has not is still refused
        for bad in ([(e, e, None, gate, w, e, u, us)] + ([] if quant else [(e, e, w, gate, w, e, u, w)])):
            with pytest.raises(G.GemmRsError):
                plan.run(*bad, rows=0, stream=s)
        with pytest.raises(G.GemmRsError):
            plan.run(e, e, w, gate, w, e, u, us, rows=1, stream=s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("rpg", [0, 4])
def test_norm_backward_zeroes_the_weights_gradients(rpg):
    say("norm backward without rows", rpg)
    w, dw = torch.ones(64, device="cuda"), torch.full((2, 64), NAN, device="cuda")
    e, g = _empty(64), _empty(64, torch.float32) if rpg else None
    s = torch.cuda.current_stream()
    with F.BlockNormPlan(8, 64, rows_per_gate=rpg, backward=1) as plan:
        for i, dxo in enumerate((e, None)):
            dw.fill_(NAN)
            plan.backward(dxo, e, e, e, w, g, w, e, e, dw[0], g, dw[1], rows=0, stream=s)
            torch.cuda.synchronize()
            assert not dw.any() and not dw.isnan().any()
        for a, b in ((None, dw[1]), (dw[0], None)):
            with pytest.raises(G.GemmRsError):
                plan.backward(e, e, e, e, w, g, w, e, e, a, g, b, rows=0, stream=s)
        with pytest.raises(G.GemmRsError):
            plan.backward(e, e, e, e, w, g, w, e, e, dw[0], g, dw[1], rows=1, stream=s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bias", [0, 1])
def test_q8(bias):
    say("q8 without rows", bias)
    q, sq, x, y = _empty(64, torch.int8), torch.empty(0, device="cuda"), _empty(64), _empty(32)
    w, sw = torch.zeros((32, 64), dtype=torch.int8, device="cuda"), torch.ones(32, device="cuda")
    s = torch.cuda.current_stream()
    F.q8_quantize(x, q, sq, 0, 64, stream=s)
    with F.Q8Plan(8, 32, 64, has_bias=bias) as plan:
        b = sw if bias else None
        plan.run(q, sq, w, sw, b, y, rows=0, stream=s)
        for bad in ((None, sw, b), (w, None, b), (w, sw, None if bias else sw)):
            with pytest.raises(G.GemmRsError):
                plan.run(q, sq, *bad, y, rows=0, stream=s)
        with pytest.raises(G.GemmRsError):
            plan.run(q, sq, w, sw, b, y, rows=1, stream=s)
    torch.cuda.synchronize()


@pytest.mark.parametrize("op", [F.GROUPED_NN, F.GROUPED_NT, F.GROUPED_TN])
@pytest.mark.parametrize("N,K", [(64, 128), (33, 7)])
def test_grouped(op, N, K):
    """No rows at all: NN and NT have nothing to write, the weight gradient is
    zeros, or what it was with `accumulate`."""
    say("grouped without rows", op, N, K)
    tn = op == F.GROUPED_TN
    a = _empty(K)
    b = _empty(N) if tn else torch.ones((3, K, N), dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    s = torch.cuda.current_stream()
    for accumulate in ((0, 1) if tn else (0,)):
        with F.GroupedPlan(10, N, K, 3, op, accumulate=accumulate) as plan:
            c = torch.full((3, K, N), 7.0, dtype=BF, device="cuda") if tn else _empty(N)
            plan.run(a, b, off, c, rows=0, stream=s)
            assert plan.status(s)[0] == G.OK
            assert not tn or bool((c == (7.0 if accumulate else 0.0)).all())
            for bad in ((a, b, None, c), (a, b, off, None) if tn else (a, None, off, c)):
                with pytest.raises(G.GemmRsError):
                    plan.run(*bad, rows=0, stream=s)
            with pytest.raises(G.GemmRsError):
                plan.run(a, b, off, c, rows=1, stream=s)
            assert plan.status(s)[0] == G.OK
