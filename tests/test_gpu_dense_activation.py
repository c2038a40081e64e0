"""The dense products' activations and slopes over all of their range, tails too,
against 64 bits: z comes as the bias of a product of zeros, the slope leaves as the
bias' gradient of one row, both in floats.

Bounds, u = 2^-24.  An exponential's argument t (of its natural form) is rounded by
at most 6.5 u t (gelu_tanh: five operations and three constants of half a u each;
the others fewer), the exponential, the sum, the reciprocal and the last product by
2 u each: 6.5 u t + 8 u of the value, which passes ACT_ERROR from t = 25 on.  There
the value is below 10 exp(-t), so what is over stays below the largest of (6.5 u t
- 1e-5) 10 exp(-t), 1e-17 (t = 26).  Values that are zero because the sigmoid or
the exponential is below the smallest float are below 100 * 2^-126.  A slope has
one term z (1 - s) f with 1 - s off by 2 u: largest for gelu_tanh at z = 5, where f =
c (1 + 3 k z^2) is 7, and 2 u * 35 is 4e-6; the others are below 2 u * 90 = 1.1e-5
only in silu's z (1 - s) at z = 90, where s is 1 and the term 0: s differs from 1 up
to z = 17.4, 2 u * 17.4 is 2e-6."""
import math

import pytest
import torch

from oracle import dense as OD
from tensor_gemm_reduce_lds_amd import ffn as F

from dense_util import ACT, BF, F32
from gpu_util import say

pytestmark = pytest.mark.gpu

TINY = 1e-17
INF = float("inf")


def exact(act, z):
    """act(z) and act'(z) in 64 bits; the tanh as the sigmoid of twice its argument, which does not cancel."""
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        t = c * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(t)
        return z * s, s + z * s * torch.sigmoid(-t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * torch.sigmoid(-z)
    return OD.act(act, z), OD.slope(act, z)


def numbers():
    far = torch.logspace(-30, 30, 4001)
    return torch.cat((torch.linspace(-120, 120, 48001), torch.linspace(-16, 16, 64001), far, -far, torch.tensor([0.0, -0.0, 3e38, -3e38]))).cuda()


def value_and_slope(act, z):
    n, s = z.numel(), torch.cuda.current_stream()
    x, w = torch.zeros((1, 8), dtype=BF, device="cuda"), torch.zeros((8, n), dtype=BF, device="cuda")
    y, dz, slope = torch.empty((1, n), device="cuda"), torch.empty((1, n), dtype=BF, device="cuda"), torch.empty(n, device="cuda")
    with F.EpiPlan(1, n, 8, act=ACT[act], out_dtype=F.F32, has_bias=1, backward=1, z_dtype=F.F32) as plan:
        plan.run(x, w, z, None, y, stream=s)
        plan.backward(torch.ones((1, n), device="cuda"), x, w, z.view(1, n) if act != "none" else None, dz, None, None, slope, stream=s)
        torch.cuda.synchronize()
    return y[0], slope


@pytest.mark.parametrize("act", OD.ACTS)
def test_values_and_slopes(act):
    say("activation", act)
    z = numbers()
    y, slope = value_and_slope(act, z)
    want, want_slope = exact(act, z.double())
    off = (y.double() - want).abs() - OD.ACT_ERROR * want.abs()
    assert bool((off <= TINY).all()), (act, float(off.max()), float(z[off.argmax()]))
    off = (slope.double() - want_slope).abs()
    assert bool((off <= OD.ACT_ERROR).all()), (act, float(off.max()), float(z[off.argmax()]))


@pytest.mark.parametrize("act", OD.ACTS)
def test_a_pairs_values_and_slopes(act):
    """The gradients of the biases of one row with dh = z_up = 1: slope and value."""
    z = numbers()
    n, s = z.numel(), torch.cuda.current_stream()
    dh, up = torch.ones((1, n), dtype=BF, device="cuda"), torch.ones((1, n), device="cuda")
    dz, db = torch.empty((2, 1, n), dtype=BF, device="cuda"), torch.empty((2, n), device="cuda")
    with F.GatedPlan(1, n, 8, act=ACT[act], has_bias=1, backward=1, z_dtype=F.F32) as plan:
        plan.backward(dh, None, None, None, z.view(1, n), up, dz[0], dz[1], None, None, None, db[0], db[1], stream=s)
        torch.cuda.synchronize()
    y, slope = value_and_slope(act, z)
    assert torch.equal(db[0], slope) and torch.equal(db[1], y)
    assert torch.equal(dz[0, 0], slope.to(BF)) and torch.equal(dz[1, 0], y.to(BF))


def test_infinities_and_nan():
    z = torch.tensor([INF, float("nan")] * 4, device="cuda")
    for act in OD.ACTS:
        y, _ = value_and_slope(act, z)
        assert bool((y[::2] == INF).all()) and bool(y[1::2].isnan().all()), act
    y, slope = value_and_slope("relu", -z)
    assert bool((y[::2] == 0).all()) and bool((slope[::2] == 0).all())
