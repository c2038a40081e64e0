"""Rows so far apart that their offsets pass 32 bits: equal bits to the same
call on tight rows, which the operators' own tests compare with the oracle (the
kernel is chosen by sizes and alignment, so both run the same one)."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu

BF, I8 = torch.bfloat16, torch.int8


class Far:
    """Tight inputs and outputs, and the same in rows `ld` elements apart (all
    bytes past 2^32 for the last ones)."""

    def __init__(self, seed):
        self.g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(self, n, cols, ld, dt=BF, fill=True):
        assert n * ld * torch.empty(0, dtype=dt).element_size() > 2 ** 32
        tight = torch.empty((n, cols), dtype=dt, device="cuda")
        if fill and dt == I8:
            tight.random_(-127, 128, generator=self.g)
        elif fill:
            tight.normal_(generator=self.g)
        far = torch.empty((n, ld), dtype=dt, device="cuda")
        if fill:
            far[:, :cols] = tight
        return tight, far


def _same(pair):
    tight, far = pair
    assert torch.equal(far[:, :tight.shape[1]].contiguous().view(torch.int8), tight.view(torch.int8))


@pytest.mark.parametrize("cols", [72, 515])
def test_norm(cols):
    say("norm far", cols)
    n, ld, f, s = 2100, 2 ** 20, Far(1), torch.cuda.current_stream()
    x, y, dxo, du = (f.rows(n, cols, ld) for _ in range(4))
    xo, u, dx, dy = (f.rows(n, cols, ld, fill=False) for _ in range(4))
    w = torch.ones((2, cols), device="cuda")
    dw = torch.zeros((2, 2, cols), device="cuda")
    lds = {"ld_" + k: ld for k in ("x", "y", "x_out", "u", "dx_out", "du", "dx", "dy")}
    for i, strides in enumerate(({}, lds)):
        with F.BlockNormPlan(n, cols, backward=1, **strides) as plan:
            plan.run(x[i], y[i], w[0], None, w[1], xo[i], u[i], stream=s)
            plan.backward(dxo[i], du[i], xo[i], y[i], w[0], None, w[1], dx[i], dy[i], dw[i][0], None, dw[i][1], stream=s)
            torch.cuda.synchronize()
    for p in (xo, u, dx, dy):
        _same(p)
    assert torch.equal(dw[0], dw[1]) and bool(dw.any())


@pytest.mark.parametrize("M", [1100, 40])
def test_q8(M):
    say("q8 far", M)
    N, K, f, s = 1100, 80, Far(2), torch.cuda.current_stream()
    ld = 2 ** 22
    a = f.rows(M, K, ld, I8) if M > 64 else (f.rows(1100, K, ld, I8)[0][:M],) * 2
    w = f.rows(N, K, ld, I8)
    d = f.rows(1100, N, 2 ** 21, fill=False)
    sa, sw = torch.rand(M, device="cuda", generator=f.g), torch.rand(N, device="cuda", generator=f.g)
    for i in (0, 1):
        with F.Q8Plan(M, N, K, lda=ld * i if M > 64 else 0, ldw=ld * i, ldd=2 ** 21 * i) as plan:
            plan.run(a[i], sa, w[i], sw, None, d[i], stream=s)
            torch.cuda.synchronize()
    _same((d[0][:M], d[1][:M]))


def test_quantize():
    say("quantize far")
    n, cols, f, s = 2100, 72, Far(3), torch.cuda.current_stream()
    x, q = f.rows(n, cols, 2 ** 20), f.rows(n, 80, 2 ** 21, I8, fill=False)
    scale = torch.zeros((2, n), device="cuda")
    for i in (0, 1):
        F.q8_quantize(x[i], q[i], scale[i], n, cols, ldx=2 ** 20 * i, ldq=2 ** 21 * i, stream=s)
    torch.cuda.synchronize()
    _same(q)
    assert torch.equal(scale[0], scale[1]) and bool(scale.all())


@pytest.mark.parametrize("op", [F.GROUPED_NN, F.GROUPED_NT, F.GROUPED_TN])
@pytest.mark.parametrize("N,K", [(72, 1032), (71, 1031)])
def test_grouped(op, N, K):
    say("grouped far", op, N, K)
    f, s, E, sizes, ld = Far(4), torch.cuda.current_stream(), 3, [900, 0, 200], 2 ** 21
    n, tn = sum(sizes), op == F.GROUPED_TN
    off = torch.tensor([0, 900, 900, 1100], dtype=torch.int32, device="cuda")
    if op == F.GROUPED_NT:
        N, K = K, N                                  # many rows of B in this form too
    a = f.rows(n, K, ld)
    b = f.rows(n, N, ld) if tn else f.rows(E * (N if op == F.GROUPED_NT else K), K if op == F.GROUPED_NT else N, ld)
    c = f.rows(E * K if tn else n, N, ld, fill=False)
    for i in (0, 1):
        ldb = b[1].shape[1] * i
        with F.GroupedPlan(n, N, K, E, op, lda=ld * i, ldb=ldb, ldc=ld * i) as plan:
            plan.run(a[i], b[i], off, c[i], stream=s)
            assert plan.status(s)[0] == G.OK
    _same(c)
