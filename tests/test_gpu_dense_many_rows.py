"""More rows than fit one launch (2^32 threads): operands of odd sizes, whose rows
are copied first, and the products themselves.  Small integers, all exact; rows
repeat with a period that no tile or launch has."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F

from dense_util import BF, F32, LAYOUT
from gpu_util import say

pytestmark = pytest.mark.gpu

PERIOD = 2 ** 20 - 3


@pytest.fixture(autouse=True)
def memory_given_back():
    yield
    torch.cuda.empty_cache()


def ternary(seed, *n):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-1, 2, n, generator=g, device="cuda", dtype=torch.int8).to(BF)


def repeated(rows, m):
    """`rows` again and again, m rows."""
    out = torch.empty((m, rows.shape[1]), dtype=rows.dtype, device="cuda")
    for at in range(0, m, len(rows)):
        out[at:at + len(rows)] = rows[:m - at]
    return out


def repeats(got, rows):
    return all(torch.equal(got[at:at + len(rows)], rows[:len(got) - at]) for at in range(0, len(got), len(rows)))


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_copies_of_more_than_2_to_the_26_rows(layout):
    M, N, K, s = 2 ** 26 + 77, 2, 3, torch.cuda.current_stream()
    say("many rows, copied", M, N, K, layout)
    x, dy, w = ternary(1, M, K), ternary(2, M, N), ternary(3, *((K, N) if layout == "kn" else (N, K)))
    y, dx, dw = torch.empty((M, N), dtype=BF, device="cuda"), torch.empty((M, K), dtype=BF, device="cuda"), torch.empty_like(w, dtype=F32)
    with F.EpiPlan(M, N, K, LAYOUT[layout], backward=1, dw_dtype=F.F32) as plan:
        plan.run(x, w, None, None, y, stream=s)
        plan.backward(dy, x, w, None, None, dx, dw, stream=s)
        torch.cuda.synchronize()
    columns = (w if layout == "kn" else w.t()).float()
    for k in range(N):
        assert torch.equal(y[:, k], sum(x[:, i].float() * columns[i, k] for i in range(K)).to(BF))
    for i in range(K):
        assert torch.equal(dx[:, i], sum(dy[:, k].float() * columns[i, k] for k in range(N)).to(BF))
        for k in range(N):
            got = dw[i, k] if layout == "kn" else dw[k, i]
            assert float(got) == float((x[:, i].float() * dy[:, k].float()).double().sum())


# (too many odd rows for copies: the kernel for any size; whole runs of 8: tiles)
@pytest.mark.parametrize("N,K", [(2, 3), (8, 8)])
def test_products_of_more_than_2_to_the_30_rows(N, K):
    M, s = 2 ** 30 + 1000, torch.cuda.current_stream()
    say("many rows", M, N, K)
    rx, rr, w = ternary(1, PERIOD, K), ternary(2, PERIOD, N), ternary(3, K, N)
    x, r = repeated(rx, M), repeated(rr, M)
    z = torch.empty_like(r)
    want = rx.float() @ w.float()
    with F.EpiPlan(M, N, K, act=F.ACT_RELU, has_residual=1) as plan:
        plan.run(x, w, None, r, r, z, stream=s)
        torch.cuda.synchronize()
    assert repeats(z, want.to(BF)) and repeats(r, (want.relu() + rr.float()).to(BF))


def test_pairs_and_their_gradient_of_more_than_2_to_the_30_rows():
    M, N, K, s = 2 ** 30 + 1000, 8, 8, torch.cuda.current_stream()
    say("many rows, pair", M, N, K)
    rx, wg, wu, rdh = ternary(1, PERIOD, K), ternary(2, K, N), ternary(3, K, N), ternary(4, PERIOD, N)
    x, dh = repeated(rx, M), repeated(rdh, M)
    h, zg, zu, dx = (torch.empty((M, n), dtype=BF, device="cuda") for n in (N, N, N, K))
    g, u, d = rx.float() @ wg.float(), rx.float() @ wu.float(), rdh.float()
    with F.GatedPlan(M, N, K, act=F.ACT_RELU, backward=1) as plan:
        plan.run(x, wg, wu, None, None, h, zg, zu, stream=s)
        torch.cuda.synchronize()
        assert repeats(zg, g.to(BF)) and repeats(zu, u.to(BF)) and repeats(h, (g.relu() * u).to(BF))
        plan.backward(dh, None, wg, wu, zg, zu, zg, zu, dx, stream=s)
        torch.cuda.synchronize()
    dg, du = d * u * (g > 0), d * g.relu()
    assert repeats(zg, dg.to(BF)) and repeats(zu, du.to(BF))
    assert repeats(dx, (dg @ wg.float().t() + du @ wu.float().t()).to(BF))
