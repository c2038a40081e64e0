"""Products grouped by expert (include/gemm_grouped.h) on the GPU against the
fp64 oracle.

Bounds: products of bfloat16 values are exact in floats; a sum of n of them in
floats, in any order, is off by at most n * 2^-24 of the sum of magnitudes; a
bfloat16 output (8 significant bits, to nearest) adds at most 2^-8 of its value.  Inputs from {-1, 0, 1} are exact."""
import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu

OPS = {"NN": F.GROUPED_NN, "NT": F.GROUPED_NT, "TN": F.GROUPED_TN}
NAN = float("nan")


def _mat(g, rows, cols, ld, ternary, scale=1.0, shift=0):
    """Rows in strided storage (gaps hold NaN), starting `shift` elements in."""
    t = torch.full((rows, ld), NAN)
    t[:, :cols] = torch.randint(-1, 2, (rows, cols), generator=g).float() if ternary else torch.randn((rows, cols), generator=g) * scale
    buf = torch.full((rows * ld + shift,), NAN, dtype=torch.bfloat16)
    buf[shift:] = t.bfloat16().view(-1)
    return buf.cuda()[shift:].view(rows, ld)


def _offsets(sizes, first=0):
    return np.concatenate([[first], first + np.cumsum(sizes)]).astype(np.int32)


def _run(op, sizes, N, K, rows=None, first=0, out=F.BF16, accumulate=0, pads=(0, 0, 0), shifts=(0, 0, 0), ternary=False,
         seed=0, capacity=None):
    off = _offsets(sizes, first)
    E = len(sizes)
    rows = int(off[-1]) if rows is None else rows
    M = max(1, rows if capacity is None else capacity)
    g = torch.Generator().manual_seed(seed)
    a_cols, b_cols = K, K if op == "NT" else N
    b_rows = M if op == "TN" else E * (N if op == "NT" else K)
    A = _mat(g, M, a_cols, a_cols + pads[0], ternary, shift=shifts[0])
    B = _mat(g, b_rows, b_cols, b_cols + pads[1], ternary, 1 / np.sqrt(K), shift=shifts[1])
    # rows in no group, and the weights of experts without rows, must not be used
    A[:off[0]], A[off[-1]:] = NAN, NAN
    if op == "TN":
        B[:off[0]], B[off[-1]:] = NAN, NAN
    else:
        per = b_rows // E
        for e in range(E):
            if sizes[e] == 0:
                B[e * per:(e + 1) * per] = NAN
    dt = torch.float32 if out == F.F32 else torch.bfloat16
    c_rows, ldc = (E * K if op == "TN" else M), N + pads[2]
    C = torch.full((c_rows * ldc + shifts[2],), NAN, dtype=dt, device="cuda")[shifts[2]:].view(c_rows, ldc)
    c0 = None
    if accumulate:
        c0 = torch.randint(-3, 4, (c_rows, N), generator=g).to(dt).cuda()
        C[:, :N] = c0
    s = torch.cuda.current_stream()
    with F.GroupedPlan(M, N, K, E, OPS[op], out, accumulate, *(c + p for c, p in zip((a_cols, b_cols, N), pads))) as plan:
        plan.run(A, B, torch.from_numpy(off).cuda(), C, rows=rows, stream=s)
        rc, detail = plan.status(s)
        assert rc == G.OK, detail
    clean = lambda t: np.nan_to_num(t.double().cpu().numpy())  # noqa: E731
    A64, B64 = clean(A[:, :a_cols]), clean(B[:, :b_cols])
    if op != "TN":
        B64 = B64.reshape(E, -1, b_cols)
    want, mag = OF.grouped(op, A64, B64, off, N, K)
    got = C.double().cpu().numpy()
    assert np.isnan(got[:, N:]).all()                      # gaps are not written
    got = got[:, :N].reshape(want.shape)
    if accumulate:
        base = c0.double().cpu().numpy().reshape(want.shape)
        want, mag = want + base, mag + np.abs(base)
    skip = np.isnan(want)
    assert np.array_equal(np.isnan(got), skip)             # rows in no group keep their NaN
    n = (max(sizes) if op == "TN" else K) + 1
    bound = (0.0 if out == F.F32 else 2.0 ** -8) * np.abs(want) + n * 2.0 ** -24 * mag
    if ternary:
        w = torch.from_numpy(np.nan_to_num(want)).to(dt).double().numpy()
        assert np.array_equal(got[~skip], w[~skip])
    bad = np.abs(got - want)[~skip] > bound[~skip]
    assert not bad.any(), int(bad.sum())
    return C


SIZES = [[1], [5], [64], [0, 0, 3, 0], [1, 0, 1, 1, 0, 0, 2], [70, 130, 0, 63, 64, 65], [256, 1, 255, 300], [513, 0, 129],
         [0, 0], [2] * 70, [3, 1] * 40]
DIMS = [(64, 64), (8, 8), (72, 136), (256, 512), (264, 200), (520, 320), (33, 65), (130, 7), (1, 1)]


@pytest.mark.parametrize("op", list(OPS))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "E%d_%d" % (len(s), sum(s)))
def test_group_sizes(op, sizes):
    for N, K in ((128, 192), (136, 72)):
        for ternary in (False, True):
            say("grouped", op, sizes[:6], N, K, ternary)
            _run(op, sizes, N, K, ternary=ternary, seed=N)


@pytest.mark.parametrize("op", list(OPS))
@pytest.mark.parametrize("N,K", DIMS)
def test_dimensions(op, N, K):
    for sizes in ([3, 0, 17], [200, 70, 1, 0, 390]):
        for out in (F.BF16, F.F32):
            say("grouped dims", op, N, K, sizes, out)
            _run(op, sizes, N, K, out=out, seed=N + K)


@pytest.mark.parametrize("op", list(OPS))
def test_large_groups(op):
    """Groups of more rows than the largest tile, where the wide tiles run."""
    for sizes, N, K in (([700, 1300, 0, 530], 768, 1024), ([2100, 1900], 520, 456), ([1500, 20, 0, 0, 900, 1100], 264, 2048)):
        for ternary in (True, False):
            say("grouped large", op, sizes, N, K, ternary)
            _run(op, sizes, N, K, ternary=ternary)


MANY = [90, 0, 141, 80] * 10


@pytest.mark.parametrize("op", list(OPS))
@pytest.mark.parametrize("sizes,N,K", [(MANY, 520, 72), (MANY, 776, 136), (MANY, 1032, 72), (MANY, 1032, 1032), ([3300, 1, 2900], 2056, 520),
                                       ([1100, 0, 37, 900], 264, 72), ([5000], 264, 136), ([700, 0, 301], 257, 131), ([450] * 8, 1288, 1288)],
                         ids=lambda v: str(sum(v)) if isinstance(v, list) else str(v))
def test_every_tile(op, sizes, N, K):
    """Numbers of tiles from a few to several rounds, so that each tile of the
    rules runs, with rows and columns that end inside it."""
    say("grouped tiles", op, len(sizes), sum(sizes), N, K)
    _run(op, sizes, N, K, seed=K)
    _run(op, sizes, N, K, out=F.F32, pads=(8, 16, 24), ternary=True, seed=N)


@pytest.mark.parametrize("op", list(OPS))
@pytest.mark.parametrize("end", range(1, 8))
def test_row_ends_of_every_length(op, end):
    """Rows that end 1..7 elements past a multiple of 8, and rows of fewer than 8."""
    for N, K in ((64 + end, 128 + end), (end, 72 + end), (72 + end, end)):
        say("grouped ends", op, N, K)
        _run(op, [70, 0, 9], N, K, pads=(1, 2, 3))
        _run(op, [70, 0, 9], N, K, out=F.F32, ternary=True)


@pytest.mark.parametrize("op", list(OPS))
def test_rows_outside_groups_strides_and_alignment(op):
    for kw in (dict(first=5, capacity=400), dict(rows=350, capacity=400), dict(first=130, rows=460, capacity=460),
               dict(pads=(8, 16, 24)), dict(pads=(3, 1, 5)), dict(shifts=(1, 0, 0)), dict(shifts=(0, 1, 0)), dict(shifts=(0, 0, 1)),
               dict(shifts=(8, 8, 8))):
        for N, K in ((136, 200), (320, 64)):
            say("grouped layout", op, kw, N, K)
            _run(op, [90, 0, 141, 80], N, K, **kw)


@pytest.mark.parametrize("out", [F.BF16, F.F32])
def test_accumulate(out):
    for sizes, N, K in (([3, 0, 140], 136, 72), ([3, 0, 140], 33, 7), ([900, 0, 600], 512, 256), ([2100, 1900], 264, 136),
                        ([5000], 72, 200)):
        say("grouped accumulate", sizes, N, K)
        _run("TN", sizes, N, K, out=out, accumulate=1)
        _run("TN", sizes, N, K, out=out, accumulate=1, ternary=out == F.F32)


@pytest.mark.parametrize("op", list(OPS))
def test_no_rows(op):
    C = _run(op, [0, 0, 0], 64, 128, rows=0, capacity=10)
    assert C.isnan().all() if op != "TN" else not C.any()
    _run("TN", [0, 0], 64, 128, rows=0, capacity=10, accumulate=1)


@pytest.mark.parametrize("op", list(OPS))
def test_offsets_out_of_range_are_clipped_and_reported(op):
    """Decreasing, negative and too large offsets: nothing outside C is written,
    the status names an expert, and the next run is right."""
    N, K, M, E = 64, 64, 300, 3
    A = torch.ones((M, K), dtype=torch.bfloat16, device="cuda")
    B = torch.ones((M if op == "TN" else E * 64, 64), dtype=torch.bfloat16, device="cuda")
    rows_c = E * K if op == "TN" else M
    guard = torch.full((rows_c + 128, N), NAN, dtype=torch.bfloat16, device="cuda")
    C = guard[64:64 + rows_c]
    s = torch.cuda.current_stream()
    with F.GroupedPlan(M, N, K, E, OPS[op]) as plan:
        for off in ([0, 200, 100, 300], [-5, 100, 200, 300], [0, 100, 200, 2**31 - 1], [400, 500, 600, 700]):
            say("grouped bad offsets", op, off)
            plan.run(A, B, torch.tensor(off, dtype=torch.int32).cuda(), C, stream=s)
            rc, detail = plan.status(s)
            assert rc == G.ERR_PROTOCOL and detail[0] == G.ERR_PROTOCOL and 0 <= detail[1] < E
            assert detail[2:] == off[detail[1]:detail[1] + 2]
            assert guard[:64].isnan().all() and guard[64 + rows_c:].isnan().all()
            assert plan.status(s)[0] == G.OK
        plan.run(A, B, torch.tensor([0, 100, 200, 300], dtype=torch.int32).cuda(), C, stream=s)
        assert plan.status(s)[0] == G.OK
        assert bool((C == (100 if op == "TN" else 64)).all())


def test_gradients_against_differences():
    """dx and dW of sum(g * y) against central differences of the product, all
    exact: inputs are small integers, the step is 1 and the product is linear."""
    sizes, N, K, E = [9, 0, 30, 2], 72, 40, 4
    off = torch.from_numpy(_offsets(sizes)).cuda()
    M = sum(sizes)
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randint(-1, 2, s, generator=g).bfloat16().cuda()  # noqa: E731
    x, w, dy, vx, vw = r(M, K), r(E, K, N), r(M, N), r(M, K), r(E, K, N)
    s = torch.cuda.current_stream()
    y = torch.empty((M, N), device="cuda")
    dx, dw = torch.empty((M, K), device="cuda"), torch.empty((E, K, N), device="cuda")
    with F.GroupedPlan(M, N, K, E, F.GROUPED_NN, F.F32) as nn, F.GroupedPlan(M, K, N, E, F.GROUPED_NT, F.F32) as nt, \
            F.GroupedPlan(M, N, K, E, F.GROUPED_TN, F.F32) as tn:
        def loss(a, b):
            nn.run(a, b, off, y, stream=s)
            return float((dy.double() * y.double()).sum())
        nt.run(dy, w, off, dx, stream=s)
        tn.run(x, dy, off, dw, stream=s)
        torch.cuda.synchronize()
        assert loss(x + vx, w) - loss(x - vx, w) == 2 * float((dx.double() * vx.double()).sum())
        assert loss(x, w + vw) - loss(x, w - vw) == 2 * float((dw.double() * vw.double()).sum())


def test_refusals():
    lib = F._library()
    t = torch.zeros(8192, device="cuda")
    p = t.data_ptr()
    with F.GroupedPlan(8, 16, 16, 2, F.GROUPED_NN) as plan:
        ok = [p, p, p, p]
        for i in range(4):
            assert lib.gemm_grouped_run(plan.handle, *(ok[:i] + [None] + ok[i + 1:]), 8, None) == G.ERR_INVALID_ARG
            assert lib.gemm_grouped_run(plan.handle, *(ok[:i] + [p + 1] + ok[i + 1:]), 8, None) == G.ERR_INVALID_ARG
        for rows in (-1, 9):
            assert lib.gemm_grouped_run(plan.handle, *ok, rows, None) == G.ERR_INVALID_ARG
        assert lib.gemm_grouped_run(plan.handle, *ok, 0, None) == G.OK


def test_another_stream_and_graph_replays():
    g = torch.Generator().manual_seed(4)
    E, N, K = 5, 264, 328
    side = torch.cuda.Stream()
    for sizes in ([2, 0, 1, 4, 1], [300, 0, 700, 40, 513]):
        M = sum(sizes)
        x, w = torch.randn((M, K), generator=g).bfloat16().cuda(), torch.randn((E, K, N), generator=g).bfloat16().cuda()
        off = torch.from_numpy(_offsets(sizes)).cuda()
        y, dw = torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((E, K, N), device="cuda")
        with F.GroupedPlan(M, N, K, E, F.GROUPED_NN) as nn, F.GroupedPlan(M, N, K, E, F.GROUPED_TN, F.F32) as tn:
            def passes(st):
                nn.run(x, w, off, y, stream=st)
                tn.run(x, y, off, dw, stream=st)
            torch.cuda.synchronize()
            passes(side)
            torch.cuda.synchronize()
            want = y.clone(), dw.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                passes(side)
            for _ in range(3):
                y.fill_(NAN)
                dw.fill_(NAN)
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(y, want[0]) and torch.equal(dw, want[1])
                passes(torch.cuda.current_stream())
                torch.cuda.synchronize()
                assert nn.status(torch.cuda.current_stream())[0] == G.OK
            del graph
