"""The 8-bit integer product and the row quantisation (include/gemm_q8.h) on
the GPU.  The integer sums are exact and the float steps after them are
stated by the interface, so float outputs without bias equal the oracle's
float32 steps bit for bit; with a bias the one fused rounding may differ from
the oracle's float64 rounding by one unit; bfloat16 outputs are those floats
rounded once."""
import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu


def _rows(g, n, ld, K, lo=-127, hi=128):
    """int8 rows whose gaps past K hold 127."""
    t = torch.full((n, ld), 127, dtype=torch.int8)
    t[:, :K] = torch.randint(lo, hi, (n, K), generator=g, dtype=torch.int8)
    return t


def _product(M, N, K, out=F.F32, bias=False, lda=0, ldw=0, ldd=0, rows=None, seed=0, extreme=False, offset=0):
    g = torch.Generator().manual_seed(seed)
    lo = -128 if extreme else -127
    a, w = _rows(g, M, lda or K, K, lo), _rows(g, N, ldw or K, K, lo)
    if extreme:
        a[0, :K], w[0, :K] = -128, -128
    sa = torch.rand(M, generator=g) * 0.01 + 1e-3
    sw = torch.rand(N, generator=g) * 0.01 + 1e-3
    b = torch.randn(N, generator=g) if bias else None
    rows = M if rows is None else rows
    dt = torch.float32 if out == F.F32 else torch.bfloat16
    ld = ldd or N
    D = torch.full((M * ld + offset,), float("nan"), dtype=dt, device="cuda")[offset:].view(M, ld)
    with F.Q8Plan(M, N, K, lda, ldw, ldd, out, int(bias)) as plan:
        plan.run(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), None if b is None else b.cuda(), D, rows=rows,
                 stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
    got = D.float().cpu().numpy()
    assert np.isnan(got[rows:]).all() and np.isnan(got[:, N:]).all()   # nothing else is written
    got = got[:rows, :N]
    acc = a[:rows, :K].numpy().astype(np.int64) @ w[:, :K].numpy().astype(np.int64).T
    v = acc.astype(np.float32) * sa[:rows].numpy()[:, None]
    if bias:
        f = (v.astype(np.float64) * sw.numpy() + b.numpy()).astype(np.float32)
        if out == F.F32:
            assert (np.abs(got - f) <= np.spacing(np.abs(f))).all()
            return
        v = f
    else:
        v = v * sw.numpy()
    if out == F.F32:
        assert np.array_equal(got, v)
    else:
        want = torch.from_numpy(v).bfloat16().float().numpy()
        tol = np.abs(want) * 2.0 ** -7 if bias else 0.0      # a one-unit float difference may cross a rounding
        assert (np.abs(got - want) <= tol).all() and (got != want).mean() <= (1e-4 if bias else 0.0)


SIZES = [(1, 1, 16), (1, 64, 128), (1, 4096, 512), (1, 1000, 3584), (2, 17, 48), (3, 333, 1040), (7, 8192, 256),
         (16, 512, 8192), (17, 130, 528), (31, 65, 144), (33, 257, 4096), (64, 3584, 1792), (65, 640, 272),
         (100, 200, 80), (128, 128, 128), (129, 255, 112), (256, 512, 640), (300, 4099, 304), (513, 1030, 1040),
         (1000, 777, 2064), (2049, 1031, 400)]


@pytest.mark.parametrize("out,bias", [(F.F32, False), (F.BF16, False), (F.F32, True), (F.BF16, True)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product(M, N, K, out, bias):
    say("q8", M, N, K, out, bias)
    _product(M, N, K, out, bias, seed=M + N + K)


@pytest.mark.parametrize("M,N", [(65, 264), (3300, 264), (6000, 264), (700, 6152), (6000, 1034), (2100, 4104)])
def test_every_tile(M, N):
    """Numbers of tiles from a few to several rounds, so that each tile of the
    rule runs, with rows and columns that end inside it."""
    say("q8 tiles", M, N)
    _product(M, N, 80, F.BF16, seed=M)
    _product(M, N, 80, F.F32, ldd=N + 3, seed=N)


@pytest.mark.parametrize("end", range(1, 8))
def test_row_ends_of_every_length(end):
    for M in (3, 70):
        for N in (64 + end, end):
            say("q8 ends", M, N)
            _product(M, N, 48, F.BF16, seed=N)
            _product(M, N, 48, F.F32, bias=True, seed=N)


@pytest.mark.parametrize("M", [1, 5, 40, 200, 700])
def test_strides_fewer_rows_and_unaligned_output(M):
    say("q8 strides", M)
    _product(M, 300, 176, F.BF16, lda=208, ldw=192, ldd=301, rows=max(1, M - 3))
    _product(M, 304, 176, F.F32, bias=True, lda=176, ldw=1024, ldd=304, offset=1)
    _product(M, 304, 176, F.BF16, ldd=312, offset=3)


@pytest.mark.parametrize("M", [1, 20, 70, 400])
def test_largest_sums_are_exact(M):
    """K just below 2^17 with rows of -128: the sum 131056 * 16384 is the
    largest the interface admits and just fits 32 bits."""
    say("q8 largest", M)
    _product(M, 130, 2**17 - 16, F.F32, extreme=True)


def test_non_finite_scales():
    M, N, K = 40, 96, 64
    g = torch.Generator().manual_seed(0)
    a, w = _rows(g, M, K, K).cuda(), _rows(g, N, K, K).cuda()
    sa, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    sa[3], sa[5] = float("nan"), 0.0
    D = torch.empty((M, N), device="cuda")
    with F.Q8Plan(M, N, K, out_dtype=F.F32) as plan:
        plan.run(a, sa, w, sw, None, D, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
    assert D[3].isnan().all() and not D[5].any() and D[[0, 1, 2, 4, 6]].isfinite().all()


@pytest.mark.parametrize("dtype", [F.BF16, F.F32])
@pytest.mark.parametrize("rows,cols,ldx,ldq", [(1, 1, 0, 0), (3, 16, 0, 0), (4, 8, 24, 32), (5, 1000, 0, 0), (2, 1000, 1001, 1024),
                                               (7, 3584, 0, 0), (3, 8192, 8200, 0), (2, 8191, 0, 0), (2, 16400, 0, 0),
                                               (1, 131071, 0, 0), (300, 40, 0, 48)])
def test_quantize_equals_the_stated_float_steps(dtype, rows, cols, ldx, ldq):
    say("quantize", rows, cols)
    g = torch.Generator().manual_seed(cols)
    t = torch.float32 if dtype == F.F32 else torch.bfloat16
    x = torch.full((rows, ldx or cols), float("nan"), dtype=t)
    x[:, :cols] = (torch.randn((rows, cols), generator=g) * torch.rand((rows, 1), generator=g) * 10).to(t)
    if rows > 2:
        x[1, :cols] = 0.0
        x[2, cols // 2] = float("inf") if cols % 3 else float("nan")
    padded = (cols + 15) // 16 * 16
    q = torch.full((rows, ldq or padded), 77, dtype=torch.int8, device="cuda")
    s = torch.full((rows,), -1.0, device="cuda")
    F.q8_quantize(x.cuda(), q, s, rows, cols, dtype, ldx, ldq, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    want_q, want_s = OF.quantize_rows(x[:, :cols].float().numpy())
    q, s = q.cpu().numpy(), s.cpu().numpy()
    assert np.array_equal(s, want_s, equal_nan=True)
    assert np.array_equal(q[:, :cols], want_q)
    assert not q[:, cols:padded].any() and (q[:, padded:] == 77).all()


@pytest.mark.parametrize("dtype", [F.BF16, F.F32])
@pytest.mark.parametrize("end", range(1, 8))
def test_quantize_row_ends_of_every_length(dtype, end):
    for cols in (end, 8 + end, 512 + end, 2048 + end, 16384 + end):
        say("quantize ends", cols)
        test_quantize_equals_the_stated_float_steps(dtype, 4, cols, cols + 1, 0)


def test_quantize_tiny_rows():
    """Rows whose largest magnitude is below 127 / FLT_MAX still fill the range."""
    x = torch.tensor([[1e-38, -5e-39, 0.0, 2e-39], [2.0 ** -133, 0, 0, -(2.0 ** -133)]])
    q = torch.empty((2, 16), dtype=torch.int8, device="cuda")
    s = torch.empty(2, device="cuda")
    F.q8_quantize(x.cuda(), q, s, 2, 4, F.F32, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert q.cpu()[:, :4].tolist() == [[127, -64, 0, 25], [127, 0, 0, -127]]


def test_refusals_and_empty_calls():
    lib = F._library()
    t = torch.zeros(8192, device="cuda")
    p = t.data_ptr()
    with F.Q8Plan(4, 32, 64) as plan, F.Q8Plan(4, 32, 64, has_bias=1) as biased:
        ok = [p, p, p, p, None, p]
        for i in (0, 1, 2, 3, 5):
            assert lib.gemm_q8_run(plan.handle, *(ok[:i] + [None] + ok[i + 1:]), 4, None) == G.ERR_INVALID_ARG
            assert lib.gemm_q8_run(plan.handle, *(ok[:i] + [p + 1] + ok[i + 1:]), 4, None) == G.ERR_INVALID_ARG
        assert lib.gemm_q8_run(plan.handle, p + 8, p, p, p, None, p, 4, None) == G.ERR_INVALID_ARG
        assert lib.gemm_q8_run(plan.handle, p, p, p, p, p, p, 4, None) == G.ERR_INVALID_ARG
        assert lib.gemm_q8_run(biased.handle, *ok, 4, None) == G.ERR_INVALID_ARG
        for rows in (-1, 5):
            assert lib.gemm_q8_run(plan.handle, *ok, rows, None) == G.ERR_INVALID_ARG
        assert lib.gemm_q8_run(plan.handle, *ok, 0, None) == G.OK
    torch.cuda.synchronize()
    assert not t.any()


def test_graph_replays_match_eager():
    g = torch.Generator().manual_seed(2)
    side = torch.cuda.Stream()
    for M in (1, 48, 600):
        N, K = 520, 1040
        x = torch.randn((M, K), generator=g).bfloat16().cuda()
        w, sw = _rows(g, N, K, K).cuda(), torch.rand(N, generator=g).cuda()
        q, s = torch.empty((M, K), dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda")
        D = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        with F.Q8Plan(M, N, K) as plan:
            def passes(st):
                F.q8_quantize(x, q, s, M, K, stream=st)
                plan.run(q, s, w, sw, None, D, stream=st)
            passes(torch.cuda.current_stream())
            torch.cuda.synchronize()
            want = D.clone()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=side):
                passes(side)
            for _ in range(3):
                D.fill_(-1)
                q.fill_(0)
                torch.cuda.synchronize()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(D, want)
                passes(torch.cuda.current_stream())
                torch.cuda.synchronize()
            del graph
