"""The operators handed to one another, as the FFN sub-layer has them."""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G
from tensor_gemm_reduce_lds_amd import inputs as I

from gpu_util import (check_tolerance, desc_fields, new_out, oracle_kw, out_to_f64, run_checked, say,
                      to_device)

pytestmark = pytest.mark.gpu

FLOAT = 64 * 2.0 ** -24        # a row's floats before the rounding (sums of a few hundred terms per thread tree)


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("extra", [0, 32])
@pytest.mark.parametrize("rows,cols", [(3, 5), (2, 16), (5, 24), (4, 993), (4, 1000), (70, 1001), (6, 1008), (3, 8184), (3, 16377)])
def test_int8_norm_into_the_product(rows, cols, extra):
    """Rows of any length: the norm pads them with zeros, so whatever lies in
    the padding of the weights does not enter the product.  Given the integers
    and scales, the product is exact up to the stated float steps; against the
    64-bit norm, each integer is off by half a unit and the float error of u
    (127 * 4 * FLOAT of a unit)."""
    say("int8 norm, product", rows, cols, extra)
    g = torch.Generator().manual_seed(cols)
    N, K = 40, (cols + 15) // 16 * 16
    x, y = (torch.randn((rows, cols), generator=g).bfloat16().cuda() for _ in range(2))
    w_post, w_pre = (1 + 0.1 * torch.randn((2, cols), generator=g)).cuda()
    w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8)      # (its padding too)
    sw = torch.rand(N, generator=g) * 0.01 + 1e-3
    x_out = torch.empty_like(x)
    q = torch.full((rows, K + extra), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    out = torch.empty((rows, N), device="cuda")
    st = torch.cuda.current_stream()
    with F.BlockNormPlan(rows, cols, quant=1, ld_u=K + extra) as norm, \
            F.Q8Plan(rows, N, K, lda=K + extra, out_dtype=F.F32) as product:
        norm.run(x, y, w_post, None, w_pre, x_out, q, s, stream=st)
        product.run(q, s, w.cuda(), sw.cuda(), None, out, stream=st)
        torch.cuda.synchronize()
    assert not q[:, cols:K].any() and bool((q[:, K:] == 77).all())
    q, s, got = q.cpu().numpy()[:, :K], s.cpu().numpy(), out.cpu().numpy()
    acc = q.astype(np.int64) @ w.numpy().astype(np.int64).T
    assert np.array_equal(got, (acc.astype(np.float32) * s[:, None]) * sw.numpy())
    _, u = OF.norm_forward(_f64(x), _f64(y), _f64(w_post), None, _f64(w_pre))
    wf = w[:, :cols].double().numpy() * sw.double().numpy()[:, None]
    unit = np.abs(u).max(1, keepdims=True) / 127
    bound = unit * (0.5 + 127 * 4 * FLOAT) * np.abs(wf).sum(1) + 4 * FLOAT * (np.abs(u) @ np.abs(wf).T)
    assert (np.abs(got - u @ wf.T) <= bound).all()


def test_int8_norm_writes_no_padding_where_rows_have_no_room():
    """Tight rows of 1000: the next row begins there."""
    x = torch.randn((5, 1000), device="cuda").bfloat16()
    one = torch.ones(1000, device="cuda")
    q = torch.full((5 * 1000 + 64,), 77, dtype=torch.int8, device="cuda")
    s = torch.empty(5, device="cuda")
    with F.BlockNormPlan(5, 1000, has_y=0, post=0, quant=1) as norm:
        norm.run(x, None, None, None, one, None, q, s, stream=torch.cuda.current_stream())
        torch.cuda.synchronize()
    assert bool((q[5000:] == 77).all())
    assert bool((q[:5000].view(5, 1000).int().abs().amax(1) == 127).all())


@pytest.mark.parametrize("M", [800, 8])
def test_a_ranks_row_chunk_into_the_norm(M):
    """The rows that the reduce-scatter leaves on each rank go to the norm as
    the block's output, as they lie in `out`: bounds for the norm's results
    given these rows (those of its own test), and the rows against the oracle."""
    W, N = 8, 512
    w = I.with_shape(I.WORKLOADS["llama70b"], W=W, M=M, N=N, K=256, tile_m=256 if M > 8 else 64, tile_n=256 if M > 8 else 128)
    x = I.make_inputs(w)
    out = new_out(w)
    say("gemm_rs, norm", M)
    dev = to_device(x, w)
    with G.Plan(**desc_fields(w)) as plan:
        run_checked(plan, dev, w, out)
    check_tolerance(out_to_f64(out, w), O.reference_rows(x["A"], x["B"], x["C"], **oracle_kw(w)), w.dtype)
    g = torch.Generator().manual_seed(M)
    rows = M // W
    stream = torch.randn((M, N), generator=g).bfloat16().cuda()
    w_post, w_pre = (1 + 0.1 * torch.randn((2, N), generator=g)).cuda()
    gate = (1 + 0.1 * torch.randn((1, N), generator=g)).cuda()
    x_out, u = torch.full_like(stream, float("nan")), torch.full_like(stream, float("nan"))
    y = out.view(torch.bfloat16)
    s = torch.cuda.current_stream()
    kw = dict(rows_per_gate=rows, res_scale=0.5)
    with F.BlockNormPlan(rows, N, **kw) as norm:
        for r in range(W):
            c = slice(r * rows, (r + 1) * rows)
            norm.run(stream[c], y[c], w_post, gate, w_pre, x_out[c], u[c], stream=s)
        torch.cuda.synchronize()
    x64 = _f64(stream)
    want_x, want_u = OF.norm_forward(x64, _f64(y), _f64(w_post), _f64(gate), _f64(w_pre), **dict(kw, rows_per_gate=M))
    root = np.sqrt((want_x ** 2).mean(1, keepdims=True) + 1e-6)
    assert (np.abs(_f64(x_out) - want_x) <= 2.0 ** -8 * np.abs(want_x) + FLOAT * (np.abs(x64) + np.abs(want_x))).all()
    mag = np.abs(want_u) + (np.abs(x64) + np.abs(want_x)) / root * np.abs(_f64(w_pre))
    assert (np.abs(_f64(u) - want_u) <= 2.0 ** -8 * np.abs(want_u) + FLOAT * mag).all()
