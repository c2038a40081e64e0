"""Arrays of another type, length, stride or place than the plan's are refused
before anything is enqueued; bfloat16 as its bits is taken."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from dense_util import BF, F32, Inputs

pytestmark = pytest.mark.gpu

M, N, K = 6, 24, 40


def new(*shape, dt=BF):
    return torch.full(shape, 7.0, dtype=dt, device="cuda")


def others(t):
    two = (t.cpu(), t.half(), t.to(F32 if t.dtype == BF else BF), t[..., :-1], torch.cat((t, t), -1)[..., ::2])
    return two + ((t[:-1], torch.cat((t, t), -1)[:, :t.shape[1]], t.t().contiguous().t()) if t.dim() == 2 else ())


def each_refused(call, args):
    """`call` with one array after the other exchanged for one that it may not have."""
    for k, good in enumerate(args):
        for bad in others(good) if good is not None else ():
            with pytest.raises(G.GemmRsError) as e:
                call(*args[:k], bad, *args[k + 1:])
            assert e.value.code == G.ERR_INVALID_ARG


def test_gated():
    i, s = Inputs(0), torch.cuda.current_stream()
    x, dh, (wg, wu), (bg, bu) = i.mat(M, K), i.mat(M, N), (i.mat(K, N) for _ in range(2)), (i.vec(N) for _ in range(2))
    outs = [h, zg, zu, dzg, dzu, dx, dwg, dwu, dbg, dbu] = [new(M, N), *(new(M, N, dt=F32) for _ in range(2)), new(M, N), new(M, N), new(M, K),
                                                            new(K, N), new(K, N), new(N, dt=F32), new(N, dt=F32)]
    with F.GatedPlan(M, N, K, has_bias=1, backward=1, z_dtype=F.F32) as plan:
        def run(*a):
            plan.run(*a, stream=s)

        def back(*a):
            plan.backward(*a, stream=s)
        each_refused(run, (x, wg, wu, bg, bu, h, zg, zu))
        each_refused(back, (dh, x, wg, wu, zg, zu, dzg, dzu, dx, dwg, dwu, dbg, dbu))
        torch.cuda.synchronize()
        assert all(bool((o == 7.0).all()) for o in outs)
        run(x, wg, wu, bg, bu, h, zg, zu)
        bits = torch.empty((M, N), dtype=torch.int16, device="cuda")
        run(x.view(torch.int16), wg.view(torch.int16), wu, bg, bu, bits, zg, zu)
        back(dh, x, wg, wu, zg, zu, dzg, dzu, dx, dwg, dwu, dbg, dbu)
        torch.cuda.synchronize()
        assert torch.equal(bits.view(BF), h) and all(bool((o != 7.0).any()) for o in outs)


@pytest.mark.parametrize("out", [BF, F32])
def test_epi(out):
    i, s = Inputs(1), torch.cuda.current_stream()
    x, w, bias, r, dy = i.mat(M, K), i.mat(K, N), i.vec(N, BF), i.mat(M, N, out), i.mat(M, N, out)
    outs = [y, z, dz, dx, dw, db] = [new(M, N, dt=out), new(M, N), new(M, N), new(M, K), new(K, N, dt=F32), new(N, dt=F32)]
    with F.EpiPlan(M, N, K, act=F.ACT_GELU, out_dtype=F.F32 if out == F32 else F.BF16, has_bias=1, bias_dtype=F.BF16, has_residual=1,
                   backward=1, dw_dtype=F.F32) as plan:
        def run(*a):
            plan.run(*a, stream=s)

        def back(*a):
            plan.backward(*a, stream=s)
        each_refused(run, (x, w, bias, r, y, z))
        each_refused(back, (dy, x, w, z, dz, dx, dw, db))
        torch.cuda.synchronize()
        assert all(bool((o == 7.0).all()) for o in outs)
        run(x, w, bias, r, y, z)
        back(dy, x, w, z, dz, dx, dw, db)
        torch.cuda.synchronize()
        assert all(bool((o != 7.0).any()) for o in outs)


def test_in_place_of_another_stride_or_size():
    """y over r, dz over z or dy: threads would overwrite what others read."""
    lib, bad, ok = F._library(), G.ERR_INVALID_ARG, G.OK
    t = torch.zeros(1 << 16, device="cuda")
    a = [t.data_ptr() + 4096 * k for k in range(16)]
    for strides, same in ((dict(), True), (dict(ldr=40, ldy=32, ldz=40, lddz=32, lddy=40), False)):
        with F.EpiPlan(8, 32, 16, act=F.ACT_GELU, has_residual=1, backward=1, **strides) as plan:
            for rows in (0, 1, 8):
                want = ok if same or rows < 2 else bad
                assert lib.gemm_epi_run(plan.handle, a[0], a[1], None, a[2], a[2], a[3], rows, None) == want
                for dz in (a[4], a[5]):                # dy, z
                    assert lib.gemm_epi_backward(plan.handle, a[4], a[0], a[1], a[5], dz, a[6], a[7], None, rows, None) == want
                assert lib.gemm_epi_backward(plan.handle, a[4], a[0], a[1], a[5], a[8], a[6], a[7], None, rows, None) == ok
        strides = {k: v for k, v in strides.items() if k in ("ldz", "lddz")}
        with F.GatedPlan(8, 32, 16, backward=1, **strides) as plan:
            for rows in (0, 1, 8):
                want = ok if same or rows < 2 else bad
                for dz in ((a[5], a[6]), (a[5], a[7]), (a[7], a[6])):
                    assert lib.gemm_gated_backward(plan.handle, a[4], a[0], a[1], a[2], a[5], a[6], *dz, a[8], a[9], a[10], None, None, rows, None) == want
    with F.EpiPlan(8, 32, 16, act=F.ACT_GELU, out_dtype=F.F32, backward=1, z_dtype=F.F32) as plan, F.GatedPlan(8, 32, 16, backward=1, z_dtype=F.F32) as gated:
        for dz in (a[4], a[5]):
            assert lib.gemm_epi_backward(plan.handle, a[4], a[0], a[1], a[5], dz, a[6], a[7], None, 1, None) == bad
        assert lib.gemm_gated_backward(gated.handle, a[4], a[0], a[1], a[2], a[5], a[6], a[5], a[6], a[8], a[9], a[10], None, None, 1, None) == bad
    torch.cuda.synchronize()
