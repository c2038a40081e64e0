"""Arrays that the dense products' plans refuse before the library is called: the
kernels know them by address alone.  The library is replaced here."""
import pytest
import torch

from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

BF, F32 = torch.bfloat16, torch.float32
M, N, K = 6, 24, 40


class OnGpu(torch.Tensor):
    """A host tensor that says it is on the first GPU."""

    device = property(lambda self: torch.device("cuda", 0))

    def get_device(self):
        return 0


def new(*shape, dt=BF):
    return torch.zeros(shape, dtype=dt).as_subclass(OnGpu)


@pytest.fixture
def calls(monkeypatch):
    class Library:
        made = []

        def __getattr__(self, name):
            return lambda *a: self.made.append((name, a)) or G.OK if name.endswith(("_run", "_backward")) else G.OK

    Library.made = []
    lib = Library()
    monkeypatch.setattr(F, "_library", lambda: lib)
    return lib.made


def arrays(family, layout, z, out, dw, bias, pad=0):
    """name -> tensor of a forward and of a backward call."""
    w = (K, N) if layout == F.WEIGHTS_KN else (N, K)

    def mat(r, c, dt=BF):
        return new(r, c + pad, dt=dt)[:, :c]
    if family == "gated":
        a = dict(x=mat(M, K), w_gate=mat(*w), w_up=mat(*w), b_gate=new(N, dt=bias), b_up=new(N, dt=bias), h=mat(M, N), z_gate=mat(M, N, z),
                 z_up=mat(M, N, z), dh=mat(M, N), dz_gate=mat(M, N), dz_up=mat(M, N), dx=mat(M, K), dw_gate=mat(*w, dw), dw_up=mat(*w, dw),
                 db_gate=new(N, dt=F32), db_up=new(1, N, dt=F32))
        return a, ("x", "w_gate", "w_up", "b_gate", "b_up", "h", "z_gate", "z_up"), ("dh", "x", "w_gate", "w_up", "z_gate", "z_up", "dz_gate", "dz_up",
                                                                                    "dx", "dw_gate", "dw_up", "db_gate", "db_up")
    a = dict(x=mat(M, K), w=mat(*w), bias=new(N, dt=bias), r=mat(M, N, out), y=mat(M, N, out), z=mat(M, N, z), dy=mat(M, N, out), dz=mat(M, N),
             dx=mat(M, K), dw=mat(*w, dw), dbias=new(N, dt=F32))
    return a, ("x", "w", "bias", "r", "y", "z"), ("dy", "x", "w", "z", "dz", "dx", "dw", "dbias")


def plan_of(family, layout=F.WEIGHTS_KN, z=BF, out=BF, dw=BF, bias=F32, pad=0):
    code = lambda dt: F.F32 if dt == F32 else F.BF16  # noqa: E731
    w, lds = N if layout == F.WEIGHTS_KN else K, {}
    if pad:
        lds = dict(ldx=K + pad, ldw=w + pad, ldz=N + pad, lddz=N + pad, lddx=K + pad, lddw=w + pad)
        lds.update(dict(ldh=N + pad, lddh=N + pad) if family == "gated" else dict(ldr=N + pad, ldy=N + pad, lddy=N + pad))
    kw = dict(layout=layout, act=F.ACT_SILU, has_bias=1, bias_dtype=code(bias), backward=1, dw_dtype=code(dw), z_dtype=code(z), **lds)
    return F.GatedPlan(M, N, K, **kw) if family == "gated" else F.EpiPlan(M, N, K, out_dtype=code(out), has_residual=1, **kw)


def call(plan, a, names, back, **kw):
    (plan.backward if back else plan.run)(*(a[n] for n in names), **kw)


def refused(plan, a, names, back, calls, **kw):
    before = len(calls)
    with pytest.raises(G.GemmRsError) as e:
        call(plan, a, names, back, **kw)
    assert e.value.code == G.ERR_INVALID_ARG and len(calls) == before
    return str(e.value)


TYPES = [dict(), dict(z=F32), dict(out=F32), dict(dw=F32), dict(bias=BF), dict(z=F32, out=F32, dw=F32, bias=BF)]


@pytest.mark.parametrize("layout", [F.WEIGHTS_KN, F.WEIGHTS_NK])
@pytest.mark.parametrize("pad", [0, 3])
@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("family", ["gated", "epi"])
def test_each_array_of_another_type_length_stride_or_place(family, types, pad, layout, calls):
    t = dict(dict(z=BF, out=BF, dw=BF, bias=F32), **types)
    plan = plan_of(family, layout, pad=pad, **t)
    a, forward, backward = arrays(family, layout, t["z"], t["out"], t["dw"], t["bias"], pad)
    for names, back in ((forward, False), (backward, True)):
        call(plan, a, names, back)
        assert calls[-1][1][1:1 + len(names)] == tuple(a[n].data_ptr() for n in names)
        for n in names:
            good = a[n]
            per_row = good.dim() == 2 and good.shape[0] == M and n not in ("w", "w_gate", "w_up")
            bad = [good.to(F32 if good.dtype == BF else BF), good.to(torch.float16), good.as_subclass(torch.Tensor),          # type, the host's
                   good[..., :-1], new(*good.shape[:-1], 2 * good.shape[-1], dt=good.dtype)[..., ::2]]                        # fewer columns, gaps
            if good.dim() == 2:
                bad += [good[:-1]]                                                                                            # fewer rows
                if good.shape[0] > 1:                                                                                         # another stride
                    bad += [new(good.shape[0], good.shape[1] + pad + 1, dt=good.dtype)[:, :good.shape[1]],
                            new(*reversed(good.shape), dt=good.dtype).t(), new(1, good.shape[1], dt=good.dtype).expand(*good.shape)]
            for b in bad:
                assert " %s (" % n in refused(plan, dict(a, **{n: b}), names, back, calls), (n, b.shape, b.stride())
            fine = [good.data_ptr(), new(good.numel() + 4 * pad * max(good.shape), dt=good.dtype)]                            # an address; an array without a shape
            if per_row:
                fine += [new(M + 2, good.shape[1] + pad, dt=good.dtype), new(2, M // 2, good.shape[1] + pad, dt=good.dtype)[..., :good.shape[1]]]
            if good.dtype == BF:
                fine.append(good.view(torch.int16).as_subclass(OnGpu))
            for f in fine:
                call(plan, dict(a, **{n: f}), names, back)
    assert not any(None in c[1][1:-1] for c in calls)


@pytest.mark.parametrize("family", ["gated", "epi"])
def test_a_calls_rows_count(family, calls):
    plan = plan_of(family)
    a, forward, backward = arrays(family, F.WEIGHTS_KN, BF, BF, BF, F32)
    few = {n: t[:2] if t.dim() == 2 and t.shape[0] == M else t for n, t in a.items()}
    none = {n: t[:0] if t.dim() == 2 and t.shape[0] == M else t for n, t in a.items()}
    for names, back in ((forward, False), (backward, True)):
        for rows in (1, 2):
            call(plan, few, names, back, rows=rows)
        refused(plan, few, names, back, calls, rows=3)
        call(plan, none, names, back, rows=0)
        for n in ("w", "w_gate", "bias", "dw", "db_up"):
            if n in names:
                refused(plan, dict(none, **{n: a[n][..., :-1]}), names, back, calls, rows=2)
    assert len(calls) == 6


def test_arrays_may_be_missing_or_have_an_address_only(calls):
    class Address:
        def data_ptr(self):
            return 4096

    plan = plan_of("gated")
    plan.run(Address(), 1, 2, None, None, Address(), rows=3)
    assert calls[-1][1][1:] == (4096, 1, 2, None, None, 4096, None, None, 3, None)
