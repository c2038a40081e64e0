"""The block norm with a row stride of its own for every array, so that two
strides exchanged would be seen: gaps hold NaN and stay as they are.  Bounds as
in test_gpu_ffn_norm.py."""
import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F

from gpu_util import say
from test_gpu_ffn_norm import EPS24, FLOAT, TYPES, _half, _t, close

pytestmark = pytest.mark.gpu

NAN = float("nan")
NAMES = ("x", "y", "x_out", "u", "dx_out", "du", "dx", "dy")


class Arrays:
    def __init__(self, rows, cols, step, st, yt, seed):
        self.rows, self.cols = rows, cols
        self.ld = {n: cols + step * (3 * i % 8 + 1) for i, n in enumerate(NAMES)}
        assert len(set(self.ld.values())) == len(NAMES)
        self.dt = {n: _t(st if "x" in n else yt) for n in NAMES}
        self.g = torch.Generator().manual_seed(seed)

    def filled(self, name, scale):
        t = torch.full((self.rows, self.ld[name]), NAN)
        t[:, :self.cols] = torch.randn((self.rows, self.cols), generator=self.g) * scale
        return t.to(self.dt[name]).cuda()

    def blank(self, name):
        return torch.full((self.rows, self.ld[name]), NAN, dtype=self.dt[name], device="cuda")

    def f64(self, t):
        return t[..., :self.cols].double().cpu().numpy()

    def gaps(self, t):
        assert t[:, self.cols:].isnan().all()


@pytest.mark.parametrize("types", TYPES, ids=["bb", "bf", "fb", "ff"])
@pytest.mark.parametrize("step", [8, 1])
@pytest.mark.parametrize("rows,cols", [(5, 320), (7, 4097), (300, 4104), (3, 9001)])
def test_every_stride_is_its_own(rows, cols, step, types):
    say("norm strides", rows, cols, step, types)
    yt, st, pt = types
    a = Arrays(rows, cols, step, st, yt, rows + cols)
    w_post, w_pre = ((0.8 + 0.3 * torch.randn(cols, generator=a.g)).to(_t(pt)).cuda() for _ in range(2))
    gate = (0.8 + 0.3 * torch.randn((-(-rows // 3), cols), generator=a.g)).to(_t(pt)).cuda()
    kw = dict(rows_per_gate=3, res_scale=0.75, weight_offset=0.0)
    x, y, dxo, du = a.filled("x", 1.5), a.filled("y", 0.5), a.filled("dx_out", 0.4), a.filled("du", 0.4)
    s = torch.cuda.current_stream()
    plan = F.BlockNormPlan(rows, cols, dtype=yt, stream_dtype=st, param_dtype=pt, backward=1,
                           **{"ld_" + n: v for n, v in a.ld.items()}, **kw)
    x_out, u = a.blank("x_out"), a.blank("u")
    plan.run(x, y, w_post, gate, w_pre, x_out, u, stream=s)
    torch.cuda.synchronize()
    x64, y64, p64 = a.f64(x), a.f64(y), [t.double().cpu().numpy() for t in (w_post, gate, w_pre)]
    want_x, want_u = OF.norm_forward(x64, y64, *p64, **kw)
    close(x_out[:, :cols], want_x, FLOAT * (np.abs(x64) + np.abs(want_x)), _half(st), "x_out")
    row = np.sqrt((want_x ** 2).mean(1, keepdims=True) + 1e-6)
    close(u[:, :cols], want_u, FLOAT * (np.abs(want_u) + (np.abs(x64) + np.abs(want_x)) / row * np.abs(p64[2])),
          _half(yt), "u")
    a.gaps(x_out)
    a.gaps(u)

    dx, dy = a.blank("dx"), a.blank("dy")
    dw = torch.full((2, cols), NAN, device="cuda")
    dg = torch.full(gate.shape, NAN, device="cuda")
    plan.backward(dxo, du, x_out, y, w_post, gate, w_pre, dx, dy, dw[0], dg, dw[1], stream=s)
    torch.cuda.synchronize()
    want = OF.norm_backward(a.f64(dxo), a.f64(du), a.f64(x_out), y64, *p64, **kw)
    got = dict(dx=dx[:, :cols], dy=dy[:, :cols], dw_post=dw[0], dgate=dg, dw_pre=dw[1])
    for k, (ref, mag) in want.items():
        sums = k in ("dw_post", "dw_pre", "dgate")
        rel = 0.0 if sums else _half(st if k == "dx" else yt)
        close(got[k], ref, (FLOAT + (rows * EPS24 if sums else FLOAT)) * mag, rel, k)
    a.gaps(dx)
    a.gaps(dy)


@pytest.mark.parametrize("post", [0, 1])
@pytest.mark.parametrize("cols", [5, 513, 1029, 4097, 8191, 16383])
def test_in_place_on_rows_of_any_length(cols, post):
    """x' over x where a row's last columns are read together with their
    neighbours', which another wave may have overwritten by then."""
    say("norm in place", cols, post)
    g = torch.Generator().manual_seed(cols)
    x, y = (torch.randn((70, cols), generator=g).bfloat16().cuda() for _ in range(2))
    w = (1 + 0.1 * torch.randn((2, cols), generator=g)).cuda()
    s = torch.cuda.current_stream()
    with F.BlockNormPlan(70, cols, post=post) as plan:
        outs = []
        for to in (torch.empty_like(x), x.clone()):
            src = x if not outs else to
            u = torch.empty_like(x)
            plan.run(src, y, w[0] if post else None, None, w[1], to, u, stream=s)
            outs.append((to, u))
        torch.cuda.synchronize()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
