"""The block norm (include/block_norm.h) on the GPU against the fp64 oracle.

Bounds, from the arithmetic: a value written as bfloat16 is rounded to 8
significant bits (to nearest: relative 2^-8 at most); everything before it is in floats with
sums of at most a few hundred terms per thread tree, so a row's values carry
at most FLOAT = 64 * 2^-24 of the magnitudes that enter them; a sum over
T rows adds (T + 64) * 2^-24 of the sum of magnitudes."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G

from gpu_util import say

pytestmark = pytest.mark.gpu

EPS24 = 2.0 ** -24
FLOAT = 64 * EPS24


def _t(dt):
    return torch.float32 if dt == F.F32 else torch.bfloat16


def _half(dt):
    return 0.0 if dt == F.F32 else 2.0 ** -8


class Case:
    """Seeded inputs in strided storage whose gaps hold NaN."""

    def __init__(self, rows, cols, dtype=F.BF16, stream_dtype=F.BF16, param_dtype=F.F32, has_y=1, post=1,
                 pre=1, rpg=0, pad=0, offset=0.0, res_scale=0.75, seed=0, quant=0, backward=0):
        self.rows, self.cols, self.pad, self.rpg = rows, cols, pad, rpg
        self.yt, self.st, self.pt = dtype, stream_dtype, param_dtype
        self.g = torch.Generator().manual_seed(seed)
        self.has_y, self.post, self.pre = has_y, post, pre
        ld = cols + pad
        self.kw = dict(rows_per_gate=rpg, res_scale=res_scale, weight_offset=offset)
        self.x = self.row(self.st, 1.5)
        self.y = self.row(self.yt, 0.5) if has_y else None
        self.w_post = self.vec() if post else None
        self.w_pre = self.vec() if pre else None
        self.gate = self.vec(-(-rows // rpg)) if rpg else None
        self.plan = F.BlockNormPlan(
            rows=rows, cols=cols, dtype=dtype, stream_dtype=stream_dtype, param_dtype=param_dtype,
            has_y=has_y, post=post, pre=pre, quant=quant, backward=backward,
            ld_x=ld, ld_y=ld, ld_x_out=ld, ld_dx_out=ld, ld_du=0 if not backward else ld, **self.kw)

    def row(self, dt, scale):
        t = torch.full((self.rows, self.cols + self.pad), float("nan"))
        t[:, :self.cols] = torch.randn((self.rows, self.cols), generator=self.g) * scale
        return t.to(_t(dt)).cuda()

    def vec(self, n=None):
        shape = (self.cols,) if n is None else (n, self.cols)
        return (0.8 + 0.3 * torch.randn(shape, generator=self.g)).to(_t(self.pt)).cuda()

    def f64(self, t):
        return None if t is None else t[..., :self.cols].double().cpu().numpy()

    def oracle(self):
        return OF.norm_forward(self.f64(self.x), self.f64(self.y), self.f64(self.w_post), self.f64(self.gate),
                               self.f64(self.w_pre), **self.kw)


def close(got, want, mag, rel, what):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    bound = rel * np.abs(want) + mag
    bad = np.abs(got - want) > bound
    assert not bad.any(), (what, int(bad.sum()), float((np.abs(got - want) / (bound + 1e-300)).max()))


SHAPES = [(1, 8), (3, 64), (5, 512), (7, 1000), (2, 1), (4, 513), (3, 2049), (2, 2056), (3, 4096), (2, 4104),
          (3, 8192), (2, 8191), (2, 16384), (2, 16383), (600, 72)]
TYPES = [(F.BF16, F.BF16, F.F32), (F.BF16, F.F32, F.BF16), (F.F32, F.BF16, F.F32), (F.F32, F.F32, F.BF16)]


def _forward(c):
    s = torch.cuda.current_stream()
    x_out = torch.full_like(c.x, float("nan")) if c.has_y else None
    u = torch.full((c.rows, c.cols), float("nan"), dtype=_t(c.yt), device="cuda") if c.pre else None
    c.plan.run(c.x, c.y, c.w_post, c.gate, c.w_pre, x_out, u, stream=s)
    torch.cuda.synchronize()
    want_x, want_u = c.oracle()
    if c.has_y:
        mag = FLOAT * (np.abs(c.f64(c.x)) + np.abs(want_x))
        close(x_out[:, :c.cols], want_x, mag, _half(c.st), "x_out")
        assert x_out[:, c.cols:].isnan().all()          # the gaps are not written
    if c.pre:
        row = np.sqrt((want_x ** 2).mean(1, keepdims=True) + 1e-6)
        w = np.abs(c.kw["weight_offset"] + c.f64(c.w_pre))
        close(u, want_u, FLOAT * (np.abs(want_u) + (np.abs(c.f64(c.x)) + np.abs(want_x)) / row * w), _half(c.yt), "u")
    return x_out, u


@pytest.mark.parametrize("types", TYPES, ids=["bb", "bf", "fb", "ff"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(rows, cols, types):
    say("norm forward", rows, cols, types)
    _forward(Case(rows, cols, *types, rpg=2, seed=rows + cols))


VARIANTS = [dict(has_y=0, post=0), dict(post=0), dict(pre=0), dict(rpg=0), dict(rpg=1), dict(rpg=100),
            dict(post=0, rpg=3, offset=1.0), dict(pad=8), dict(pad=5), dict(offset=1.0), dict(has_y=0, post=0, pad=3)]


@pytest.mark.parametrize("kw", VARIANTS, ids=str)
@pytest.mark.parametrize("cols", [320, 4097])
def test_forward_variants(cols, kw):
    say("norm forward variant", cols, kw)
    _forward(Case(9, cols, **kw))


def test_forward_in_place_fewer_rows_and_none():
    c = Case(9, 640)
    s = torch.cuda.current_stream()
    want, _ = _forward(c)
    x = c.x.clone()
    u = torch.full((9, 640), 7.0, dtype=torch.bfloat16, device="cuda")
    c.plan.run(x, c.y, c.w_post, None, c.w_pre, x, u, rows=0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(x, c.x) and bool((u == 7.0).all())
    c.plan.run(x, c.y, c.w_post, None, c.w_pre, x, u, rows=4, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(x[:4], want[:4]) and torch.equal(x[4:], c.x[4:]) and bool((u[4:] == 7.0).all())


def test_special_rows():
    """A zero row gives zeros, a row with a NaN or infinity spoils itself only."""
    c = Case(4, 1024, rpg=0)
    c.x[0], c.y[0] = 0.0, 0.0
    c.y[1, 17] = float("nan")
    c.x[2, 3] = float("inf")
    x_out, u = torch.empty_like(c.x), torch.empty_like(c.y)
    c.plan.run(c.x, c.y, c.w_post, None, c.w_pre, x_out, u, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert not x_out[0].any() and not u[0].any()
    assert x_out[1].isnan().all() and u[1].isnan().all()
    assert x_out[2, 3].isinf() and x_out[2].isfinite().sum() == 1023 and u[2, 3].isnan()
    assert u[2, 4:].float().abs().max() == 0          # finite / infinite root mean square
    assert x_out[3].isfinite().all() and u[3].isfinite().all()


@pytest.mark.parametrize("cols", [16, 1000, 1001, 8192])
def test_quantised_output(cols):
    """int8 rows: u_scale is max|u|/127 and every integer is the nearest of the
    oracle's u/u_scale, up to the float error where that is nearly a tie."""
    c = Case(6, cols, quant=1, rpg=2)
    c.x[4], c.y[4] = 0.0, 0.0
    c.x[5, cols - 1] = float("inf")
    x_out = torch.empty_like(c.x)
    q = torch.full((6, cols), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((6,), -1.0, device="cuda")
    c.plan.run(c.x, c.y, c.w_post, c.gate, c.w_pre, x_out, q, scale, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    c.x[5] = 0.0
    _, want = c.oracle()
    q, scale = q.cpu().numpy().astype(np.float64), scale.cpu().numpy().astype(np.float64)
    assert scale[4] == 0 and not q[4].any() and np.isnan(scale[5]) and not q[5].any()
    amax = np.abs(want[:4]).max(1)
    assert np.abs(scale[:4] - amax / 127).max() <= 4 * FLOAT * amax.max() / 127
    exact = want[:4] / (amax / 127)[:, None]
    assert np.abs(q[:4] - exact).max() <= 0.5 + 127 * 4 * FLOAT
    assert np.abs(q[:4]).max(1).tolist() == [127.0] * 4


def _backward(c, with_dxo=True):
    s = torch.cuda.current_stream()
    dxo = c.row(c.st, 0.4) if with_dxo else None
    du = c.row(c.yt, 0.4) if c.pre else None
    nan = lambda t, *shape: torch.full(shape, float("nan"), dtype=t, device="cuda")  # noqa: E731
    G_ = c.gate.shape[0] if c.rpg else 0
    o = dict(dx=nan(_t(c.st), c.rows, c.cols))
    if c.has_y:
        o["dy"] = nan(_t(c.yt), c.rows, c.cols)
    if c.post:
        o["dw_post"] = nan(torch.float32, c.cols)
    if c.rpg:
        o["dgate"] = nan(torch.float32, G_, c.cols)
    if c.pre:
        o["dw_pre"] = nan(torch.float32, c.cols)

    def run():
        c.plan.backward(dxo, du, c.x if c.pre else None, c.y, c.w_post, c.gate, c.w_pre, o["dx"], o.get("dy"),
                        o.get("dw_post"), o.get("dgate"), o.get("dw_pre"), stream=s)
        torch.cuda.synchronize()

    run()
    want = OF.norm_backward(c.f64(dxo), c.f64(du), c.f64(c.x), c.f64(c.y), c.f64(c.w_post), c.f64(c.gate),
                            c.f64(c.w_pre), **c.kw)
    assert set(want) == set(o)
    for k, (ref, mag) in want.items():
        sums = k.startswith("dw") or k == "dgate"
        rel = 0.0 if sums else _half(c.st if k == "dx" else c.yt)
        close(o[k], ref, (FLOAT + (c.rows * EPS24 if sums else FLOAT)) * mag, rel, k)
    first = {k: t.clone() for k, t in o.items()}
    for t in o.values():
        t.fill_(float("nan"))
    run()
    for k, t in o.items():                               # fixed order: equal bits
        assert torch.equal(t, first[k]), k
    return o


@pytest.mark.parametrize("types", TYPES, ids=["bb", "bf", "fb", "ff"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(rows, cols, types):
    say("norm backward", rows, cols, types)
    _backward(Case(rows, cols, *types, rpg=2, seed=rows + cols, backward=1))


@pytest.mark.parametrize("types", TYPES, ids=["bb", "bf", "fb", "ff"])
@pytest.mark.parametrize("end", range(1, 8))
def test_row_ends_of_every_length(end, types):
    """Rows that end 1..7 elements past a multiple of 8, and rows of fewer than 8."""
    for cols in (end, 8 + end, 512 + end):
        for pad in (0, 3):
            say("norm ends", cols, types)
            _forward(Case(3, cols, *types, rpg=2, pad=pad, seed=cols))
            _backward(Case(3, cols, *types, rpg=2, pad=pad, seed=cols, backward=1))


@pytest.mark.parametrize("rows,cols", [(260, 4104), (257, 8191), (1100, 2056)])
def test_many_rows(rows, cols):
    """More rows than CUs, where long rows take fewer threads each, and more than
    the workgroups of a backward launch."""
    say("norm many rows", rows, cols)
    _forward(Case(rows, cols, rpg=100))
    _backward(Case(rows, cols, rpg=100, backward=1))


@pytest.mark.parametrize("kw", VARIANTS, ids=str)
@pytest.mark.parametrize("cols", [320, 4097])
def test_backward_variants(cols, kw):
    say("norm backward variant", cols, kw)
    _backward(Case(9, cols, backward=1, **kw))


@pytest.mark.parametrize("rpg", [0, 1, 3, 7, 64, 129, 1000, 1500, 5000])
def test_backward_gate_groups_against_row_runs(rpg):
    """More rows than workgroups, so runs of rows begin and end inside gate
    groups of every kind (shorter, longer, equal, the last one ragged)."""
    say("norm backward gate groups", rpg)
    _backward(Case(2500, 4096, rpg=rpg, backward=1, seed=rpg))


def test_backward_without_stream_gradient_and_without_rows():
    c = Case(11, 768, backward=1)
    _backward(c, with_dxo=False)
    dw = torch.full((2, 768), float("nan"), device="cuda")
    t = torch.full((11, 768), 5.0, dtype=torch.bfloat16, device="cuda")
    c.plan.backward(t, t, c.x, c.y, c.w_post, None, c.w_pre, t, t, dw[0], None, dw[1], rows=0,
                    stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert not dw.any() and bool((t == 5.0).all())


def test_gradient_against_differences_of_the_kernel():
    """Central differences of the forward kernel along random directions in
    32-bit types against the backward's inner products.  With step h the
    difference carries 2 * FLOAT * sum|terms| / (2h) of rounding; its
    truncation is computed by the same difference in float64."""
    c = Case(6, 264, F.F32, F.F32, F.F32, rpg=4, backward=1, seed=11)
    g = torch.Generator().manual_seed(5)
    dxo, du = (torch.randn((6, 264), generator=g).cuda() for _ in range(2))
    s = torch.cuda.current_stream()

    def outputs(**t):
        v = dict(x=c.x, y=c.y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre)
        v.update(t)
        xo, u = torch.empty_like(c.x), torch.empty_like(c.x)
        c.plan.run(v["x"], v["y"], v["w_post"], v["gate"], v["w_pre"], xo, u, stream=s)
        ref = OF.norm_forward(*(c.f64(v[k]) for k in ("x", "y", "w_post", "gate", "w_pre")), **c.kw)
        return (xo.double().cpu().numpy(), u.double().cpu().numpy()), ref

    (xo, u), _ = outputs()
    d64, u64 = c.f64(dxo), c.f64(du)
    terms = np.abs(d64 * xo).sum() + np.abs(u64 * u).sum()
    xo_t = torch.from_numpy(xo).float().cuda()
    o = {k: torch.empty_like(v) for k, v in dict(x=c.x, y=c.y, w_post=c.w_post, gate=c.gate, w_pre=c.w_pre).items()}
    c.plan.backward(dxo, du, xo_t, c.y, c.w_post, c.gate, c.w_pre, o["x"], o["y"], o["w_post"], o["gate"], o["w_pre"],
                    stream=s)
    torch.cuda.synchronize()
    ref = OF.norm_backward(d64, u64, xo, c.f64(c.y), c.f64(c.w_post), c.f64(c.gate), c.f64(c.w_pre), **c.kw)
    h = 2.0 ** -6
    for k, name in (("x", "dx"), ("y", "dy"), ("w_post", "dw_post"), ("gate", "dgate"), ("w_pre", "dw_pre")):
        base = getattr(c, k)
        v = torch.randn(base.shape, generator=g).cuda()
        (hi, ref_hi), (lo, ref_lo) = outputs(**{k: base + h * v}), outputs(**{k: base - h * v})
        L = lambda t: (d64 * t[0]).sum() + (u64 * t[1]).sum()  # noqa: E731
        fd, fd64 = (L(hi) - L(lo)) / (2 * h), (L(ref_hi) - L(ref_lo)) / (2 * h)
        v64 = v.double().cpu().numpy()
        got = (o[k].double().cpu().numpy() * v64).sum()
        want, mag = (ref[name][0] * v64).sum(), (ref[name][1] * np.abs(v64)).sum()
        bound = abs(fd64 - want) + 2 * FLOAT * terms / (2 * h) + 2 * FLOAT * mag
        assert abs(fd - got) <= bound, (k, fd, got, bound)


def test_refusals():
    lib = F._library()
    c = Case(4, 64, rpg=2, backward=1)
    x, y, w, gt, p = (t.data_ptr() for t in (c.x, c.y, c.w_post, c.gate, c.w_pre))
    o = torch.empty((4, 64), dtype=torch.bfloat16, device="cuda").data_ptr()
    h = c.plan.handle
    ok = [x, y, w, gt, p, o, o + 256, None]

    def run(args, rows=4):
        return lib.block_norm_run(h, *args, rows, None)

    for i in range(7):
        assert run(ok[:i] + [None] + ok[i + 1:]) == G.ERR_INVALID_ARG, i
        assert run(ok[:i] + [ok[i] + 1] + ok[i + 1:]) == G.ERR_INVALID_ARG, i
    assert run(ok[:7] + [o]) == G.ERR_INVALID_ARG                      # a scale without quant
    assert run(ok, 5) == G.ERR_INVALID_ARG and run(ok, -1) == G.ERR_INVALID_ARG
    args = [o, o, x, y, w, gt, p, o, o, w, gt, p]
    for i in range(1, 12):
        bad = args[:i] + [None] + args[i + 1:]
        assert lib.block_norm_backward(h, *bad, 4, None) == G.ERR_INVALID_ARG, i
    with Case(4, 64).plan as plain:
        assert lib.block_norm_backward(plain.handle, *args, 4, None) == G.ERR_INVALID_ARG
    assert ctypes.sizeof(F.block_norm_info_t) == 16 and c.plan.info.gate_rows == 2


def test_graph_replays_match_eager():
    c = Case(300, 2048, rpg=7, backward=1)
    o = _backward(c)
    x_out, u = _forward(Case(300, 2048, rpg=7))
    dxo, du = c.row(c.st, 0.4), c.row(c.yt, 0.4)
    side = torch.cuda.Stream()
    xo, uu = torch.empty_like(x_out), torch.empty_like(u)

    def passes(s):
        c.plan.run(c.x, c.y, c.w_post, c.gate, c.w_pre, xo, uu, stream=s)
        c.plan.backward(dxo, du, xo, c.y, c.w_post, c.gate, c.w_pre, o["dx"], o["dy"], o["dw_post"], o["dgate"],
                        o["dw_pre"], stream=s)

    passes(torch.cuda.current_stream())
    torch.cuda.synchronize()
    want = [t.clone() for t in (xo, uu, *o.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        passes(side)
    for _ in range(3):
        for t in (xo, uu, *o.values()):
            t.fill_(-1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((xo, uu, *o.values()), want):
            assert torch.equal(a, b)
        passes(torch.cuda.current_stream())
        torch.cuda.synchronize()
