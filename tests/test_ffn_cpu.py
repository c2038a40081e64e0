"""CPU checks of the FFN operators' interface and oracle: the library exports
what the headers declare, the bound structs match the C layout, bad
descriptors and arguments are rejected before any HIP call, and the oracle's
formulas agree with differences and with hand values."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

from oracle import ffn as OF
from tensor_gemm_reduce_lds_amd import ffn as F
from tensor_gemm_reduce_lds_amd import gemm_rs as G


def test_library_exports_every_declared_function():
    names = F.header_functions()
    assert names == sorted(
        ["block_norm_" + s for s in ("plan", "run", "backward", "query", "destroy")] +
        ["gemm_q8_" + s for s in ("plan", "run", "quantize", "query", "destroy")] +
        ["gemm_grouped_" + s for s in ("plan", "run", "status", "query", "destroy")])
    lib = G.load_library()
    for n in names:
        assert hasattr(lib, n), n


STRUCTS = ["block_norm_desc_t", "block_norm_info_t", "gemm_q8_desc_t", "gemm_q8_info_t",
           "gemm_grouped_desc_t", "gemm_grouped_info_t"]


def test_struct_layout_matches_c_compiler(tmp_path):
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "block_norm.h"',
           '#include "gemm_q8.h"', '#include "gemm_grouped.h"', "int main(void) {"]
    for s in STRUCTS:
        src.append('  printf("%s %%zu\\n", sizeof(%s));' % (s, s))
        for f, _ in getattr(F, s)._fields_:
            src.append('  printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (s, f, s, f))
    src.append("  return 0; }")
    c, exe = tmp_path / "layout.c", tmp_path / "layout"
    c.write_text("\n".join(src))
    subprocess.run(["gcc", "-I", os.path.dirname(G.HEADER), str(c), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    lay = dict(line.split() for line in out.splitlines())
    for s in STRUCTS:
        cls = getattr(F, s)
        assert int(lay[s]) == ctypes.sizeof(cls), s
        for f, _ in cls._fields_:
            assert int(lay["%s.%s" % (s, f)]) == getattr(cls, f).offset, (s, f)


def _rc(make, **kw):
    try:
        make(**kw).close()
    except G.GemmRsError as e:
        return e.code
    return G.OK


INVALID, UNSUPPORTED = G.ERR_INVALID_ARG, G.ERR_UNSUPPORTED

NORM_BAD = [
    (dict(rows=0), INVALID), (dict(cols=0), INVALID), (dict(dtype=2), INVALID),
    (dict(stream_dtype=-1), INVALID), (dict(param_dtype=9), INVALID), (dict(has_y=2), INVALID),
    (dict(has_y=0), INVALID), (dict(has_y=0, post=0, pre=0), INVALID),
    (dict(has_y=0, post=0, rows_per_gate=4), INVALID), (dict(pre=0, quant=1), INVALID),
    (dict(quant=1, backward=1), INVALID), (dict(res_scale=float("nan")), INVALID),
    (dict(weight_offset=float("inf")), INVALID), (dict(eps_pre=-1.0), INVALID),
    (dict(rows_per_gate=-1), INVALID), (dict(ld_x=63), INVALID), (dict(ld_dy=1), INVALID),
    (dict(pad=1), INVALID), (dict(cols=16385), UNSUPPORTED), (dict(rows=2**31), UNSUPPORTED),
    (dict(rows_per_gate=2**31), UNSUPPORTED), (dict(ld_u=2**31), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", NORM_BAD)
def test_bad_norm_descriptors(kw, want):
    assert _rc(F.BlockNormPlan, **dict(dict(rows=8, cols=64), **kw)) == want


Q8_BAD = [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(out_dtype=2), INVALID),
    (dict(has_bias=2), INVALID), (dict(lda=48), INVALID), (dict(ldw=16), INVALID),
    (dict(ldd=31), INVALID), (dict(lda=-16), INVALID), (dict(K=72), UNSUPPORTED),
    (dict(lda=72), UNSUPPORTED), (dict(ldw=65), UNSUPPORTED), (dict(K=2**17), UNSUPPORTED),
    (dict(M=2**31), UNSUPPORTED), (dict(N=2**31), UNSUPPORTED), (dict(lda=2**23), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", Q8_BAD)
def test_bad_q8_descriptors(kw, want):
    assert _rc(F.Q8Plan, **dict(dict(M=8, N=32, K=64), **kw)) == want


GROUPED_BAD = [
    (dict(M=0), INVALID), (dict(N=0), INVALID), (dict(K=-8), INVALID), (dict(E=0), INVALID),
    (dict(op=3), INVALID), (dict(op=-1), INVALID), (dict(out_dtype=5), INVALID),
    (dict(accumulate=1), INVALID), (dict(op=F.GROUPED_TN, accumulate=2), INVALID),
    (dict(lda=63), INVALID), (dict(ldb=31), INVALID), (dict(ldc=31), INVALID),
    (dict(op=F.GROUPED_NT, ldb=32), INVALID), (dict(E=1025), UNSUPPORTED),
    (dict(M=2**31), UNSUPPORTED), (dict(K=2**23), UNSUPPORTED), (dict(ldc=2**23), UNSUPPORTED),
    (dict(M=2**30, N=2**20, ldb=2**20), UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", GROUPED_BAD)
def test_bad_grouped_descriptors(kw, want):
    assert _rc(F.GroupedPlan, **dict(dict(M=8, N=32, K=64, E=4, op=F.GROUPED_NN), **kw)) == want


def test_null_handles_and_bad_quantize_arguments():
    lib = F._library()
    for fam in ("block_norm", "gemm_q8", "gemm_grouped"):
        h = ctypes.c_void_p(7)
        assert getattr(lib, fam + "_plan")(None, ctypes.byref(h)) == INVALID
        assert getattr(lib, fam + "_query")(None, None) == INVALID
        assert getattr(lib, fam + "_destroy")(None) == G.OK
    assert lib.block_norm_run(*([None] * 9), 0, None) == INVALID
    assert lib.block_norm_backward(*([None] * 13), 0, None) == INVALID
    assert lib.gemm_q8_run(*([None] * 7), 0, None) == INVALID
    assert lib.gemm_grouped_run(*([None] * 5), 0, None) == INVALID
    assert lib.gemm_grouped_status(None, None, None) == INVALID
    p = 4096   # a well-aligned address that is never dereferenced
    bad = [(None, 0, 1, 16, 16, p, 16, p), (p, 2, 1, 16, 16, p, 16, p), (p, 0, -1, 16, 16, p, 16, p),
           (p, 0, 1, 0, 16, p, 16, p), (p, 0, 1, 16, 15, p, 16, p), (p, 0, 1, 17, 17, p, 17, p),
           (p + 1, 0, 1, 16, 16, p, 16, p), (p, 0, 1, 16, 16, p, 16, p + 2), (p, 0, 1, 16, 16, None, 16, p)]
    for a in bad:
        assert lib.gemm_q8_quantize(*a, None) == INVALID, a
    assert lib.gemm_q8_quantize(p, 0, 1, 2**17, 2**17, p, 2**17, p, None) == UNSUPPORTED
    assert lib.gemm_q8_quantize(p, 0, 0, 16, 16, p, 16, p, None) == G.OK


# ---- the oracle's own pins ----------------------------------------------------
def test_norm_hand_values():
    x, u = OF.norm_forward(np.array([[1.0, 2.0]]), np.array([[3.0, 4.0]]), np.array([1.0, 2.0]),
                           np.array([[2.0, 0.5]]), np.array([0.0, 1.0]), rows_per_gate=1,
                           res_scale=0.5, eps_post=0.0, eps_pre=0.0)
    r2 = 1 / np.sqrt(12.5)
    want = np.array([[0.5 + 2.0 * 3.0 * r2, 1.0 + 0.5 * 4.0 * r2 * 2.0]])
    assert np.allclose(x, want, rtol=1e-15)
    assert u[0, 0] == 0.0 and np.isclose(u[0, 1], want[0, 1] / np.sqrt((want**2).mean()), rtol=1e-15)
    x, u = OF.norm_forward(np.array([[3.0, 4.0]]), w_pre=np.array([1.0, 1.0]), eps_pre=0.0,
                           weight_offset=1.0)
    assert np.allclose(u, 2 * np.array([[3.0, 4.0]]) / np.sqrt(12.5), rtol=1e-15)


@pytest.mark.parametrize("post,gated,pre,offset", [(1, 1, 1, 0.0), (0, 1, 1, 1.0), (1, 0, 1, 1.0),
                                                   (1, 1, 0, 0.0), (0, 0, 1, 0.0)])
def test_norm_gradient_formulas_against_differences(post, gated, pre, offset):
    """Every gradient against central differences of the forward in float64
    (step 1e-5: truncation ~1e-10 of the third derivative, rounding ~1e-11)."""
    g = np.random.default_rng(3)
    T, H, rpg = 5, 7, 2
    v = dict(x=g.standard_normal((T, H)), y=g.standard_normal((T, H)),
             w_post=g.standard_normal(H) if post else None,
             gate=g.standard_normal((3, H)) if gated else None,
             w_pre=g.standard_normal(H) if pre else None)
    dxo, du = g.standard_normal((T, H)), g.standard_normal((T, H)) if pre else None
    kw = dict(rows_per_gate=rpg, res_scale=0.7, weight_offset=offset)

    def loss(**t):
        xo, u = OF.norm_forward(**t, **kw)
        return (dxo * xo).sum() + ((du * u).sum() if pre else 0.0)

    xo, _ = OF.norm_forward(**v, **kw)
    got = OF.norm_backward(dxo, du, xo, v["y"], v["w_post"], v["gate"], v["w_pre"], **kw)
    for name, key in (("dx", "x"), ("dy", "y"), ("dw_post", "w_post"), ("dgate", "gate"), ("dw_pre", "w_pre")):
        if v[key] is None:
            assert name not in got
            continue
        d = np.zeros_like(v[key])
        for i in np.ndindex(d.shape):
            hi, lo = v[key].copy(), v[key].copy()
            hi[i] += 1e-5
            lo[i] -= 1e-5
            d[i] = (loss(**{**v, key: hi}) - loss(**{**v, key: lo})) / 2e-5
        assert np.allclose(got[name][0], d, rtol=1e-6, atol=1e-7), name


def test_quantize_hand_values():
    q, s = OF.quantize_rows(np.array([[127.0, -127.0, 0.5, 1.5, 2.5], [0, 0, 0, 0, 0],
                                      [np.inf, 1, 2, 3, 4]], dtype=np.float32))
    assert q[0].tolist() == [127, -127, 0, 2, 2] and s[0] == 1.0
    assert not q[1].any() and s[1] == 0.0
    assert not q[2].any() and np.isnan(s[2])


def test_q8_and_grouped_hand_values():
    y = OF.q8_product(np.array([[1, 2]], dtype=np.int8), np.array([0.5]), np.array([[3, 4], [-1, 0]], dtype=np.int8),
                      np.array([2.0, 4.0]), np.array([1.0, 0.0]))
    assert y.tolist() == [[12.0, -2.0]]
    A, B = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]]), np.array([[[1.0], [1.0]], [[2.0], [0.0]]])
    C, mag = OF.grouped("NN", A, B, [0, 1, 2], 1, 2)
    assert C[:2, 0].tolist() == [3.0, 6.0] and np.isnan(C[2, 0])
    C, _ = OF.grouped("NT", A, B.transpose(0, 2, 1), [1, 1, 3], 1, 2)
    assert np.isnan(C[0, 0]) and C[1:, 0].tolist() == [6.0, 10.0]
    C, _ = OF.grouped("TN", A, A[:, :1], [0, 0, 2], 1, 2)
    assert not C[0].any() and C[1, :, 0].tolist() == [10.0, 14.0]
