"""fp64 oracle of the FFN sub-layer's operators (test infrastructure only;
shares no code with the HIP path): the block norm and its gradients, row
quantisation, the 8-bit product, and the products grouped by expert.

Inputs are float64 arrays holding the exact values of the device's bfloat16
or float inputs.
"""
from __future__ import annotations

import numpy as np


def _rms(v, eps):
    return 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)


def gate_rows(gate, rows_per_gate, rows):
    """gate[i // rows_per_gate] for each row, or None without a gate."""
    return None if gate is None else gate[np.arange(rows) // rows_per_gate]


def norm_forward(x, y=None, w_post=None, gate=None, w_pre=None, *, rows_per_gate=0, res_scale=1.0,
                 weight_offset=0.0, eps_post=1e-6, eps_pre=1e-6):
    """(x', u); y None: no block; w_post / w_pre None: no such norm."""
    if y is not None:
        z = y if w_post is None else y * _rms(y, eps_post) * (weight_offset + w_post)
        g = gate_rows(gate, rows_per_gate, x.shape[0])
        x = res_scale * x + (z if g is None else g * z)
    return x, None if w_pre is None else x * _rms(x, eps_pre) * (weight_offset + w_pre)


def norm_backward(dx_out, du, x_out, y=None, w_post=None, gate=None, w_pre=None, *, rows_per_gate=0,
                  res_scale=1.0, weight_offset=0.0, eps_post=1e-6, eps_pre=1e-6):
    """Gradients by the formulas, each with the magnitude that its rounding
    error scales with: {name: (value, magnitude)}."""
    n = (y if y is not None else x_out).shape[0]
    out = {}
    d = np.zeros_like(x_out if x_out is not None else y) if dx_out is None else dx_out
    dmag = np.abs(d)
    if w_pre is not None:
        r1 = _rms(x_out, eps_pre)
        xh, a = x_out * r1, du * (weight_offset + w_pre)
        d = d + r1 * (a - xh * (a * xh).mean(axis=1, keepdims=True))
        dmag = dmag + r1 * (np.abs(a) + np.abs(xh) * np.abs(a * xh).mean(axis=1, keepdims=True))
        out["dw_pre"] = (du * xh).sum(axis=0), np.abs(du * xh).sum(axis=0)
    if y is None:
        out["dx"] = d, dmag
        return out
    out["dx"] = res_scale * d, abs(res_scale) * dmag
    g = gate_rows(gate, rows_per_gate, n)
    r2 = np.ones((n, 1)) if w_post is None else _rms(y, eps_post)
    wp = 1.0 if w_post is None else weight_offset + w_post
    yh = y * r2
    if g is not None:
        terms, mags = d * yh * wp, dmag * np.abs(yh * wp)
        G = gate.shape[0]
        at = np.arange(n) // rows_per_gate
        dg, mg = np.zeros((G, y.shape[1])), np.zeros((G, y.shape[1]))
        np.add.at(dg, at, terms)
        np.add.at(mg, at, mags)
        out["dgate"] = dg, mg
        d, dmag = d * g, dmag * np.abs(g)
    if w_post is None:
        out["dy"] = d, dmag
        return out
    out["dw_post"] = (d * yh).sum(axis=0), (dmag * np.abs(yh)).sum(axis=0)
    b, bmag = d * wp, dmag * np.abs(wp)
    out["dy"] = (r2 * (b - yh * (b * yh).mean(axis=1, keepdims=True)),
                 r2 * (bmag + np.abs(yh) * (bmag * np.abs(yh)).mean(axis=1, keepdims=True)))
    return out


def quantize_rows(x32):
    """(q, scale) of float32 rows, in the float32 steps the interface states."""
    x32 = np.asarray(x32, dtype=np.float32)
    q = np.zeros(x32.shape, dtype=np.int8)
    scale = np.zeros(x32.shape[0], dtype=np.float32)
    for i, row in enumerate(x32):
        if not np.isfinite(row).all():
            scale[i] = np.nan
            continue
        amax = np.abs(row).max()
        if amax > 0:
            scale[i] = amax / np.float32(127)
            q[i] = np.rint(row * (np.float32(127) * (np.float32(1) / amax))).astype(np.int8)
    return q, scale


def q8_product(q, scale, w, w_scale, bias=None):
    """The exact value in float64 (the integer sum is exact)."""
    acc = q.astype(np.int64) @ w.astype(np.int64).T
    y = acc.astype(np.float64) * scale.astype(np.float64)[:, None] * w_scale.astype(np.float64)
    return y if bias is None else y + bias


def grouped(op, A, B, offsets, N, K):
    """{NN, NT: C rows (NaN where a row is in no group); TN: C per expert} and
    the sums of magnitudes."""
    E = len(offsets) - 1
    shape = (E, K, N) if op == "TN" else (A.shape[0], N)
    C = np.zeros(shape) if op == "TN" else np.full(shape, np.nan)
    mag = np.zeros(shape)
    for e in range(E):
        s = slice(int(offsets[e]), int(offsets[e + 1]))
        if op == "TN":
            C[e], mag[e] = A[s].T @ B[s], np.abs(A[s]).T @ np.abs(B[s])
        else:
            Be = B[e] if op == "NN" else B[e].T
            C[s], mag[s] = A[s] @ Be, np.abs(A[s]) @ np.abs(Be)
    return C, mag
