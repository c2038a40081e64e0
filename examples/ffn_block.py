"""The FFN sub-layer's operators together, as a model would call them.

    python examples/ffn_block.py             # hidden size 4096, 8 experts of 1792
    python examples/ffn_block.py --small

Two passes on one GPU:

* training: block norm -> expert products (up, SiLU, down) -> block norm,
  forward and backward, with tokens already sorted by expert;
* dense serving in 8 bits: block norm with int8 output -> up-projection ->
  SiLU -> row quantisation -> down-projection, for a batch and for one token.

Each result is compared with the same computation in torch, in 32 bits.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from tensor_gemm_reduce_lds_amd import ffn as F  # noqa: E402


def rms(v):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6)


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def training(T, H, I, E, g):
    """x' = x + gate * norm(y), u = norm(x'), z = silu(u W1) W2 per expert, and
    the gradients of all of it for a given gradient of z."""
    dev, s = "cuda", torch.cuda.current_stream()
    r = lambda *n, k=1.0: (torch.randn(n, generator=g, device=dev) * k).bfloat16()  # noqa: E731
    x, y, dz = r(T, H), r(T, H), r(T, H)
    w1, w2 = r(E, H, I, k=H ** -0.5), r(E, I, H, k=I ** -0.5)
    wp = 1 + 0.1 * torch.randn(2, H, generator=g, device=dev)
    gate = torch.rand((1, H), generator=g, device=dev)
    cut = torch.sort(torch.randint(0, T + 1, (E - 1,), generator=g, device=dev)).values
    offsets = torch.cat([cut.new_zeros(1), cut, cut.new_full((1,), T)]).int()

    norm = F.BlockNormPlan(T, H, rows_per_gate=T, backward=1)
    up, down = (F.GroupedPlan(T, n, k, E, F.GROUPED_NN) for n, k in ((I, H), (H, I)))
    d_up, d_down = (F.GroupedPlan(T, n, k, E, F.GROUPED_NT) for n, k in ((H, I), (I, H)))
    dw_up, dw_down = (F.GroupedPlan(T, n, k, E, F.GROUPED_TN, out_dtype=F.F32) for n, k in ((I, H), (H, I)))

    x_out, u = torch.empty_like(x), torch.empty_like(x)
    norm.run(x, y, wp[0], gate, wp[1], x_out, u, stream=s)
    h, z = torch.empty((T, I), dtype=u.dtype, device=dev), torch.empty_like(x)
    up.run(u, w1, offsets, h, stream=s)
    a = torch.nn.functional.silu(h.float()).to(h.dtype)
    down.run(a, w2, offsets, z, stream=s)

    da, du = torch.empty_like(a), torch.empty_like(u)
    dw1, dw2 = torch.empty((E, H, I), device=dev), torch.empty((E, I, H), device=dev)
    dw_down.run(a, dz, offsets, dw2, stream=s)
    d_down.run(dz, w2, offsets, da, stream=s)
    hf = h.float()
    sg = torch.sigmoid(hf)
    dh = (da.float() * sg * (1 + hf * (1 - sg))).to(h.dtype)
    dw_up.run(u, dh, offsets, dw1, stream=s)
    d_up.run(dh, w1, offsets, du, stream=s)
    dx, dy = torch.empty_like(x), torch.empty_like(y)
    dw_post, dw_pre, dgate = (torch.empty(n, device=dev) for n in ((H,), (H,), (1, H)))
    norm.backward(None, du, x_out, y, wp[0], gate, wp[1], dx, dy, dw_post, dgate, dw_pre, stream=s)

    t = [v.float().requires_grad_() for v in (x, y, w1, w2, wp, gate)]
    tx, ty, t1, t2, tw, tg = t
    tu = rms(tx + tg * rms(ty) * tw[0]) * tw[1]
    o = offsets.tolist()
    tz = torch.cat([torch.nn.functional.silu(tu[o[e]:o[e + 1]] @ t1[e]) @ t2[e] for e in range(E)])
    tz.backward(dz.float())
    return {"z": off(z, tz.detach()), "dx": off(dx, tx.grad), "dy": off(dy, ty.grad), "dw1": off(dw1, t1.grad),
            "dw2": off(dw2, t2.grad), "dw_post": off(dw_post, tw.grad[0]), "dw_pre": off(dw_pre, tw.grad[1]),
            "dgate": off(dgate, tg.grad)}


def serving(T, H, I, g):
    """u = norm(x + norm(y)) in int8, z = silu(u W1^T) W2^T with int8 weights."""
    dev, s = "cuda", torch.cuda.current_stream()
    x, y = (torch.randn((T, H), generator=g, device=dev).bfloat16() for _ in range(2))
    wp = 1 + 0.1 * torch.randn(2, H, generator=g, device=dev)
    w, q, sc = [], [], []
    for n, k in ((I, H), (H, I)):        # weights quantised once, per channel
        w.append((torch.randn((n, k), generator=g, device=dev) * k ** -0.5).bfloat16())
        q.append(torch.empty((n, k), dtype=torch.int8, device=dev))
        sc.append(torch.empty(n, device=dev))
        F.q8_quantize(w[-1], q[-1], sc[-1], n, k, stream=s)
    norm = F.BlockNormPlan(T, H, quant=1)
    up, down = F.Q8Plan(T, I, H), F.Q8Plan(T, H, I)

    x_out, z = torch.empty_like(x), torch.empty_like(x)
    uq, us = torch.empty((T, H), dtype=torch.int8, device=dev), torch.empty(T, device=dev)
    h = torch.empty((T, I), dtype=x.dtype, device=dev)
    hq, hs = torch.empty((T, I), dtype=torch.int8, device=dev), torch.empty(T, device=dev)
    norm.run(x, y, wp[0], None, wp[1], x_out, uq, us, stream=s)
    up.run(uq, us, q[0], sc[0], None, h, stream=s)
    h = torch.nn.functional.silu(h.float()).to(h.dtype)
    F.q8_quantize(h, hq, hs, T, I, stream=s)
    down.run(hq, hs, q[1], sc[1], None, z, stream=s)

    tx = x.float() + rms(y.float()) * wp[0]
    want = torch.nn.functional.silu(rms(tx) * wp[1] @ w[0].float().t()) @ w[1].float().t()
    return {"x_out": off(x_out, tx), "z": off(z, want)}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--small", action="store_true", help="sizes that finish at once")
    a = ap.parse_args()
    H, I, T = (256, 448, 200) if a.small else (4096, 1792, 4096)
    g = torch.Generator(device="cuda").manual_seed(0)
    results = {"training": training(T, H, I, 8, g), "serving": serving(64, H, I, g), "one token": serving(1, H, I, g)}
    for name, r in results.items():
        print("%-10s" % name, "  ".join("%s %.1e" % kv for kv in r.items()))
    # bfloat16 results carry 2^-9 each, a chain of four of them about 1e-2 at
    # most; int8 activations add about 1% per quantisation
    assert all(v < 0.02 for v in results["training"].values())
    assert all(v < 0.05 for k in ("serving", "one token") for v in results[k].values())


if __name__ == "__main__":
    main()
