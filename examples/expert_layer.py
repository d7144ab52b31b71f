#!/usr/bin/env python3
"""One layer of experts, forward and backward, on one MI355X.

The norm with the residual's addition, the router's choice (torch), tokens
sorted by expert, the two grouped FP8 products with SwiGLU between them, and
the weighted way back onto the residual; then the gradient of all of it down to
the layer's inputs, the norm's weights and the router's weights.  Quantization is
passed by the gradient unchanged.  The gradients of the experts' weights are not
computed here.

    python examples/expert_layer.py [--tokens 4096] [--hidden 2048] [--experts 16]

It prints the time of the forward and of the backward pass.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fp8_fine_grained_fp8bs_amd import fp8bs  # noqa: E402


def quantized(w):
    """Expert weights bf16 [E][N][K]: codes and scales, and those of the transposes."""
    q, s = zip(*(fp8bs.quant_w_128x128(x) for x in w))
    qt, st = zip(*(fp8bs.transpose_w_128x128(*x) for x in zip(q, s)))
    return tuple(torch.stack(x) for x in (q, s, qt, st))


class ExpertLayer:
    def __init__(self, hidden=2048, inner=1024, experts=16, choices=4, seed=0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        draw = lambda *n: torch.randn(n, generator=g, device="cuda").mul_(n[-1] ** -0.5).bfloat16()  # noqa: E731
        self.inner, self.experts, self.choices = inner, experts, choices
        self.gamma = 1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")
        self.router = draw(experts, hidden)
        self.up = quantized(draw(experts, 2 * inner, hidden))        # gate and up halves
        self.down = quantized(draw(experts, hidden, inner))

    def forward(self, x, residual):
        """x, residual bf16 [T][hidden] -> (the new residual stream, what the backward pass needs)."""
        q, s, h, n, rstd = fp8bs.rmsnorm_quant_1x128(x, self.gamma, residual, with_y=True, with_rstd=True)
        top, ids = (n.float() @ self.router.float().t()).topk(self.choices, dim=1)
        w = top.softmax(dim=1)
        rows, rows_s, _, offsets, slot = fp8bs.moe_dispatch(q, ids, self.experts, s_in=s)
        up = fp8bs.grouped_gemm(rows, rows_s, *self.up[:2], offsets)
        y = fp8bs.grouped_gemm(*fp8bs.swiglu_quant_1x128(up[:, :self.inner], up[:, self.inner:]), *self.down[:2], offsets)
        out = fp8bs.moe_combine(y, slot, w, add=h)
        return out, dict(h=h, rstd=rstd, ids=ids, w=w, offsets=offsets, slot=slot, up=up, y=y, rows=rows, rows_s=rows_s)

    def backward(self, dout, kept):
        """Gradient of the residual stream -> that of x and of residual (the same),
        of gamma, and of the router's weights; and what lies between."""
        offsets, slot, w, ids = (kept[n] for n in ("offsets", "slot", "w", "ids"))
        gate, up = kept["up"][:, :self.inner], kept["up"][:, self.inner:]
        q, s, _, dw = fp8bs.moe_combine_bwd(dout, slot, w, kept["y"])
        dh = fp8bs.grouped_gemm(q, s, *self.down[2:], offsets)
        q2, s2, _, _ = fp8bs.swiglu_bwd_quant_1x128(dh, gate, up)
        drows = fp8bs.grouped_gemm(q2, s2, *self.up[2:], offsets)
        # through the router: softmax over the chosen ones, a product with its weights
        dtop = w * (dw - (w * dw).sum(dim=1, keepdim=True))
        dlogits = torch.zeros((len(dout), self.experts), device="cuda").scatter_(1, ids, dtop)
        dn = fp8bs.moe_combine(drows, slot, add=(dlogits @ self.router.float()).bfloat16())
        dx, dgamma = fp8bs.rmsnorm_bwd(dn, kept["h"], self.gamma, kept["rstd"], dres=dout)
        n = kept["h"].float() * kept["rstd"][:, None] * self.gamma
        drouter = dlogits.t() @ n
        return dx, dgamma, drouter, dict(dw=dw, q=q, s=s, dh=dh, q2=q2, s2=s2, drows=drows, dlogits=dlogits, dn=dn)


def run(tokens=4096, hidden=2048, inner=1024, experts=16, choices=4, verbose=True):
    layer = ExpertLayer(hidden, inner, experts, choices)
    x, residual = (torch.randn((tokens, hidden), device="cuda").bfloat16() for _ in range(2))
    dout = (0.01 * torch.randn((tokens, hidden), device="cuda")).bfloat16()

    def timed(f):
        f()                                     # a first call loads the kernels
        torch.cuda.synchronize()
        t = time.perf_counter()
        y = f()
        torch.cuda.synchronize()
        return y, (time.perf_counter() - t) * 1e6

    (out, kept), t_forward = timed(lambda: layer.forward(x, residual))
    grads, t_backward = timed(lambda: layer.backward(dout, kept))
    if verbose:
        print(f"{tokens} tokens of {hidden}, {choices} of {experts} experts of {inner}: "
              f"forward {t_forward:.0f} us, backward {t_backward:.0f} us")
    return layer, x, residual, dout, out, kept, grads


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--choices", type=int, default=4)
    a = ap.parse_args()
    run(a.tokens, a.hidden, a.inner, a.experts, a.choices)
