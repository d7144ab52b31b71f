"""GPU: the example's layer of experts, the operators in a run together: every step
of the forward and the backward pass against binary64 on what the step before
it gave, and the whole captured into a graph.

Allowances: those of the operators' own tests; a grouped product within 1e-3 of
the sum of its terms' magnitudes (the bar of the products here) and half a BF16
step."""
import importlib.util
import os

import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.gpu_common import announce
from tests.moe_ref import E4M3, U, check_bf16, check_f32, check_tiles, norm, sorted_rows, swiglu_grads
from tests.test_gpu_norm import bwd_want
from tests.test_gpu_swiglu_bwd import allowances

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(q, s):
    """What codes with 1x128 scales stand for."""
    return E4M3[q.cpu().long()] * s.cpu().double().repeat_interleave(128, dim=1)


def weights(q, s):
    """What expert codes with 128x128 scales stand for."""
    s = s.cpu().double().repeat_interleave(128, dim=1)[:, :q.shape[1]].repeat_interleave(128, dim=2)
    return E4M3[q.cpu().long()] * s


def check_product(name, got, a, w, offsets):
    for e in range(len(w)):
        rows = slice(int(offsets[e]), int(offsets[e + 1]))
        check_bf16(f"{name} of expert {e}", got[rows], a[rows] @ w[e].t(), 1e-3 * (a[rows].abs() @ w[e].abs().t()))


@pytest.mark.parametrize("tokens,hidden,inner,experts,choices", [(37, 256, 128, 5, 2), (300, 384, 256, 8, 3), (1, 128, 128, 2, 1)])
def test_every_step(tokens, hidden, inner, experts, choices):
    announce(f"expert layer: {tokens} tokens of {hidden}, {choices} of {experts} experts of {inner}")
    layer, x, residual, dout, out, kept, (dx, dgamma, drouter, t) = example().run(tokens, hidden, inner, experts, choices,
                                                                                verbose=False)
    h = (x.float() + residual.float()).bfloat16()
    assert torch.equal(h, kept["h"])
    n, f = norm(h.cpu(), layer.gamma.cpu(), 1e-6)
    check_f32("rstd", kept["rstd"], f, 24 * U * f)
    offsets, slot = sorted_rows(kept["ids"].cpu(), experts, 0, tokens * choices)
    assert torch.equal(offsets, kept["offsets"].cpu()) and torch.equal(slot, kept["slot"].cpu())
    token = torch.empty(tokens * choices, dtype=torch.long)
    token[slot.long().flatten()] = torch.arange(tokens).repeat_interleave(choices)
    check_tiles("rows", kept["rows"], kept["rows_s"], n[token], 26 * U * n[token].abs())
    up_w, down_w = weights(*layer.up[:2]), weights(*layer.down[:2])
    check_product("up", kept["up"], values(kept["rows"], kept["rows_s"]), up_w, offsets)
    gate, up = kept["up"][:, :inner], kept["up"][:, inner:]
    check_product("down", kept["y"], values(*fp8bs.swiglu_quant_1x128(gate, up)), down_w, offsets)
    y, w, at = kept["y"].cpu().double(), kept["w"].cpu().double(), slot.long()
    terms = y[at] * w[..., None]
    check_bf16("out", out, terms.sum(1) + h.cpu().double(),
               (choices + 1) * U * (terms.abs().sum(1) + h.cpu().double().abs()))
    # and back
    d = dout.cpu().double()
    check_f32("dw", t["dw"], (d[:, None] * y[at]).sum(2), 64 * U * (d[:, None] * y[at]).abs().sum(2))
    grad = torch.empty_like(y)
    grad[at.flatten()] = (d[:, None] * w[..., None]).flatten(0, 1)
    check_tiles("dy", t["q"], t["s"], grad, 4 * U * grad.abs())
    check_product("dh", t["dh"], values(t["q"], t["s"]), down_w.transpose(1, 2), offsets)
    dh, g, u = (z.cpu() for z in (t["dh"], gate, up))
    dg, du, _ = swiglu_grads(dh, g, u)
    eg, eu, _ = allowances(dh, g, u)
    check_tiles("dg, du", t["q2"], t["s2"], torch.cat([dg, du], 1), torch.cat([eg, eu], 1))
    check_product("drows", t["drows"], values(t["q2"], t["s2"]), up_w.transpose(1, 2), offsets)
    terms = torch.cat([t["drows"].cpu().double()[at], (t["dlogits"] @ layer.router.float()).bfloat16().cpu().double()[:, None]], 1)
    check_bf16("dn", t["dn"], terms.sum(1), (choices + 1) * U * terms.abs().sum(1))
    want, want_g, err, size = bwd_want(t["dn"].cpu(), dout.cpu(), h.cpu(), layer.gamma.cpu(), kept["rstd"].cpu())
    check_bf16("dx", dx, want, err)
    check_f32("dgamma", dgamma, want_g, (tokens / 8 + 132) * U * size)


@pytest.mark.parametrize("tokens", [40, 700, 1100])
def test_captured(tokens):
    """The whole of it in a graph, replayed on new inputs with eager work between
    the replays: the eager pass's bits every time.  (The three token counts take
    the sort's three forms.)"""
    announce(f"expert layer captured, {tokens} tokens")
    layer = example().ExpertLayer(256, 128, 12, 8)
    x, residual, dout = (torch.empty((tokens, 256), dtype=torch.bfloat16, device="cuda") for _ in range(3))

    def fill(seed):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        for t in (x, residual, dout):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))

    def whole():
        out, kept = layer.forward(x, residual)
        dx, dgamma, drouter, t = layer.backward(dout, kept)
        return [out, kept["offsets"], kept["slot"], kept["rows"], kept["rows_s"], t["dw"], t["q"], t["s"], t["q2"], t["s2"],
                t["dn"], dx, dgamma]

    fill(0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        whole()
    torch.cuda.current_stream().wait_stream(st)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = whole()
    for seed in (1, 2, 3):
        fill(seed)
        want = whole()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b)
