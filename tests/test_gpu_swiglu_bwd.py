"""SwiGLU's gradient against binary64.

Allowances, with U = 2^-24: e^-|g| is within 3 U (the hardware's 2^x one unit
in the last place, 2 U, and the reduction), 1 + e and its reciprocal (one unit, 2
U) bring sigma and 1 - sigma to under 8 U; silu and h have 9 U and 10 U; the
slope sigma + silu (1 - sigma) has 18 U of its terms' sizes, and dg two products
more; du has 10 U.
"""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.gpu_common import announce, native_loaded
from tests.moe_ref import U, check_bf16, check_tiles, randn, swiglu_grads

pytestmark = pytest.mark.gpu


def halves(T, I, seed, scale=2.0):
    x = randn(T, 2 * I, seed=seed, scale=scale)
    x[:, ::41] *= 8
    return x.bfloat16()


def allowances(dh, g, u):
    dh, g, u = dh.double(), g.double(), u.double()
    sig = torch.sigmoid(g)
    terms = sig + (g * sig * torch.sigmoid(-g)).abs()
    return (dh * u).abs() * terms * 21 * U, (dh * g * sig).abs() * 10 * U, (g * sig * u).abs() * 10 * U


@pytest.mark.parametrize("T,I", [(1, 128), (3, 384), (33, 2048), (130, 640), (2500, 256)])
def test_gradient(T, I):
    native_loaded()
    announce(f"swiglu gradient {T}x{I}")
    up, dh = halves(T, I, 1), randn(T, I, seed=2, scale=0.01).bfloat16()
    g, u = up[:, :I], up[:, I:]
    wide = torch.full((T, 2 * I + 16), 5.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :2 * I] = up
    q, s, d, h = fp8bs.swiglu_bwd_quant_1x128(dh.cuda(), wide[:, :I], wide[:, I:2 * I], with_d=True, with_h=True)
    dg, du, hw = swiglu_grads(dh, g, u)
    eg, eu, eh = allowances(dh, g, u)
    check_bf16("dg", d[:, :I], dg, eg)
    check_bf16("du", d[:, I:], du, eu)
    check_bf16("h", h, hw, eh)
    check_tiles("codes", q, s, torch.cat([dg, du], 1), torch.cat([eg, eu], 1))
    # h has the bits of the forward pass, and each output alone its own
    assert torch.equal(h, fp8bs.swiglu_quant_1x128(wide[:, :I], wide[:, I:2 * I], with_h=True)[2])
    args = dh.cuda(), wide[:, :I], wide[:, I:2 * I]
    q1, s1 = fp8bs.swiglu_bwd_quant_1x128(*args)[:2]
    assert torch.equal(q1, q) and torch.equal(s1, s)
    assert torch.equal(fp8bs.swiglu_bwd_quant_1x128(*args, codes=False, with_d=True)[2], d)
    assert torch.equal(fp8bs.swiglu_bwd_quant_1x128(*args, codes=False, with_h=True)[3], h)


def test_edge_gates():
    """Gates at zero, far out on both sides, at the slope's zero; zero rows."""
    native_loaded()
    announce("swiglu gradient, edge gates")
    T, I = 8, 256
    g, u, dh = torch.zeros((T, I)), randn(T, I, seed=1), randn(T, I, seed=2)
    g[1] = -1.2785
    g[2] = -60.0
    g[3] = 60.0
    g[4] = randn(I, seed=3) * 1e-6
    g[5] = torch.linspace(-80, 80, I)
    g[6] = 1.0
    u[6] = 0.0
    dh[7] = 0.0
    g, u, dh = g.bfloat16(), u.bfloat16(), dh.bfloat16()
    q, s, d, h = fp8bs.swiglu_bwd_quant_1x128(dh.cuda(), g.cuda(), u.cuda(), with_d=True, with_h=True)
    dg, du, hw = swiglu_grads(dh, g, u)
    eg, eu, eh = allowances(dh, g, u)
    check_bf16("dg", d[:, :I], dg, eg)
    check_bf16("du", d[:, I:], du, eu)
    check_bf16("h", h, hw, eh)
    check_tiles("codes", q, s, torch.cat([dg, du], 1), torch.cat([eg, eu], 1))
    assert (s[7] == 0).all() and (s[6, :2] == 0).all()


def test_tiny_gradients():
    """Scales below 2^-100: the encoder's slow path."""
    native_loaded()
    announce("swiglu gradient, tiny")
    T, I = 5, 256
    up, dh = halves(T, I, 1), (randn(T, I, seed=2) * 2.0 ** -112).bfloat16()
    q, s, d, _ = fp8bs.swiglu_bwd_quant_1x128(dh.cuda(), up[:, :I].cuda(), up[:, I:].cuda(), with_d=True)
    dg, du, _ = swiglu_grads(dh, up[:, :I], up[:, I:])
    eg, eu, _ = (e + 2.0 ** -149 for e in allowances(dh, up[:, :I], up[:, I:]))
    check_bf16("dg", d[:, :I], dg, eg)
    check_bf16("du", d[:, I:], du, eu)
    check_tiles("codes", q, s, torch.cat([dg, du], 1), torch.cat([eg, eu], 1))


def test_against_differences():
    """Central differences of the binary64 SwiGLU along a direction: steps of
    1e-5 leave under 1e-8 of the magnitudes, the outputs' rounding 2^-8."""
    native_loaded()
    announce("swiglu gradient against differences")
    T, I = 5, 384
    up, dh = halves(T, I, 1, 1.5), randn(T, I, seed=2).bfloat16()
    d = fp8bs.swiglu_bwd_quant_1x128(dh.cuda(), up[:, :I].cuda(), up[:, I:].cuda(), with_d=True)[2].cpu().double()
    way = randn(T, 2 * I, seed=3).double()

    def value(x):
        return (dh.double() * x[:, :I] * torch.sigmoid(x[:, :I]) * x[:, I:]).sum()

    slope = (value(up.double() + 1e-5 * way) - value(up.double() - 1e-5 * way)) / 2e-5
    assert abs((d * way).sum() - slope) <= (2.0 ** -8 + 1e-6) * (d * way).abs().sum()


def test_writes_nothing_else():
    native_loaded()
    announce("swiglu gradient in wider rows")
    T, I = 21, 384
    up, dh = halves(T, I, 1).cuda(), randn(T, I, seed=2).bfloat16().cuda()
    want = fp8bs.swiglu_bwd_quant_1x128(dh, up[:, :I], up[:, I:], with_d=True, with_h=True)
    q = torch.full((T + 1, 2 * I + 16), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full((T + 1, 9), -1.0, device="cuda")
    d = torch.full((T + 1, 2 * I + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    h = torch.full((T + 1, I + 8), 3.0, dtype=torch.bfloat16, device="cuda")
    outs = [(q, 2 * I), (s, 6), (d, 2 * I), (h, I)]
    fp8bs.fp8bs_swiglu_bwd_quant_1x128(dh, up[:, :I], up[:, I:], *(t[:T, :w] for t, w in outs))
    for (t, w), x in zip(outs, want):
        assert torch.equal(t[:T, :w], x)
        rest = t.clone()
        rest[:T, :w] = t[T, 0]
        assert (rest == t[T, 0]).all()


def test_past_32_bits():
    native_loaded()
    T, I = 2 ** 31 // 4096 + 40, 2048
    announce(f"swiglu gradient {T}x{I}")
    up = torch.empty((T, 2 * I), dtype=torch.bfloat16, device="cuda")
    part = torch.randn((4096, 2 * I), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    for a in range(0, T, 4096):
        up[a:a + 4096] = part[:min(4096, T - a)] * (1 + a / T)
    dh = up[:, :I]
    q, s, d, h = fp8bs.swiglu_bwd_quant_1x128(dh, up[:, :I], up[:, I:], with_d=True, with_h=True)
    last = up[-70:].clone()
    for a, b in zip((q, s, d, h), fp8bs.swiglu_bwd_quant_1x128(last[:, :I], last[:, :I], last[:, I:], with_d=True,
                                                              with_h=True)):
        assert torch.equal(a[-70:], b)
