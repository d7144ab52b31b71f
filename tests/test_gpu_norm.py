"""The norm with the residual's addition, quantized, and its gradient, against
binary64.

Allowances, with U = 2^-24 and V <= 2 vectors of 8 values a lane:
- rstd: a lane's chain of 8 V fused sums, 6 levels over the wave, up to 15 more
  over the waves, all of positive terms: (16 + 6 + 15) U of the sum; mean and
  eps 2 U more; root (halves it), its rounding and the quotient's 2 U: under 24 U.
- n: two products more: 26 U |n|.
- dx: a = gamma dn and u = h rstd carry U each, so the sum of a u carries
  (37 + 3) U of sum |a u| and the mean 2 U more; then two fused steps.
- dgamma: chains of rows, of workers' parts and of groups, none longer than 512 in
  all here (T / 256 rows of a worker, 4096 / 128 parts, 16 + 8 groups; or 512 / 8
  rows and 128 groups), u's rounding 2 more: all U of sum |dn u|.
"""
import math

import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.gpu_common import announce, native_loaded
from tests.moe_ref import U, check_bf16, check_f32, check_tiles, norm, randn

pytestmark = pytest.mark.gpu
EPS = 1e-6


def pad(t, extra):
    """The tensor on the GPU as a part of wider rows."""
    wide = torch.full((t.shape[0], t.shape[1] + extra), 7.0, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def rows_of(T, C, seed, scale=1.0):
    x = randn(T, C, seed=seed, scale=scale)
    x[:, ::37] *= 30
    return (x * (0.2 + torch.rand((T, 1), generator=torch.Generator().manual_seed(seed)))).bfloat16()


def gamma_of(C, kind, seed):
    g = 1 + 0.3 * randn(C, seed=seed)
    return g.bfloat16() if kind == "bf16" else g


CASES = [(1, 128, True, "bf16"), (3, 256, False, "f32"), (5, 7168, True, "bf16"), (129, 512, True, "f32"),
         (77, 640, False, "bf16"), (64, 1152, True, "bf16"), (7, 8192, True, "f32"), (9, 8320, True, "bf16"),
         (4, 16384, False, "f32"), (2049, 384, True, "f32"), (1025, 2048, True, "bf16")]


@pytest.mark.parametrize("T,C,residual,kind", CASES)
def test_norm(T, C, residual, kind):
    native_loaded()
    announce(f"norm {T}x{C} {residual} {kind}")
    x, r, gamma = rows_of(T, C, 1), rows_of(T, C, 2, 3.0), gamma_of(C, kind, 3)
    h_want = (x.float() + r.float()).bfloat16() if residual else x
    q, s, h, y, rstd = fp8bs.rmsnorm_quant_1x128(pad(x, 8), gamma.cuda(), pad(r, 24) if residual else None, EPS,
                                                 with_y=True, with_rstd=True)
    assert (h is not None) == residual
    if residual:
        assert torch.equal(h.cpu(), h_want)
    n, f = norm(h_want, gamma, EPS)
    check_f32("rstd", rstd, f, 24 * U * f)
    check_bf16("y", y, n, 26 * U * n.abs())
    check_tiles("codes", q, s, n, 26 * U * n.abs())
    # each output alone has the same bits
    q1, s1 = fp8bs.rmsnorm_quant_1x128(x.cuda(), gamma.cuda(), r.cuda() if residual else None, EPS)[:2]
    y1 = fp8bs.rmsnorm_quant_1x128(x.cuda(), gamma.cuda(), r.cuda() if residual else None, EPS, codes=False,
                                   with_y=True)[3]
    assert torch.equal(q1, q) and torch.equal(s1, s) and torch.equal(y1, y)


def test_norm_edges():
    """Rows of zeros, of one value, tiny and large ones; a zero tile."""
    native_loaded()
    C = 512
    x = torch.zeros((7, C))
    x[1, 3] = 5.0
    x[2] = 1e-20
    x[3] = randn(C, seed=5) * 1e15
    x[4] = randn(C, seed=6) * 1e-4
    x[5, :128] = 1.0
    x[6] = -1.0
    x, gamma = x.bfloat16(), gamma_of(C, "f32", 7)
    gamma[130:140] = 0.0
    announce("norm edges")
    q, s, _, y, rstd = fp8bs.rmsnorm_quant_1x128(x.cuda(), gamma.cuda(), with_y=True, with_rstd=True)
    n, f = norm(x, gamma, 1e-6)
    check_f32("rstd", rstd, f, 24 * U * f)
    check_bf16("y", y, n, 26 * U * n.abs())
    check_tiles("codes", q, s, n, 26 * U * n.abs())
    assert (s[0] == 0).all() and (s[1, 1:] == 0).all() and (q[0] & 127 == 0).all()


def test_norm_of_tiny_weights():
    """Scales below 2^-100 (the encoder's slow path) and outputs down to FP32's
    subnormals, whose products are off by up to 2^-149 each."""
    native_loaded()
    T, C = 9, 512
    announce("norm, tiny weights")
    x = rows_of(T, C, 1)
    gamma = gamma_of(C, "f32", 2) * torch.tensor([2.0 ** -60, 2.0 ** -110, 2.0 ** -125, 2.0 ** -138]).repeat_interleave(128)
    q, s, _, y, _ = fp8bs.rmsnorm_quant_1x128(x.cuda(), gamma.cuda(), with_y=True)
    n, _ = norm(x, gamma, 1e-6)
    check_bf16("y", y, n, 26 * U * n.abs() + 2.0 ** -149)
    check_tiles("codes", q, s, n, 26 * U * n.abs() + 2.0 ** -149)


@pytest.mark.parametrize("which", ["x", "r"])
@pytest.mark.parametrize("T,C", [(6, 384), (300, 4096)])
def test_norm_in_place(which, T, C):
    native_loaded()
    announce(f"norm in place of {which} {T}x{C}")
    x, r, gamma = rows_of(T, C, 1).cuda(), rows_of(T, C, 2).cuda(), gamma_of(C, "bf16", 3).cuda()
    want = fp8bs.rmsnorm_quant_1x128(x, gamma, r)
    h = x if which == "x" else r
    q, s = torch.empty_like(want[0]), torch.empty_like(want[1])
    fp8bs.fp8bs_rmsnorm_quant_1x128(x, r, gamma, 1e-6, h, q, s, None, None)
    assert torch.equal(h, want[2]) and torch.equal(q, want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("T", [1, 40, 3000])
def test_norm_writes_nothing_else(T):
    native_loaded()
    C = 256
    announce(f"norm outputs in wider rows, T {T}")
    x, r, gamma = rows_of(T, C, 1).cuda(), rows_of(T, C, 2).cuda(), gamma_of(C, "bf16", 3).cuda()
    wide = {"h": torch.full((T + 1, C + 8), 3.0, dtype=torch.bfloat16, device="cuda"),
            "q": torch.full((T + 1, C + 16), 0x5A, dtype=torch.uint8, device="cuda"),
            "s": torch.full((T + 1, 5), -1.0, device="cuda"),
            "y": torch.full((T + 1, C + 24), 3.0, dtype=torch.bfloat16, device="cuda"),
            "rstd": torch.full((T + 1,), -1.0, device="cuda")}
    fp8bs.fp8bs_rmsnorm_quant_1x128(x, r, gamma, EPS, wide["h"][:T, :C], wide["q"][:T, :C], wide["s"][:T, :2],
                                    wide["y"][:T, :C], wide["rstd"][:T])
    want = fp8bs.rmsnorm_quant_1x128(x, gamma, r, EPS, with_y=True, with_rstd=True)
    for (name, w), t in zip((("q", C), ("s", 2), ("h", C), ("y", C)), want):
        assert torch.equal(wide[name][:T, :w], t), name
        rest = wide[name].clone()
        rest[:T, :w] = rest[T, 0]
        assert (rest == rest[T, 0]).all(), name
    assert torch.equal(wide["rstd"][:T], want[4]) and wide["rstd"][T] == -1


def bwd_want(dn, dres, h, gamma, rstd):
    """(dx, dgamma, allowance of dx, sum of |dn u|) in binary64."""
    dn, h, gamma, f = dn.double(), h.double(), gamma.double(), rstd.double()[:, None]
    a, u = dn * gamma, h * f
    mean = (a * u).mean(dim=1, keepdim=True)
    dx = f * (a - u * mean) + (0 if dres is None else dres.double())
    size = (a * u).abs().mean(dim=1, keepdim=True)
    err = f * (a.abs() * 2 * U + u.abs() * (42 * U * size + 3 * U * mean.abs()) + (a - u * mean).abs() * U) + dx.abs() * U
    return dx, (dn * u).sum(dim=0), err, (dn * u).abs().sum(dim=0)


BWD = [(1, 128, False, "bf16"), (511, 128, True, "bf16"), (512, 7168, True, "f32"), (513, 384, False, "f32"),
       (9000, 128, False, "bf16"), (3, 384, True, "f32"), (131, 1280, False, "bf16"), (700, 512, True, "bf16"),
       (5000, 256, True, "f32"), (513, 7168, True, "f32"), (1537, 640, False, "bf16"), (8, 8192, True, "bf16"),
       (600, 8320, True, "f32"), (3, 16384, False, "bf16")]


@pytest.mark.parametrize("T,C,dres,kind", BWD)
def test_gradient(T, C, dres, kind):
    native_loaded()
    announce(f"norm gradient {T}x{C} {dres} {kind}")
    h, dn, gamma = rows_of(T, C, 1), randn(T, C, seed=2, scale=0.01).bfloat16(), gamma_of(C, kind, 3)
    dr = randn(T, C, seed=4, scale=0.01).bfloat16() if dres else None
    rstd = norm(h, gamma, EPS)[1].float()
    dx, dgamma = fp8bs.rmsnorm_bwd(pad(dn, 8), pad(h, 16), gamma.cuda(), rstd.cuda(), pad(dr, 24) if dres else None)
    want, want_g, err, size = bwd_want(dn, dr, h, gamma, rstd)
    check_bf16("dx", dx, want, err)
    few = T <= 512
    chain = math.ceil(T / 8) + 128 if few else math.ceil(T / 256) + 32 + 24
    check_f32("dgamma", dgamma, want_g, (chain + 3) * U * size)
    # twice, without dgamma, and in place of dres: the same bits
    again = fp8bs.rmsnorm_bwd(dn.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(), dr.cuda() if dres else None)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dgamma)
    alone = fp8bs.rmsnorm_bwd(dn.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(), dr.cuda() if dres else None,
                              with_dgamma=False)
    assert torch.equal(alone[0], dx) and alone[1] is None
    if dres:
        place = dr.cuda()
        ws = torch.empty((max(1, fp8bs.fp8bs_rmsnorm_bwd_ws(T, C)),), dtype=torch.uint8, device="cuda")
        g = torch.empty((C,), device="cuda")
        fp8bs.fp8bs_rmsnorm_bwd(dn.cuda(), place, h.cuda(), gamma.cuda(), rstd.cuda(), place, g, ws)
        assert torch.equal(place, dx) and torch.equal(g, dgamma)


def test_gradient_of_nothing():
    native_loaded()
    announce("norm gradient of no rows")
    x, gamma = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda"), torch.ones(256, device="cuda")
    dx, dgamma = fp8bs.rmsnorm_bwd(x, x, gamma, torch.empty(0, device="cuda"))
    assert dx.shape == (0, 256) and (dgamma == 0).all()
    q, s, h, y, rstd = fp8bs.rmsnorm_quant_1x128(x, gamma, x)
    assert q.shape == (0, 256) and h.shape == (0, 256)


def test_gradient_against_differences():
    """The directional derivative of sum(w n) + sum(v h) against a central
    difference of the binary64 norm: for steps of 1e-5 of h its own error is
    under 1e-8 of the sums of magnitudes, against the BF16 rounding of dx."""
    native_loaded()
    T, C = 9, 384
    announce("norm gradient against differences")
    h, gamma = rows_of(T, C, 1), gamma_of(C, "f32", 2)
    w, v = randn(T, C, seed=3).bfloat16(), randn(T, C, seed=4).bfloat16()
    rstd = norm(h, gamma, EPS)[1].float()
    dx, dgamma = fp8bs.rmsnorm_bwd(w.cuda(), h.cuda(), gamma.cuda(), rstd.cuda(), v.cuda())
    way, way_g = randn(T, C, seed=5).double() * h.double().abs(), randn(C, seed=6).double()

    def value(x, g):
        return (w.double() * norm(x, g, EPS)[0]).sum() + (v.double() * x).sum()

    step = 1e-5
    slope = (value(h.double() + step * way, gamma.double()) - value(h.double() - step * way, gamma.double())) / (2 * step)
    size = (dx.cpu().double() * way).abs().sum()
    assert abs((dx.cpu().double() * way).sum() - slope) <= (2.0 ** -8 + 1e-6) * size
    slope = (value(h.double(), gamma + step * way_g) - value(h.double(), gamma - step * way_g)) / (2 * step)
    assert abs((dgamma.cpu().double() * way_g).sum() - slope) <= 1e-5 * (dgamma.cpu().double() * way_g).abs().sum()


def test_norm_past_32_bits():
    """Rows past 2^31 values: the last ones against the same rows alone."""
    native_loaded()
    T, C = 2 ** 31 // 7168 + 50, 7168
    announce(f"norm and gradient {T}x{C}")
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.empty((T, C), dtype=torch.bfloat16, device="cuda")
    part = torch.randn((1024, C), generator=g, device="cuda").bfloat16()
    for a in range(0, T, 1024):
        x[a:a + 1024] = part[:min(1024, T - a)] * (1 + a / T)
    gamma = gamma_of(C, "bf16", 1).cuda()
    q, s, h, _, rstd = fp8bs.rmsnorm_quant_1x128(x, gamma, x, with_rstd=True)
    last = x[-70:].clone()
    q1, s1, h1, _, rstd1 = fp8bs.rmsnorm_quant_1x128(last, gamma, last, with_rstd=True)
    assert torch.equal(q[-70:], q1) and torch.equal(s[-70:], s1) and torch.equal(h[-70:], h1)
    assert torch.equal(rstd[-70:], rstd1)
    del q, s
    dx = fp8bs.rmsnorm_bwd(x, h, gamma, rstd, x)[0]
    assert torch.equal(dx[-70:], fp8bs.rmsnorm_bwd(last, h1, gamma, rstd1, last, with_dgamma=False)[0])
