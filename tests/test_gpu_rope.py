"""GPU: the rotary table and rotation.

The rotation is checked bit for bit against FP32 NumPy (each product and sum
rounded, the result rounded once to BF16) and, for the gradient, against the
transpose of the map and against differences.  The table is binary64 rounded
once: half an FP32 step of values up to mscale, plus the binary64 error of
the angle itself (angle * 2^-50).
"""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs, synth
from tests import attn_ref as ref
from tests.gpu_common import announce, bf16_dev, dev, f32_dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(factor=8.0), dict(base=500000.0, factor=4.0, orig_len=2048.0, hi=16.0),
                                dict(factor=32.0, orig_len=4096.0, mscale=1.25)])
@pytest.mark.parametrize("n,rot", [(1, 16), (700, 128), (200000, 64)])
def test_table(n, rot, kw):
    announce(f"rope table {n} x {rot} {kw}")
    want = ref.table(n, rot, **kw)
    mine = {dict(lo="turns_lo", hi="turns_hi").get(k, k): v for k, v in kw.items()}
    got = host(fp8bs.rope_table(n, rot, device=dev(), **mine)).astype(np.float64)
    ms = kw.get("mscale", 1.0)
    assert (np.abs(got - want) <= ms * (2.0 ** -24 + n * 2.0 ** -50)).all()


CASES = [(1, 1, 64, 64, 0), (3, 40, 128, 128, 0), (33, 5, 128, 64, 64), (17, 7, 64, 32, 8), (5, 3, 96, 48, 16),
         (9, 2, 512, 256, 256), (300, 12, 192, 64, 128)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,H,D,rot,off", CASES)
def test_rotation(T, H, D, rot, off, inverse, layout):
    rng = np.random.default_rng(T + D + rot)
    announce(f"rope {T}x{H}x{D} rot {rot}+{off} {layout} inverse {inverse}")
    bits = synth.bf16_bits(rng.standard_normal((T, H, D)).astype(np.float32) * 4)
    pos = rng.integers(0, 500, T).astype(np.int32)
    cs = ref.table(500, rot).astype(np.float32)
    want = ref.bf16_round(ref.rotate(ref.bf16_values(bits), cs[pos], rot, off, layout, inverse))
    x, p, c = bf16_dev(bits), torch.from_numpy(pos).to(dev()), f32_dev(cs)
    y = fp8bs.rope(x, p, c, rot_offset=off, layout=layout, inverse=inverse)
    assert np.array_equal(host(y), want)
    fp8bs.fp8bs_rope(x, x, p, off, layout, inverse, c)          # in place
    assert np.array_equal(host(x), want)


def test_strides_leave_the_rest_alone():
    x = torch.randn((6, 9, 64), device=dev()).bfloat16()
    y = torch.full((6, 10, 64), 2.0, dtype=torch.bfloat16, device=dev())
    pos = torch.arange(6, dtype=torch.int32, device=dev())
    cs = f32_dev(ref.table(6, 32))
    fp8bs.fp8bs_rope(x[:, 2:7], y[:, 1:6], pos, 32, "half", False, cs)
    assert torch.equal(y[:, 1:6], fp8bs.rope(x[:, 2:7].contiguous(), pos, cs, rot_offset=32))
    assert (y[:, 0] == 2).all() and (y[:, 6:] == 2).all()


def test_positions_are_cut_to_the_table():
    x = torch.randn((4, 2, 64), device=dev()).bfloat16()
    cs = f32_dev(ref.table(10, 64))
    at = lambda *p: torch.tensor(p, dtype=torch.int32, device=dev())  # noqa: E731
    assert torch.equal(fp8bs.rope(x, at(-5, 3, 9, 2000000000), cs), fp8bs.rope(x, at(0, 3, 9, 9), cs))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_gradient(layout):
    """L = sum(w * rope(x)): dL/dx is the inverse rotation of w.  The map is
    linear, so central differences of the FP64 loss are exact up to FP64
    rounding (2^-30 allowed at step 1); the kernel's gradient is its FP32
    value rounded to BF16: 2^-8 of it plus 2^-22 of the magnitudes summed."""
    rng = np.random.default_rng(2)
    T, H, D, rot, off = 4, 2, 64, 48, 16
    x = rng.standard_normal((T, H, D))
    wb = synth.bf16_bits(rng.standard_normal((T, H, D)).astype(np.float32))
    w = ref.bf16_values(wb).astype(np.float64)
    pos = np.array([0, 7, 123, 499])
    cs = ref.table(500, rot).astype(np.float32)
    loss = lambda z: (w * ref.rotate(z, cs[pos].astype(np.float64), rot, off, layout)).sum()  # noqa: E731
    grad = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[i] = 1.0
        grad[i] = (loss(x + e) - loss(x - e)) / 2
    formula = ref.rotate(w, cs[pos].astype(np.float64), rot, off, layout, inverse=True)
    assert (np.abs(grad - formula) <= 2.0 ** -30).all()
    got = host(fp8bs.rope(bf16_dev(wb), torch.tensor(pos, dtype=torch.int32, device=dev()), f32_dev(cs),
                          rot_offset=off, layout=layout, inverse=True))
    mag = 2 * np.abs(w).max()
    assert (np.abs(ref.bf16_values(got) - formula) <= 2.0 ** -8 * np.abs(formula) + 2.0 ** -22 * mag).all()


def test_forward_then_inverse_is_the_identity():
    """Two BF16 roundings and FP32 arithmetic: 2^-7 of the pair's length."""
    x = torch.randn((50, 4, 128), device=dev()).bfloat16()
    pos = torch.arange(50, dtype=torch.int32, device=dev())
    cs = fp8bs.rope_table(50, 128, device=dev())
    back = fp8bs.rope(fp8bs.rope(x, pos, cs), pos, cs, inverse=True).double()
    length = (x.double()[..., :64] ** 2 + x.double()[..., 64:] ** 2).sqrt().repeat(1, 1, 2)
    assert ((back - x.double()).abs() <= 2.0 ** -7 * length).all()


def test_past_32_bits():
    """More than 2^31 values: the last rows equal a small call's."""
    T, H, D = 140000, 128, 128
    assert T * H * D > 2 ** 31
    x = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev())
    x.copy_(torch.randn((1, H, D), device=dev()).bfloat16())
    pos = (torch.arange(T, device=dev()) % 1000).int()
    cs = fp8bs.rope_table(1000, 128, device=dev())
    y = fp8bs.rope(x, pos, cs)
    assert torch.equal(y[-1000:], fp8bs.rope(x[-1000:], pos[-1000:].contiguous(), cs))
    assert torch.equal(y[:1000], fp8bs.rope(x[:1000], pos[:1000].contiguous(), cs))
