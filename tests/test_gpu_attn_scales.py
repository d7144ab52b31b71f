"""GPU: attention under value scales of every size: zero, tiny, huge, and side
by side.  Mixed caches are checked as in test_gpu_attn, whose tolerances hold
here too; a long context under one tiny scale has a closed form."""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests import test_gpu_attn as ta
from tests.gpu_common import announce, dev, host

pytestmark = pytest.mark.gpu

# tokens of the call, a sequence each: few rows, two groups of them, many
ROWS = [1, 20, 70]


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale_log2", [-99, None])
def test_long_context_under_one_tiny_scale(rows, d, scale_log2):
    """Keys of zeros: every weight is the same, the output is the mean of the
    values and lse the logarithm of their number.  Scales of zero (None) are taken
    as 2^-100.  The denominator in units of the scale, 2^99 and more
    a key, would pass FP32's range here.

    Tolerance: half a BF16 step; weights are powers of two, exact; the FP32 sums
    of at most 2^12 values a lane and their joins are off by 2^-24 a sum, 2^-12 of
    the mean of |v|; so is the denominator, in lse 2^-12."""
    n, page = 3_000_000, 128
    pages = -(-n // page)
    g = torch.Generator(device=dev())
    g.manual_seed(rows + d)
    kc = torch.zeros((pages, 1, page, d), dtype=torch.uint8, device=dev())
    vc = torch.randint(0, 127, kc.shape, generator=g, device=dev(), dtype=torch.uint8)
    vc ^= (torch.rand(kc.shape, generator=g, device=dev()) < 0.4).to(torch.uint8) * 128
    ks = torch.ones((pages, 1), device=dev())
    vs = torch.full((pages, 1), 0.0 if scale_log2 is None else 2.0 ** scale_log2, device=dev())
    q = torch.randn((rows, 1, d), generator=g, device=dev()).bfloat16()
    tab = torch.randperm(pages, generator=g, device=dev()).int()[None]
    kv = torch.tensor([n], dtype=torch.int32, device=dev())
    off = torch.tensor([0, rows], dtype=torch.int32, device=dev())
    announce(f"attn {rows} rows over {n} tokens, heads of {d}, value scales 2^{scale_log2}")
    out, lse = fp8bs.attn_paged(q, kc, ks, vc, vs, tab, kv, off, rows, causal=False, with_lse=True)
    v = torch.cat([vc[i.long(), 0] for i in tab[0].split(1000)]).reshape(-1, d)[:n].view(torch.float8_e4m3fn)
    mean = sum(x.double().sum(0) for x in v.split(1 << 16)) / n
    mag = sum(x.double().abs().sum(0) for x in v.split(1 << 16)) / n
    by = max(float(vs[0, 0]), 2.0 ** -100)
    assert bool(((out[:, 0].double() - mean * by).abs() <= (2.0 ** -8 * mean.abs() + 2.0 ** -12 * mag) * by).all())
    assert bool(((lse.double() - np.log(n)).abs() <= 2.0 ** -12).all()), lse


def split(seed, rows, d, page, hkv=2, n=900, **kw):
    return ta.make(seed, [n, 333], [rows, max(1, rows // 3)], 2 * hkv, hkv, d, page, **kw)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 128)])
@pytest.mark.parametrize("log2", [0, 30, 60, 75])
def test_blocks_of_zeros_beside_large_values(rows, d, page, log2):
    """Keys whose values are zeros under a zero scale count in the denominator
    however large the other blocks' scales are."""
    c = split(rows + page + log2, rows, d, page, spread=0.25)
    zero = np.random.default_rng(log2).random(c["vs"].shape) < 0.5
    c["vs"] = np.where(zero, 0, c["vs"] * np.float32(2.0 ** log2)).astype(np.float32)
    c["vc"][zero] = 0x80 * (np.arange(d) % 2)
    ta.check(c)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("d,page", [(64, 16), (64, 32), (128, 16), (128, 64)])
@pytest.mark.parametrize("low,high", [(-99, -92), (-99, -30), (-36, -28), (-99, 60), (-31, 75), (70, 100)])
def test_scales_of_a_range(rows, d, page, low, high):
    """Scales spread over a range, and scores that rise along the sequence, so
    that the softmax's reference moves again and again."""
    c = split(rows + page + abs(low), rows, d, page, qscale=4.0)
    rng = np.random.default_rng(rows + abs(high))
    c["vs"] = np.where(np.isnan(c["vs"]), np.nan, 2.0 ** rng.uniform(low, high, c["vs"].shape)).astype(np.float32)
    for row in c["tab"]:
        ids = row[row >= 0]
        c["ks"][ids] = (2.0 ** np.linspace(-13, -7, len(ids)))[:, None].astype(np.float32)
    ta.check(c)


def test_a_scale_is_no_less_than_its_limit():
    """Scales below 2^-100 are taken as 2^-100: equal bits."""
    for rows in ROWS:
        c = split(rows, rows, 64, 32)
        got = []
        for s in (0.0, 2.0 ** -130, 2.0 ** -100):
            vs = torch.full(c["vs"].shape, s, device=dev())
            a = [ta.u8_dev(c["kc"]), ta.f32_dev(c["ks"]), ta.u8_dev(c["vc"]), vs]
            rest = [torch.from_numpy(c[n]).to(dev()) for n in ("tab", "kv_len", "off")]
            got.append(host(fp8bs.attn_paged(ta.bf16_dev(c["q"]), *a, *rest, max_q=rows)))
        assert np.array_equal(got[0], got[2]) and np.array_equal(got[1], got[2])
