"""GPU: batches of more tokens than one grid has threads for (2^32 in all): the
operators by token take them in several launches.  Rows that repeat with a period
that does not divide the launches' share give outputs with the same period; sparse
batches name rows on both sides of the border between launches."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.gpu_common import announce, native_loaded

pytestmark = pytest.mark.gpu
PERIOD = 65537
NARROW = 2 ** 26 - 4      # tokens of a launch with four a workgroup of 256


@pytest.fixture(autouse=True)
def memory():
    native_loaded()
    yield
    torch.cuda.empty_cache()


def randn(*shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def repeated(t, T):
    """T rows of t again and again."""
    big = torch.empty((T,) + t.shape[1:], dtype=t.dtype, device="cuda")
    step = PERIOD * 64
    block = t.repeat((64,) + (1,) * (t.dim() - 1))
    for a in range(0, T, step):
        big[a:a + step] = block[:T - a]
    return big


def check_repeats(name, big, t):
    step = PERIOD * 64
    block = t.repeat((64,) + (1,) * (t.dim() - 1))
    for a in range(0, len(big), step):
        assert torch.equal(big[a:a + step], block[:len(big) - a]), f"{name}: rows {a} on"


def test_norm():
    T, C = NARROW + 9, 128
    announce(f"norm {T}x{C}")
    x, gamma = randn(PERIOD, C, seed=1).bfloat16(), 1 + 0.1 * randn(C, seed=2)
    big = repeated(x, T)
    out = fp8bs.rmsnorm_quant_1x128(big, gamma, big, with_rstd=True)
    for name, a, b in zip(("q", "s", "h", "y", "rstd"), out, fp8bs.rmsnorm_quant_1x128(x, gamma, x, with_rstd=True)):
        assert (a is None) == (b is None)
        if b is not None:
            check_repeats(name, a, b)


def near(T, border, n=9):
    """Tokens around the border between two launches, and the last."""
    return torch.cat([torch.arange(3), torch.arange(border - n, border + 4), torch.arange(T - 2, T)]).unique()


# BF16 and codes, four tokens a workgroup; codes of two waves a token
@pytest.mark.parametrize("T,C,border,codes", [(NARROW + 9, 128, NARROW, False), (NARROW + 9, 128, NARROW, True),
                                              (2 ** 25 + 7, 1152, 2 ** 25 - 1, True)])
def test_dispatch(T, C, border, codes):
    announce(f"dispatch {T}x{C}, {'codes' if codes else 'bf16'}")
    at, E = near(T, border), 3
    rows, some = len(at), randn(len(at), C, seed=3).bfloat16()
    scales = None
    if codes:
        some, s = fp8bs.quant_act_1x128(some)
        scales = torch.zeros((T, C // 128), device="cuda")
        scales[at.cuda()] = s
    x = torch.empty((T, C), dtype=some.dtype, device="cuda")
    x[at.cuda()] = some
    ids = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    ids[at.cuda(), 0] = torch.arange(rows, device="cuda", dtype=torch.int32) % E
    q, s, _, offsets, slot = fp8bs.moe_dispatch(x, ids, E, s_in=scales, rows=rows)
    want = fp8bs.moe_dispatch(some, ids[at.cuda()], E, s_in=None if scales is None else scales[at.cuda()], rows=rows)
    assert torch.equal(offsets, want[3]) and torch.equal(slot[at.cuda()], want[4])
    assert int((slot >= 0).sum()) == rows
    assert torch.equal(q, want[0]) and torch.equal(s, want[1])


@pytest.mark.parametrize("T,N", [(NARROW + 9, 128), (2 ** 25 + 7, 1152)])
def test_combine(T, N):
    announce(f"combine {T}x{N}")
    M = 1000
    y, w = randn(M, N, seed=4).bfloat16(), randn(PERIOD, 1, seed=5)
    slot = torch.randint(-1, M, (PERIOD, 1), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    add = randn(PERIOD, N, seed=7).bfloat16()
    big = repeated(add, T)
    check_repeats("out", fp8bs.moe_combine(y, repeated(slot, T), repeated(w, T), big), fp8bs.moe_combine(y, slot, w, add))


def test_combine_gradient():
    T, N, M = NARROW + 9, 128, 64
    announce(f"combine gradient {T}x{N}")
    at = near(T, NARROW).cuda()
    dout, w = randn(PERIOD, N, seed=8).bfloat16(), randn(PERIOD, 1, seed=9)
    big, weights = repeated(dout, T), repeated(w, T)
    y = randn(M, N, seed=10).bfloat16()
    slot = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    slot[at, 0] = torch.arange(len(at), dtype=torch.int32, device="cuda")
    out = [(torch.zeros((M, N), dtype=torch.uint8, device="cuda"), torch.zeros((M, 1), device="cuda"),
            torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")) for _ in range(2)]
    *rows, dw = fp8bs.moe_combine_bwd(big, slot, weights, y, out=out[0])
    *want, few = fp8bs.moe_combine_bwd(big[at], slot[at], weights[at], y, out=out[1])
    for a, b in zip(rows, want):
        assert torch.equal(a, b)
    assert torch.equal(dw[at], few)
    dw[at] = 0
    assert not dw.any()


def test_swiglu_gradient():
    T, I = 2 ** 28 + 3, 128      # 16 tiles of a row each a workgroup
    announce(f"swiglu gradient {T}x{I}")
    x = randn(PERIOD, I, seed=11).bfloat16()
    big = repeated(x, T)
    want = fp8bs.swiglu_bwd_quant_1x128(x, x, x, with_h=True)
    h = fp8bs.swiglu_bwd_quant_1x128(big, big, big, codes=False, with_h=True)[3]
    check_repeats("h", h, want[3])
    del h
    q, s, _, _ = fp8bs.swiglu_bwd_quant_1x128(big, big, big)
    check_repeats("q", q, want[0])
    check_repeats("s", s, want[1])
