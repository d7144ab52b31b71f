"""GPU: attention as a serving program calls it: prompts' pieces beside single
tokens in one call, tables wider than any context, streams other than the
current one with working memory of their own, pieces long enough for every part of
the many-rows kernel's ring to be filled and read again.  Tolerances are those of
test_gpu_attn."""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests import test_gpu_attn as ta
from tests.gpu_common import announce, bf16_dev, dev, f32_dev, u8_dev

pytestmark = pytest.mark.gpu


def device(c):
    """Cache, table, lengths and offsets on the device, in the order of the helper."""
    return [u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"])] + \
        [torch.from_numpy(c[n]).to(dev()) for n in ("tab", "kv_len", "off")]


def needs_ws(c, max_q):
    T, hq, d = c["q"].shape
    B, width = c["tab"].shape
    return fp8bs.fp8bs_attn_paged_ws(B, T, max_q, hq, c["kc"].shape[1], d, width, c["kc"].shape[2])


@pytest.mark.parametrize("d,page,hq,hkv", [(64, 16, 8, 2), (64, 32, 4, 4), (128, 64, 8, 2), (128, 16, 7, 1)])
@pytest.mark.parametrize("shared", [True, False])
def test_a_piece_beside_single_tokens(d, page, hq, hkv, shared):
    """One tile height serves the whole call; its items lie on the shared line, or
    are whole where more tiles than the line holds are asked for."""
    rng = np.random.default_rng(d + page)
    few = 40 if shared else 2100
    lens = rng.integers(1, 2500 if shared else 60, few).tolist() + [2900, 600, 0]
    new = [1] * few + [300, 77, 0]
    order = rng.permutation(len(lens))
    c = ta.make(d + page + few, [lens[i] for i in order], [new[i] for i in order], hq, hkv, d, page)
    assert (needs_ws(c, 300) > 0) == shared
    ta.check(c, name="mixed")
    ta.check(c, window=130, name="mixed, window")


@pytest.mark.parametrize("new", [[1, 1, 1, 1], [3, 1, 0, 2], [100, 70, 1, 0]])
@pytest.mark.parametrize("d,page", [(64, 32), (128, 64)])
@pytest.mark.parametrize("width", [200, 4000])
def test_a_table_wider_than_the_contexts(new, d, page, width):
    """The table's other entries name no page; short contexts then lie on the shared
    line too."""
    c = ta.make(width + d + new[0], [700, 90, 33, 1200], new, 8, 2, d, page, width=width)
    assert needs_ws(c, max(new)) > 0
    ta.check(c)
    ta.check(c, causal=False, window=50)


@pytest.mark.parametrize("new", [[1, 1], [2, 3], [70, 90]])
def test_streams_with_working_memory(new):
    """The helper's working memory belongs to the stream of the call: what is
    allocated on the current stream right after the call does not get it."""
    c = ta.make(sum(new), [4000, 900], new, 4, 2, 64, 32)
    need = needs_ws(c, max(new))
    assert need > 0
    q, a = bf16_dev(c["q"]), device(c)
    want, lse = fp8bs.attn_paged(q, *a, max_q=max(new), with_lse=True)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    announce(f"attn on another stream, rows {new}, working memory {need}")
    for stream in (st, st.cuda_stream):
        torch.cuda._sleep(1000000)     # the current stream is busy: its memory is not yet free
        for kw in (dict(), dict(with_lse=True), dict(ws=torch.empty(need, dtype=torch.uint8, device=dev()))):
            got = fp8bs.attn_paged(q, *a, max_q=max(new), stream=stream, **kw)
            over = [torch.full((need,), 255, dtype=torch.uint8, device=dev()) for _ in range(4)]
            st.synchronize()
            if kw.get("with_lse"):
                got, l = got
                assert torch.equal(l, lse)
            assert torch.equal(got, want)
            del over
    torch.cuda.synchronize()


@pytest.mark.parametrize("d,page,hkv,n", [(64, 64, 96, 40009), (64, 128, 96, 40009), (128, 64, 64, 40009), (64, 32, 96, 20009),
                                          (128, 16, 64, 10009)])
def test_the_ring_is_gone_round_twice(d, page, hkv, n):
    """As many equal items as workers, so that a piece is a whole item: n keys pass
    the ring's 256 groups of 16 to 64 keys at least twice, both of its halves filled again
    and read.  Sampled heads against binary64 on the GPU."""
    B, q = 8, 70      # times heads: three or two workers a compute unit
    assert n > 2 * 256 * min(page, 64)
    g = torch.Generator(device=dev())
    g.manual_seed(d + page)
    per = -(-n // page)
    codes = lambda: torch.randint(0, 127, (per, hkv, page, d), generator=g, device=dev(), dtype=torch.uint8)  # noqa: E731
    kc, vc = codes(), codes()
    vc ^= (torch.rand(vc.shape[:3], generator=g, device=dev()) < 0.5)[..., None].to(torch.uint8) * 128
    ks, vs = ((torch.rand((per, hkv), generator=g, device=dev()) + 0.5) * 2.0 ** -9 for _ in range(2))
    tab = torch.stack([torch.randperm(per, generator=g, device=dev()) for _ in range(B)]).int()    # the pages are shared
    qq = torch.randn((B * q, hkv, d), generator=g, device=dev()).bfloat16()
    off = torch.arange(0, B * q + 1, q, dtype=torch.int32, device=dev())
    kv = torch.full((B,), n, dtype=torch.int32, device=dev())
    announce(f"attn ring: {B} x {q} rows over {n}, {hkv} heads of {d}, pages of {page}")
    out = fp8bs.attn_paged(qq, kc, ks, vc, vs, tab, kv, off, q)
    scale = d ** -0.5
    for b, h in ((0, 0), (3, hkv // 2), (7, hkv - 1)):
        ids = tab[b].long()
        deco = lambda c, s: (c[ids, h].view(torch.float8_e4m3fn).double() * s[ids, h].double()[:, None, None]).reshape(-1, d)[:n]  # noqa: E731
        k, v = deco(kc, ks), deco(vc, vs)
        x = qq[b * q:(b + 1) * q, h].double()
        sc = x @ k.t().contiguous() * scale
        p = torch.softmax(sc.masked_fill(torch.arange(n, device=dev()) > (n - q + torch.arange(q, device=dev()))[:, None],
                                         float("-inf")), -1)
        want, mag = p @ v, p @ v.abs()
        E = (d + 16) * 2.0 ** -24 * (x.abs() @ k.abs().t().contiguous()).max() * scale + 2.0 ** -20
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * E) * mag + n * 2.0 ** -33 * 448 * vs.max()
        got = out[b * q:(b + 1) * q, h].double()
        assert bool(((got - want).abs() <= tol).all()), (b, h, float((got - want).abs().max()))
