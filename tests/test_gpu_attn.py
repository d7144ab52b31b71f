"""GPU: attention over the paged E4M3 cache against binary64.

Tolerance of an output, derived from the arithmetic: half a BF16 step of the
value (2^-8 of it) for its one rounding; each weight is rounded to FP16 (2^-11
of it, or 2^-25 where it is small: the largest weight is held at 2^8 or
more, which makes 2^-33 of a largest value a key); and each score carries FP32
rounding, (D + 16) 2^-24 of scale sum |q||k| plus 2^-20 for the exponential
and logarithm, twice that in a normalised weight:
  2^-8 |o| + (2^-11 + 2 E) sum p|v| + n 2^-33 448 max vs,  E = (D+16) 2^-24 S + 2^-20
and E plus 2^-22 |lse| for the logarithm of the denominator.
"""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs, synth
from tests import attn_ref as ref
from tests.gpu_common import announce, bf16_dev, dev, f32_dev, host, u8_dev

pytestmark = pytest.mark.gpu


def make(seed, lens, new, hq, hkv, d, page, spread=1.0, poison=True, width=None, extra=2, qscale=1.5):
    """A cache of random blocks under scales of different sizes; what no
    sequence has written holds NaN codes and NaN scales."""
    rng = np.random.default_rng(seed)
    per = [(n + page - 1) // page for n in lens]
    pages = sum(per) + extra
    kc = rng.integers(0, 256, (pages, hkv, page, d)).astype(np.uint8)
    kc[(kc & 0x7F) == 0x7F] = 0x30
    vc = rng.permutation(kc.reshape(-1)).reshape(kc.shape)
    ks = (2.0 ** rng.uniform(-9, -9 + 2 * spread, (pages, hkv))).astype(np.float32)
    vs = (2.0 ** rng.uniform(-8, -8 + 4 * spread, (pages, hkv))).astype(np.float32)
    order = rng.permutation(pages)
    tab = np.full((len(lens), width or max(1, max(per))), -7, np.int32)
    at, used = 0, np.zeros((pages, page), bool)
    for b, n in enumerate(per):
        tab[b, :n] = order[at:at + n]
        for p in range(n):
            used[order[at + p], :min(page, lens[b] - p * page)] = True
        at += n
    if poison:
        kc[~used.any(1)[:, None, None, None] & np.ones_like(kc, bool)] = 0x7F
        kc.swapaxes(1, 2)[~used] = 0x7F
        vc.swapaxes(1, 2)[~used] = 0xFF
        ks[~used.any(1)] = np.nan
        vs[~used.any(1)] = np.nan
    T = sum(new)
    q = synth.bf16_bits((qscale * rng.standard_normal((T, hq, d))).astype(np.float32))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    return dict(q=q, kc=kc, ks=ks, vc=vc, vs=vs, tab=tab, kv_len=np.array(lens, np.int32), off=off)


def check(c, scale=None, causal=True, window=0, max_q=None, no_off=False, name=""):
    D, page = c["kc"].shape[3], c["kc"].shape[2]
    scale = D ** -0.5 if scale is None else scale
    announce(f"attn {name} lens {c['kv_len'].tolist()[:8]} rows {np.diff(c['off']).tolist()[:8]} q {c['q'].shape} "
             f"page {page} causal {causal} window {window}")
    args = [u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"]), torch.from_numpy(c["tab"]).to(dev()),
            torch.from_numpy(c["kv_len"]).to(dev()), None if no_off else torch.from_numpy(c["off"]).to(dev())]
    if max_q is None:
        max_q = max(1, int(np.diff(c["off"]).max()))
    T, Hq, _ = c["q"].shape
    out, lse = fp8bs.attn_paged(bf16_dev(c["q"]), *args, max_q=max_q, scale=scale, causal=causal, window=window,
                                with_lse=True)
    again = fp8bs.attn_paged(bf16_dev(c["q"]), *args, max_q=max_q, scale=scale, causal=causal, window=window)
    got, l = ref.bf16_values(host(out)).astype(np.float64), host(lse).astype(np.float64)
    assert np.array_equal(host(out), host(again)), "equal calls, different bits"
    want, wl, mag, sabs = ref.attention(ref.bf16_values(c["q"]).astype(np.float64), c["kc"], c["ks"], c["vc"], c["vs"],
                                        c["tab"], c["kv_len"], c["off"], scale, causal, window)
    E = (D + 16) * 2.0 ** -24 * sabs + 2.0 ** -20
    small = max(1, int(c["kv_len"].max())) * 2.0 ** -33 * 448 * np.nan_to_num(c["vs"]).max()
    tol = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2 * E[..., None]) * mag + small
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outputs off, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {want[bad][0]!r}, tolerance {tol[bad][0]:.3g}")
    empty = np.isinf(wl)
    assert np.array_equal(np.isneginf(l), empty)
    assert (np.abs(l[~empty] - wl[~empty]) <= E[~empty] + 2.0 ** -22 * np.abs(wl[~empty])).all()
    assert (got[empty] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_one_token_each(d, page):
    lens = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 1000, 0, 257]
    check(make(page + d, lens, [1] * len(lens), 8, 2, d, page), no_off=True)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (5, 5), (7, 1), (12, 4), (16, 1), (24, 1), (40, 2), (70, 1)])
def test_groups(hq, hkv):
    check(make(hq, [77, 300], [1, 1], hq, hkv, 128, 32), no_off=True)


@pytest.mark.parametrize("hq,hkv,d,new", [(8, 2, 128, [1, 5, 0, 3, 2]), (7, 1, 64, [6, 1, 9, 0, 4]),
                                          (8, 8, 128, [33, 2, 17, 65, 1]), (40, 8, 64, [40, 129, 1, 64, 0])])
@pytest.mark.parametrize("window", [0, 1, 50])
def test_several_rows(hq, hkv, d, new, window):
    lens = [n + x for n, x in zip(new, (0, 200, 11, 63, 500))]
    check(make(sum(new) + window, lens, new, hq, hkv, d, 16), window=window)


def test_whole_prompts():
    lens = [1, 130, 64, 257, 400]
    check(make(3, lens, lens, 8, 2, 128, 64))
    check(make(4, lens, lens, 10, 2, 64, 32), window=100)


def test_not_causal():
    check(make(5, [90, 33, 300], [3, 33, 40], 8, 4, 128, 16), causal=False)
    check(make(6, [90, 33, 300], [3, 33, 40], 8, 4, 64, 64), causal=False, window=20)


def test_rows_that_see_nothing():
    """More rows than tokens in the cache: the first ones see no key; an empty
    cache; a sequence without rows."""
    check(make(7, [3, 0, 5, 70], [8, 2, 0, 90], 8, 2, 128, 16))
    check(make(8, [0, 0], [1, 1], 4, 4, 64, 32), no_off=True)


def test_long_axis_is_split():
    """One sequence shared among many workers, and one long among short ones."""
    check(make(9, [20000], [1], 8, 1, 128, 64), no_off=True)
    check(make(10, [5, 9000, 40, 1], [1, 1, 1, 1], 8, 2, 64, 16), no_off=True)
    check(make(11, [7000, 300], [3, 40], 8, 1, 128, 64))


@pytest.mark.parametrize("window", [1, 100, 1400, 1600, 5000])
def test_windows_over_long_contexts(window):
    """Windows that are short and long contexts that are not, a token and several at a
    time; without causality a window bounds the keys from below only."""
    check(make(window, [7000, 2, 1500, 4001], [1, 1, 1, 1], 8, 2, 128, 32), window=window, no_off=True)
    check(make(window + 1, [6000, 33, 2500], [3, 5, 0], 10, 2, 64, 16), window=window)
    check(make(window + 2, [3000, 700], [2, 4], 4, 1, 128, 64), window=window, causal=False)


def test_scales_of_very_different_size():
    c = make(12, [900, 400], [1, 2], 8, 2, 128, 16, spread=4.0)
    c["vs"][::3] *= np.float32(2.0 ** 20)
    check(c)
    c["vc"][::2] = 0          # blocks of zero values have a zero scale
    c["vs"][::2] = 0
    check(c)


def test_peaked_and_rising_scores():
    """Scores that grow along the sequence move the softmax's reference again
    and again; one key far above the rest takes all the weight."""
    c = make(13, [600, 600], [1, 1], 4, 1, 64, 32, qscale=6.0)
    for b in range(2):
        ids = c["tab"][b, :19]
        c["ks"][ids, 0] = np.float32(2.0) ** np.linspace(-12, -4, 19).astype(np.float32)
    check(c)


def test_order_of_lengths_does_not_matter_past_the_table():
    """Lengths past what the table holds are cut to it."""
    c = make(14, [64, 128], [1, 1], 4, 2, 64, 16)
    want = dict(c)
    c = dict(c, kv_len=np.array([64, 100000], np.int32))
    a = [u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"]), torch.from_numpy(c["tab"]).to(dev())]
    x = fp8bs.attn_paged(bf16_dev(c["q"]), *a, torch.from_numpy(c["kv_len"]).to(dev()))
    y = fp8bs.attn_paged(bf16_dev(c["q"]), *a, torch.from_numpy(want["kv_len"]).to(dev()))
    assert torch.equal(x, y)


def test_many_sequences():
    """More tiles than the shared line holds: one workgroup an item."""
    rng = np.random.default_rng(15)
    lens = rng.integers(0, 40, 2100).tolist()
    check(make(15, lens, [1] * 2100, 2, 1, 64, 16), no_off=True)


@pytest.mark.parametrize("B", [65, 100, 256, 300, 700])
def test_ragged_batches_share_their_work(B):
    """Batches that fill one, two or four slots a lane, and those past them,
    with sequences without rows in between."""
    rng = np.random.default_rng(B)
    lens = np.exp(rng.uniform(0, 7, B)).astype(int)
    lens[B // 2] = 3000
    new = (rng.random(B) < 0.9).astype(int)
    new[0] = 1
    check(make(B, lens.tolist(), new.tolist(), 4, 2, 64, 16), name="ragged")
    check(make(B + 1, lens.tolist(), (2 * new).tolist(), 16, 1, 128, 32), name="ragged two rows")


def test_many_prompts_whole_items():
    """Tiles enough to fill the GPU: one workgroup an item."""
    check(make(19, [260] * 8, [260] * 8, 64, 8, 64, 16))
    check(make(20, [190, 1, 333, 260, 70, 300, 250, 320], [190, 1, 333, 260, 70, 300, 250, 320], 96, 12, 128, 64), window=77)


@pytest.mark.parametrize("d,page", [(64, 16), (64, 128), (128, 64), (128, 16), (64, 32), (128, 32)])
def test_long_prompt_pieces(d, page):
    """Contexts long enough for the many-rows kernel to go round its ring of
    page numbers and scales several times; sampled heads against binary64 on the
    GPU, with the tolerance above."""
    hkv, G, q, n = 64, 2, 128, 18000 if page >= 32 else 6000
    hq, B = hkv * G, 8
    g = torch.Generator(device=dev())
    g.manual_seed(d + page)
    lens = [n - 17 * b for b in range(B)]
    per = [(x + page - 1) // page for x in lens]
    pages = sum(per)
    kc = torch.randint(0, 127, (pages, hkv, page, d), generator=g, device=dev(), dtype=torch.uint8)
    vc = torch.randint(0, 127, (pages, hkv, page, d), generator=g, device=dev(), dtype=torch.uint8)
    vc ^= (torch.rand(vc.shape[:3], generator=g, device=dev()) < 0.5)[..., None].to(torch.uint8) * 128
    ks, vs = (torch.rand((2, pages, hkv), generator=g, device=dev()) + 0.5) * 2.0 ** -9
    ks, vs = ks.contiguous(), vs.contiguous()
    order = torch.randperm(pages, generator=g, device=dev()).int()
    tab = torch.full((B, max(per)), -1, dtype=torch.int32, device=dev())
    at = 0
    for b in range(B):
        tab[b, :per[b]] = order[at:at + per[b]]
        at += per[b]
    qq = torch.randn((B * q, hq, d), generator=g, device=dev()).bfloat16()
    off = torch.arange(0, B * q + 1, q, dtype=torch.int32, device=dev())
    kv = torch.tensor(lens, dtype=torch.int32, device=dev())
    announce(f"attn long pieces d {d} page {page}: {B} x {q} rows over {n}, {hq}/{hkv} heads")
    out = fp8bs.attn_paged(qq, kc, ks, vc, vs, tab, kv, off, q)
    scale = d ** -0.5
    for b, h in ((0, 0), (3, 77), (7, hq - 1)):
        ids = tab[b, :per[b]].long()
        deco = lambda c, s: (c[ids, h // G].view(torch.float8_e4m3fn).double()  # noqa: E731
                             * s[ids, h // G].double()[:, None, None]).reshape(-1, d)[:lens[b]]
        k, v = deco(kc, ks), deco(vc, vs)
        x = qq[b * q:(b + 1) * q, h].double()
        sc = x @ k.t().contiguous() * scale
        hide = torch.arange(lens[b], device=dev()) > (lens[b] - q + torch.arange(q, device=dev()))[:, None]
        p = torch.softmax(sc.masked_fill(hide, float("-inf")), -1)
        want, mag = p @ v, p @ v.abs()
        sabs = (x.abs() @ k.abs().t().contiguous()).max() * scale
        E = (d + 16) * 2.0 ** -24 * sabs + 2.0 ** -20
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2 * E) * mag + n * 2.0 ** -33 * 448 * vs.max()
        got = out[b * q:(b + 1) * q, h].double()
        assert bool(((got - want).abs() <= tol).all()), (b, h, float((got - want).abs().max()))


def test_strides_and_another_stream():
    """Queries and outputs as parts of wider rows, on a stream of their own."""
    c = make(16, [100, 40], [2, 3], 4, 2, 64, 32)
    wide = torch.randn((5, 11, 64), device=dev()).bfloat16()
    wide[:, 3:7] = bf16_dev(c["q"])
    res = torch.full((5, 8, 64), 3.0, dtype=torch.bfloat16, device=dev())
    a = [u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"]), torch.from_numpy(c["tab"]).to(dev()),
         torch.from_numpy(c["kv_len"]).to(dev()), torch.from_numpy(c["off"]).to(dev())]
    want = fp8bs.attn_paged(bf16_dev(c["q"]), *a, max_q=3)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    need = fp8bs.fp8bs_attn_paged_ws(2, 5, 3, 4, 2, 64, c["tab"].shape[1], 32)
    ws = torch.empty(need, dtype=torch.uint8, device=dev())
    fp8bs.fp8bs_attn_paged(wide[:, 3:7], res[:, 2:6], None, a[6], a[5], 3, a[4], *a[:4], 0.125, True, 0, ws, st)
    st.synchronize()
    assert torch.equal(res[:, 2:6], want)
    assert (res[:, :2] == 3).all() and (res[:, 6:] == 3).all()


def test_graph_replays():
    """Captured once and replayed, with eager work in between."""
    c = make(17, [900, 33, 2000], [1, 1, 1], 8, 2, 128, 64)
    a = [u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"]), torch.from_numpy(c["tab"]).to(dev()),
         torch.from_numpy(c["kv_len"]).to(dev())]
    q = bf16_dev(c["q"])
    out = torch.empty_like(q)
    ws = torch.empty(fp8bs.fp8bs_attn_paged_ws(3, 3, 1, 8, 2, 128, c["tab"].shape[1], 64), dtype=torch.uint8,
                     device=dev())
    run = lambda: fp8bs.fp8bs_attn_paged(q, out, None, None, a[5], 1, a[4], *a[:4], 0.1, True, 0, ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        q.copy_(torch.roll(q, 1, 0))
        a[5].copy_(torch.roll(a[5], 0, 0) - i)
        graph.replay()
        got = out.clone()
        run()
        assert torch.equal(got, out)
        torch.cuda.synchronize()


def test_cache_past_32_bits():
    """A cache of more than 4 GiB whose sequence lies at its far end."""
    page, hkv, d, pages = 128, 8, 128, 34000
    kc = torch.zeros((pages, hkv, page, d), dtype=torch.uint8, device=dev())
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 32
    c = make(18, [700, 90], [1, 4], 16, hkv, d, page, poison=False, extra=0)
    n = c["kc"].shape[0]
    kc[pages - n:], vc[pages - n:] = u8_dev(c["kc"]), u8_dev(c["vc"])
    ks, vs = torch.zeros((2, pages, hkv), dtype=torch.float32, device=dev())
    ks[pages - n:], vs[pages - n:] = f32_dev(c["ks"]), f32_dev(c["vs"])
    tab, far = torch.from_numpy(c["tab"]).to(dev()), torch.from_numpy(c["tab"]).to(dev()) + (pages - n)
    rest = (torch.from_numpy(c["kv_len"]).to(dev()), torch.from_numpy(c["off"]).to(dev()))
    announce("attn over a cache of %d codes" % kc.numel())
    near = fp8bs.attn_paged(bf16_dev(c["q"]), u8_dev(c["kc"]), f32_dev(c["ks"]), u8_dev(c["vc"]), f32_dev(c["vs"]), tab,
                            *rest, max_q=4)
    assert torch.equal(fp8bs.attn_paged(bf16_dev(c["q"]), kc, ks.contiguous(), vc, vs.contiguous(), far, *rest,
                                        max_q=4), near)
