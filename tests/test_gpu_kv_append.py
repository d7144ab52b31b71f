"""GPU: the append to the paged cache, codes and scales bit for bit against
NumPy (rotation and max-abs in binary64, an FP32 scale, nearest-even codes
decided by exact comparisons), over pages that fill
across calls, ragged prompts, scales that grow, and everything the call must
leave alone."""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs, synth
from tests import attn_ref as ref
from tests.gpu_common import announce, bf16_dev, dev, f32_dev, host, u8_dev

pytestmark = pytest.mark.gpu


def setup(seed, lens, new, hq, hkv, d, page, grow=1.0, rot=None):
    rng = np.random.default_rng(seed)
    per = [(n + page - 1) // page for n in lens]
    pages = sum(per) + 2
    kc = rng.integers(0, 256, (2, pages, hkv, page, d)).astype(np.uint8)
    kc[(kc & 0x7F) == 0x7F] = 0x41
    sc = (2.0 ** rng.uniform(-9, -6, (2, pages, hkv))).astype(np.float32)
    order, at = rng.permutation(pages), 0
    tab = np.full((len(lens), max(1, max(per))), -1, np.int32)
    for b, n in enumerate(per):
        tab[b, :n] = order[at:at + n]
        at += n
    T = sum(new)
    x = rng.standard_normal((T, hq + 2 * hkv, d)) * np.exp2(rng.integers(-2, 3, (T, 1, 1))) * grow
    return dict(kc=kc[0], vc=kc[1], ks=sc[0], vs=sc[1], tab=tab, lens=np.array(lens, np.int32),
                off=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), qkv=synth.bf16_bits(x.astype(np.float32)),
                hq=hq, hkv=hkv, cs=ref.table(1 << 14, rot or d).astype(np.float32))


def device(c):
    i32 = lambda a: torch.from_numpy(a).to(dev())  # noqa: E731
    qkv = bf16_dev(c["qkv"])
    return dict(q=qkv[:, :c["hq"]], k=qkv[:, c["hq"]:c["hq"] + c["hkv"]], v=qkv[:, c["hq"] + c["hkv"]:], kc=u8_dev(c["kc"]),
                vc=u8_dev(c["vc"]), ks=f32_dev(c["ks"]), vs=f32_dev(c["vs"]), tab=i32(c["tab"]), lens=i32(c["lens"]),
                off=i32(c["off"]), cs=f32_dev(c["cs"]))


def expect(c, rot, off, layout):
    f = ref.bf16_values(c["qkv"])
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(c["lens"], np.diff(c["off"]))]).astype(int)
    hq, hkv = c["hq"], c["hkv"]
    turn = lambda x: ref.rotate(x, c["cs"][pos].astype(x.dtype), rot, off, layout) if rot else x  # noqa: E731
    k, v = f[:, hq:].astype(np.float64)[:, :hkv], f[:, hq:].astype(np.float64)[:, hkv:]
    return ref.bf16_round(turn(f[:, :hq])), ref.append(turn(k), v, c["kc"], c["ks"], c["vc"], c["vs"], c["tab"], c["lens"], c["off"])


def check(c, off=0, layout="half", rotate=True, queries=True, no_off=False, max_q=None):
    d = device(c)
    rot = c["cs"].shape[1] if rotate else 0
    announce(f"append lens {c['lens'].tolist()[:8]} new {np.diff(c['off']).tolist()[:8]} cache {c['kc'].shape} rot {rot}+{off} "
             f"{layout}")
    q = fp8bs.kv_append(d["k"], d["v"], d["kc"], d["ks"], d["vc"], d["vs"], d["tab"], d["lens"],
                        None if no_off else d["off"], max_q or max(1, int(np.diff(c["off"]).max())),
                        q=d["q"] if queries else None, cs=d["cs"] if rotate else None, rot_offset=off, layout=layout)
    wq, (kc, ks, vc, vs) = expect(c, rot, off, layout)
    if queries:
        assert np.array_equal(host(q), wq), "queries"
    for name, got, want in (("ks", d["ks"], ks), ("vs", d["vs"], vs)):
        assert np.array_equal(host(got).view(np.uint32), want.view(np.uint32)), name
    for name, got, want in (("kc", d["kc"], kc), ("vc", d["vc"], vc)):
        bad = np.argwhere(host(got) != want)
        assert not len(bad), f"{name}: {len(bad)} codes differ, first at {bad[0]}"
    return d


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("grow", [0.02, 30.0])
def test_one_token_each(d, page, grow):
    """Into fresh pages, into the middle and the last place of one; small new
    values keep the block's scale, large ones raise it."""
    lens = [1, 2, page - 1, page, page + 1, 2 * page, 2 * page + 5, 300]
    check(setup(page + d, lens, [1] * 8, 4, 2, d, page, grow), no_off=True)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("d,rot,off", [(128, 128, 0), (128, 64, 64), (64, 16, 8), (128, 96, 32)])
def test_rotated_part(d, rot, off, layout):
    check(setup(rot, [40, 7, 90], [40, 3, 20], 6, 3, d, 32, rot=rot), off=off, layout=layout)


@pytest.mark.parametrize("page", [16, 128])
def test_prompts(page):
    """Whole prompts, pieces that start inside a page, sequences without rows."""
    check(setup(page, [1, 130, 64, 257, 20, 333], [1, 130, 64, 100, 0, 5], 5, 1, 128, page))
    check(setup(page + 1, [500, 17], [500, 16], 2, 2, 64, page))


def test_without_rotation_or_queries():
    c = setup(3, [50, 20, 5], [10, 20, 1], 2, 2, 128, 16)
    check(c, rotate=False, queries=False)
    check(c, queries=False)


def test_filling_a_page_call_by_call():
    """The cache after many one-token calls, each checked."""
    page, hkv, d = 16, 2, 64
    c = setup(4, [33], [1], 2, hkv, d, page)
    rng = np.random.default_rng(5)
    for n in range(1, 34):
        c["lens"][:] = n
        c["qkv"] = synth.bf16_bits((rng.standard_normal((1, 2 + 2 * hkv, d)) * 1.1 ** n).astype(np.float32))
        got = check(c)
        c.update(kc=host(got["kc"]), vc=host(got["vc"]), ks=host(got["ks"]), vs=host(got["vs"]))


def test_zeros_and_tiny_values():
    """All-zero tokens give zero scales and signed-zero codes; subnormal scales
    are kept."""
    c = setup(6, [20, 9, 40], [20, 9, 3], 2, 2, 64, 16)
    c["qkv"][:20, 2:] = 0x8000
    c["qkv"][20:29, 2:] = synth.bf16_bits((np.random.default_rng(1).standard_normal((9, 4, 64)) * 2.0 ** -128).astype(np.float32))
    check(c)


def test_many_sequences_are_found():
    """More sequences than one probe of the search covers."""
    rng = np.random.default_rng(7)
    new = rng.integers(0, 4, 300)
    lens = new + rng.integers(0, 30, 300) * (new > 0)
    c = setup(7, lens.tolist(), new.tolist(), 1, 1, 64, 16)
    check(c)
    check(c, max_q=1000)      # a loose bound: slots are searched, not split


def test_bad_tables_write_nothing():
    """Pages that the table does not name, or names out of range, are skipped."""
    c = setup(8, [40, 16], [40, 16], 1, 1, 64, 16)
    d = device(c)
    tab = d["tab"].clone()
    tab[0, 1], tab[0, 2], tab[1, 0] = -1, 1000000, 2 ** 31 - 1
    before = [d[n].clone() for n in ("kc", "vc", "ks", "vs")]
    fp8bs.kv_append(d["k"], d["v"], d["kc"], d["ks"], d["vc"], d["vs"], tab, d["lens"], d["off"], 40, cs=d["cs"])
    first = int(c["tab"][0, 0])
    for x, y in zip(before, (d["kc"], d["vc"], d["ks"], d["vs"])):
        keep = torch.ones(x.shape[0], dtype=torch.bool, device=dev())
        keep[first] = False
        assert torch.equal(x[keep], y[keep]) and not torch.equal(x[first], y[first])


def test_cache_past_32_bits():
    page, hkv, d, pages = 128, 8, 128, 34000
    kc, ks, vc, vs = fp8bs.paged_cache(pages, hkv, page, d, dev())
    assert kc.numel() > 2 ** 32
    k, v = torch.randn((2, 300, hkv, d), device=dev()).bfloat16()
    lens = torch.tensor([300], dtype=torch.int32, device=dev())
    off = torch.tensor([0, 300], dtype=torch.int32, device=dev())
    far = torch.tensor([[pages - 1, pages - 3, 33000]], dtype=torch.int32, device=dev())
    announce("append to a cache of %d codes" % kc.numel())
    fp8bs.kv_append(k, v, kc, ks, vc, vs, far, lens, off, 300)
    small = fp8bs.paged_cache(3, hkv, page, d, dev())
    fp8bs.kv_append(k, v, *small, torch.tensor([[0, 1, 2]], dtype=torch.int32, device=dev()), lens, off, 300)
    for big, few in zip((kc, ks, vc, vs), small):
        assert torch.equal(big[far[0].long()], few)
    assert int(kc.view(torch.int32).ne(0).sum(dtype=torch.int64)) == int(small[0].view(torch.int32).ne(0).sum())
