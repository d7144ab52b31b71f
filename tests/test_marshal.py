"""The binding's compiled short way into the attention operators: it takes what
the binding's own checks take, and turns everything else back (None), so that
those checks say what is wrong.  CPU: all of these are turned back before a
tensor's memory is looked at.  GPU: both ways give the same bits."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs

NAMES = ("fp8bs_rope", "fp8bs_kv_append", "fp8bs_attn_paged")


def arguments(dev, name, seed=0):
    """Valid arguments after the entry point's address."""
    g = torch.Generator().manual_seed(seed)
    B, page, hq, hkv, d = 3, 16, 4, 2, 64
    heads = torch.randn((B, hq + 2 * hkv, d), generator=g).bfloat16().to(dev)
    q, k, v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
    cs = torch.rand((50, d), generator=g).to(dev)
    if name == "fp8bs_rope":
        return [q, torch.arange(B, dtype=torch.int32, device=dev), cs, 0, fp8bs.ROPE_HALF, False, fp8bs._current_stream]
    kc, ks, vc, vs = fp8bs.paged_cache(B * 2, hkv, page, d, device=dev)
    table = torch.arange(B * 2, dtype=torch.int32, device=dev).view(B, 2)
    kv_len = torch.tensor([1, 17, 20], dtype=torch.int32, device=dev)
    off = torch.arange(B + 1, dtype=torch.int32, device=dev)
    if name == "fp8bs_kv_append":
        return [kc, ks, vc, vs, table, kv_len, off, k, v, q, cs, 0, fp8bs.ROPE_HALF, 1, fp8bs._current_stream]
    kc.random_(0, 120)
    vc.random_(0, 120)
    ks.fill_(2.0 ** -8)
    vs.fill_(2.0 ** -8)
    return [kc, ks, vc, vs, table, kv_len, off, fp8bs._address("fp8bs_attn_paged_ws"), q, 1, 0.125, True, 0,
            fp8bs._current_stream]


def misfits(x):
    """Replacements of one argument that no call may take."""
    if not isinstance(x, torch.Tensor):
        return ["text", object()] if isinstance(x, int) and not isinstance(x, bool) else []
    # a longer table of angles is one, and rows past the last offset are nobody's
    longer = [] if x.shape[0] == 50 or x.dtype == torch.bfloat16 else [torch.cat([x, x])]
    return [None, 3, "text", x.double(), x.unsqueeze(0), x[..., ::2]] + longer


@pytest.mark.parametrize("name", NAMES)
def test_host_tensors_and_wrong_counts_are_turned_back(name):
    a = arguments("cpu", name)
    assert fp8bs._short(name, *a) is None
    assert fp8bs._short(name, *a[:-1]) is None
    assert fp8bs._short(name, *a, 1) is None
    assert fp8bs._short(name) is None


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_misfits_are_turned_back(name):
    a = arguments("cuda", name)
    for i, x in enumerate(a):
        off = name != "fp8bs_rope" and i == 6
        for bad in misfits(x):
            if off and bad is None or (i == 4 and name != "fp8bs_rope" and isinstance(bad, torch.Tensor) and bad.shape == (3, 1)):
                continue   # one row a sequence needs no offsets; a table's rows may lie apart
            assert fp8bs._short(name, *a[:i], bad, *a[i + 1:]) is None, (name, i, bad)
        if isinstance(x, torch.Tensor):
            assert fp8bs._short(name, *a[:i], x.cpu(), *a[i + 1:]) is None, (name, i, "host")
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_both_ways_give_the_same_bits(monkeypatch):
    short = fp8bs._short
    taken = []

    def watched(name, *args):
        r = short(name, *args)
        taken.append(r is not None)
        return r

    def all_three():
        x, pos, cs, *_ = arguments("cuda", "fp8bs_rope")
        kc, ks, vc, vs, table, kv_len, off, k, v, q, _, *_ = arguments("cuda", "fp8bs_kv_append")
        y = [fp8bs.rope(x, pos, cs, layout=w, inverse=i) for w in ("half", "interleaved") for i in (False, True)]
        y.append(fp8bs.kv_append(k, v, kc, ks, vc, vs, table, kv_len, off, 1, q=q, cs=cs))
        torch.manual_seed(1)
        kc, ks, vc, vs, table, kv_len, off, _, q, *_ = arguments("cuda", "fp8bs_attn_paged")
        y += [fp8bs.attn_paged(q, kc, ks, vc, vs, table, kv_len, off), fp8bs.attn_paged(q, kc, ks, vc, vs, table, kv_len),
              fp8bs.attn_paged(q, kc, ks, vc, vs, table, kv_len, scale=0.3, causal=False, window=7)]
        return y

    monkeypatch.setattr(fp8bs, "_short", watched)
    a = all_three()
    assert taken == [True] * 8
    monkeypatch.setattr(fp8bs, "_short", lambda *_: None)
    b = all_three()
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.gpu
def test_a_refusal_of_the_library_is_raised():
    x, pos, cs, *_ = arguments("cuda", "fp8bs_rope")
    with pytest.raises(fp8bs.Fp8bsError):
        fp8bs.rope(x, pos, cs[:, :24].contiguous())     # rot not a multiple of 16
