"""CPU tests of the attention entry points: what they refuse, on the host,
before any HIP call (fake device addresses, never dereferenced), through the C
ABI and through the binding; and the plain reference the GPU tests use."""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests import attn_ref as ref

A = 0x100000
NULL = None
INV, SHAPE, ALIGN, OK = fp8bs.ERR_INVALID_ARG, fp8bs.ERR_UNSUPPORTED_SHAPE, fp8bs.ERR_MISALIGNED, fp8bs.OK
NAN = float("nan")


def rope_table(cs=A, n_pos=8, rot=64, base=1e4, factor=1.0, orig=0.0, lo=1.0, hi=32.0, mscale=1.0):
    return fp8bs.load().fp8bs_rope_table(cs, n_pos, rot, base, factor, orig, lo, hi, mscale, NULL)


def rope(x=A, ldx=256, y=A + 4096, ldy=256, pos=A, T=4, H=2, D=128, rot=64, off=0, layout=0, inverse=0, cs=A, n_pos=9):
    return fp8bs.load().fp8bs_rope(x, ldx, y, ldy, pos, T, H, D, rot, off, layout, inverse, cs, n_pos, NULL)


def append(q=A, ldq=512, qo=A, ldqo=512, Hq=4, k=A, ldk=256, v=A, ldv=256, Hkv=2, D=128, cs=A, n_pos=9, rot=64, off=0,
           layout=0, q_off=A, kv_len=A, B=3, T=4, max_q=2, table=A, ldt=5, max_pages=5, page=16, kc=A, ks=A, vc=A, vs=A,
           n_pages=7):
    return fp8bs.load().fp8bs_kv_append(q, ldq, qo, ldqo, Hq, k, ldk, v, ldv, Hkv, D, cs, n_pos, rot, off, layout, q_off,
                                        kv_len, B, T, max_q, table, ldt, max_pages, page, kc, ks, vc, vs, n_pages, NULL)


def attn(q=A, ldq=512, out=A, ldo=512, lse=A, ldl=4, q_off=A, kv_len=A, B=3, T=4, max_q=2, Hq=4, Hkv=2, D=128, table=A,
         ldt=5, max_pages=5, page=16, kc=A, ks=A, vc=A, vs=A, n_pages=7, scale=0.1, causal=1, window=0, ws=A,
         ws_bytes=1 << 40):
    return fp8bs.load().fp8bs_attn_paged(q, ldq, out, ldo, lse, ldl, q_off, kv_len, B, T, max_q, Hq, Hkv, D, table, ldt,
                                         max_pages, page, kc, ks, vc, vs, n_pages, scale, causal, window, ws, ws_bytes,
                                         NULL)


@pytest.mark.parametrize("call,expect", [
    (lambda: rope_table(n_pos=-1), INV), (lambda: rope_table(rot=0), INV), (lambda: rope_table(rot=24), SHAPE),
    (lambda: rope_table(rot=528), SHAPE), (lambda: rope_table(base=0.0), INV), (lambda: rope_table(base=NAN), INV),
    (lambda: rope_table(factor=0.0), INV), (lambda: rope_table(orig=-1.0), INV), (lambda: rope_table(mscale=NAN), INV),
    (lambda: rope_table(orig=5.0, lo=4.0, hi=4.0), INV), (lambda: rope_table(cs=NULL), INV),
    (lambda: rope_table(cs=A + 4), ALIGN), (lambda: rope_table(n_pos=0, cs=NULL), OK),
    (lambda: rope_table(n_pos=1 << 31), SHAPE),
    (lambda: rope(T=-1), INV), (lambda: rope(H=0), INV), (lambda: rope(D=120, ldx=240), SHAPE), (lambda: rope(rot=40), SHAPE),
    (lambda: rope(rot=0), INV), (lambda: rope(off=4), SHAPE), (lambda: rope(off=72), SHAPE), (lambda: rope(off=-8), INV),
    (lambda: rope(layout=2), INV), (lambda: rope(x=NULL), INV), (lambda: rope(ldx=248), INV), (lambda: rope(ldy=260), ALIGN),
    (lambda: rope(y=A + 8), ALIGN), (lambda: rope(x=A, y=A, ldy=512), INV), (lambda: rope(cs=NULL), INV),
    (lambda: rope(cs=A + 8), ALIGN), (lambda: rope(n_pos=0), INV), (lambda: rope(pos=NULL), INV),
    (lambda: rope(pos=A + 2), ALIGN), (lambda: rope(T=0, x=NULL, y=NULL, pos=NULL), OK),
    (lambda: append(Hkv=0), INV), (lambda: append(Hq=0), INV), (lambda: append(cs=NULL), INV), (lambda: append(qo=NULL), INV),
    (lambda: append(D=96, ldq=1024, ldk=1024, ldv=1024), SHAPE), (lambda: append(D=256, ldk=512, ldv=512, ldq=1024), SHAPE),
    (lambda: append(rot=24), SHAPE), (lambda: append(off=80), SHAPE), (lambda: append(layout=-1), INV),
    (lambda: append(B=-1), INV), (lambda: append(T=-1), INV), (lambda: append(max_q=0), INV), (lambda: append(q_off=NULL), INV),
    (lambda: append(page=8), SHAPE), (lambda: append(page=48), SHAPE), (lambda: append(page=256), SHAPE),
    (lambda: append(page=0), INV), (lambda: append(max_pages=0), INV), (lambda: append(n_pages=0), INV),
    (lambda: append(max_pages=1 << 28, ldt=1 << 28), SHAPE), (lambda: append(ldt=4), INV), (lambda: append(ldk=128), INV),
    (lambda: append(ldv=260), ALIGN), (lambda: append(k=A + 2), ALIGN), (lambda: append(kc=A + 8), ALIGN),
    (lambda: append(ks=A + 2), ALIGN), (lambda: append(vs=NULL), INV), (lambda: append(table=NULL), INV),
    (lambda: append(kv_len=A + 1), ALIGN), (lambda: append(n_pos=0), INV), (lambda: append(Hkv=1 << 17), SHAPE),
    (lambda: append(T=0, B=0, k=NULL, v=NULL, kc=NULL), OK),
    (lambda: attn(Hq=0), INV), (lambda: attn(Hq=5), INV), (lambda: attn(Hkv=-1), INV),
    (lambda: attn(Hq=2050, Hkv=2, ldq=1 << 19, ldo=1 << 19, ldl=4096), SHAPE), (lambda: attn(scale=0.0), INV),
    (lambda: attn(scale=NAN), INV), (lambda: attn(scale=float("inf")), INV), (lambda: attn(window=-1), INV),
    (lambda: attn(T=1 << 30, B=1 << 30, Hq=8, Hkv=2, ldq=1024, ldo=1024, ldl=8), SHAPE),
    (lambda: attn(max_pages=1 << 27, ldt=1 << 27), SHAPE), (lambda: attn(D=32), SHAPE), (lambda: attn(page=24), SHAPE), (lambda: attn(T=1 << 32), SHAPE), (lambda: attn(max_q=-1), INV),
    (lambda: attn(max_q=0), INV), (lambda: attn(q_off=NULL), INV), (lambda: attn(q=NULL), INV), (lambda: attn(out=NULL), INV),
    (lambda: attn(ldq=256), INV), (lambda: attn(ldo=516), ALIGN), (lambda: attn(q=A + 2), ALIGN), (lambda: attn(ldl=3), INV),
    (lambda: attn(lse=A + 2), ALIGN), (lambda: attn(kc=NULL), INV), (lambda: attn(vc=A + 4), ALIGN),
    (lambda: attn(q_off=A + 2), ALIGN), (lambda: attn(ldt=2), INV), (lambda: attn(ws=NULL, max_pages=500, ldt=500), INV),
    (lambda: attn(ws_bytes=16, max_pages=500, ldt=500), INV),
    (lambda: attn(ws=A + 8), ALIGN), (lambda: attn(T=0, B=0, q=NULL, ws=NULL, ws_bytes=0), OK),
])
def test_refusals(call, expect):
    assert call() == expect


def test_working_memory_sizes():
    f = fp8bs.fp8bs_attn_paged_ws
    assert f(0, 0, 1, 8, 2, 128, 10, 64) == 0
    assert f(4, 4, 1, 8, 3, 128, 10, 64) == -1 and f(4, 4, 1, 8, 2, 100, 10, 64) == -1 and f(-1, 4, 1, 8, 2, 128, 10, 64) == -1
    assert 0 < f(1, 1, 1, 8, 2, 128, 2048, 64) < 1 << 28
    assert f(5000, 5000, 1, 8, 2, 128, 1000, 64) == 0        # one workgroup an item
    assert f(4, 4, 1, 8, 2, 128, 5, 16) == 0                 # contexts too short to share


def tensors(T=4, Hq=4, Hkv=2, D=64, B=2, pages=5, page=16):
    z = torch.zeros
    return dict(q=z((T, Hq, D), dtype=torch.bfloat16), kc=z((pages, Hkv, page, D), dtype=torch.uint8),
                ks=z((pages, Hkv)), vc=z((pages, Hkv, page, D), dtype=torch.uint8), vs=z((pages, Hkv)),
                table=z((B, 3), dtype=torch.int32), kv_len=z(B, dtype=torch.int32), q_off=z(B + 1, dtype=torch.int32))


@pytest.mark.parametrize("change", [
    dict(q=torch.zeros((4, 4, 64))), dict(q=torch.zeros((4, 256), dtype=torch.bfloat16)),
    dict(q=torch.zeros((4, 64, 4), dtype=torch.bfloat16).transpose(1, 2)),
    dict(q=torch.zeros((4, 4, 128), dtype=torch.bfloat16)), dict(ks=torch.zeros((5, 3))), dict(vs=torch.zeros((5, 2)).double()),
    dict(vc=torch.zeros((5, 2, 16, 64), dtype=torch.int8)), dict(vc=torch.zeros((5, 2, 32, 64), dtype=torch.uint8)),
    dict(kc=torch.zeros((5, 2, 64, 16), dtype=torch.uint8).transpose(2, 3)), dict(table=torch.zeros((2, 3), dtype=torch.int64)),
    dict(table=torch.zeros((3, 2), dtype=torch.int32).t()), dict(kv_len=torch.zeros(3, dtype=torch.int32)),
    dict(kv_len=torch.zeros(2, dtype=torch.int64)), dict(q_off=torch.zeros(2, dtype=torch.int32)), dict(q_off=None),
    {},                                           # host tensors are refused last
])
def test_binding_refuses(change):
    t = {**tensors(), **change}
    out = torch.empty_like(t["q"])
    with pytest.raises(ValueError):
        fp8bs.fp8bs_attn_paged(t["q"], out, None, t["q_off"], t["kv_len"], 2, t["table"], t["kc"], t["ks"], t["vc"], t["vs"],
                               0.1, True, 0, None, 0)
    if "q" not in change:
        k = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
        with pytest.raises(ValueError):
            fp8bs.fp8bs_kv_append(None, None, k, k, None, 0, "half", t["q_off"], t["kv_len"], 2, t["table"], t["kc"],
                                  t["ks"], t["vc"], t["vs"], 0)


def test_binding_refuses_rope_arguments():
    x, pos, cs = torch.zeros((4, 2, 64), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros((9, 64))
    for a in ((x, x[:3], pos, 0, "half", False, cs), (x, x, pos[:2], 0, "half", False, cs), (x, x, pos, 0, "both", False, cs),
              (x, x, pos, 0, "half", False, cs.double()), (x, x, pos.long(), 0, "half", False, cs), (x, x, pos, 0, "half", False, cs)):
        with pytest.raises(ValueError):
            fp8bs.fp8bs_rope(*a, 0)


def test_reference_encoder_against_torch():
    """The reference's codes at unit scale are torch's E4M3 conversion."""
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(2000) * 100, ref.MIDS, -ref.MIDS, ref.E4M3_POS]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.encode(x, np.float32(1)), want)
    assert np.array_equal(ref.decode(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_reference_attention_against_torch():
    rng = np.random.default_rng(1)
    n, m, hq, hkv, d = 37, 5, 4, 2, 64
    kc, vc = rng.integers(0, 0x70, (2, 3, hkv, 16, d)).astype(np.uint8)
    ks, vs = rng.random((2, 3, hkv)).astype(np.float32) / 64
    q = rng.standard_normal((m, hq, d))
    tab = np.array([[2, 0, 1]])
    out, lse, _, _ = ref.attention(q, kc, ks, vc, vs, tab, [n], [0, m], 0.2)
    flat = lambda c, s: torch.from_numpy((ref.decode(c[tab[0]]) * s[tab[0]][:, :, None, None]).swapaxes(0, 1).reshape(  # noqa: E731
        hkv, -1, d)[:, :n]).repeat_interleave(2, 0)
    s = torch.from_numpy(q).transpose(0, 1) @ flat(kc, ks).transpose(1, 2) * 0.2
    s = s.masked_fill(torch.arange(n) > torch.arange(n - m, n)[:, None], -np.inf)
    assert np.allclose(out, (s.softmax(-1) @ flat(vc, vs)).transpose(0, 1).numpy(), atol=1e-12)
    assert np.allclose(lse, s.logsumexp(-1).t().numpy(), atol=1e-12)
