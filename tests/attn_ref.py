"""Plain implementations of the attention operators for the tests: NumPy,
binary64 (or exact comparisons) from the definitions, sharing no code with
the library.
"""
from __future__ import annotations

import numpy as np

from fp8_fine_grained_fp8bs_amd import synth

E4M3_POS = np.array([(m if e == 0 else 8 + m) * 2.0 ** (max(e, 1) - 10) for e in range(16) for m in range(8)][:127])
MIDS = 0.5 * (E4M3_POS[:-1] + E4M3_POS[1:])
DEC = np.concatenate([E4M3_POS, [np.nan], -E4M3_POS, [np.nan]])


def bf16_values(bits):
    return synth.bf16_to_f32(bits)


def bf16_round(x32):
    return synth.bf16_bits(np.asarray(x32, np.float32))


def encode(x, s):
    """Nearest-even E4M3 codes of the exact quotients x / s (s one scale)."""
    x = np.asarray(x, np.float64)
    sign = (np.signbit(x).astype(np.uint8) << 7)
    if s == 0:
        return sign
    a = np.abs(x)
    t = MIDS * np.float64(s)                    # exact: 5 bits by 24
    i = np.searchsorted(t, a, side="left")      # thresholds below a
    tie = (i < len(t)) & (a == t[np.minimum(i, len(t) - 1)])
    i = i + (tie & (i % 2 == 1))
    return i.astype(np.uint8) | sign


def decode(codes):
    return DEC[codes]


def table(n, rot, base=10000.0, factor=1.0, orig_len=0.0, lo=1.0, hi=32.0, mscale=1.0):
    """Angles in binary64: [n][rot] = cos | sin."""
    f = base ** (-np.arange(rot // 2) * 2.0 / rot)
    if orig_len > 0:
        w = np.clip((orig_len * f / (2 * np.pi) - lo) / (hi - lo), 0, 1)
        f = (1 - w) * f / factor + w * f
    else:
        f = f / factor
    a = np.arange(n)[:, None] * f
    return np.concatenate([np.cos(a), np.sin(a)], 1) * mscale


def pairs(rot, off, layout):
    i = np.arange(rot // 2)
    return (off + i, off + rot // 2 + i) if layout == "half" else (off + 2 * i, off + 2 * i + 1)


def rotate(x, cs, rot, off, layout, inverse=False):
    """x [T][H][D], cs [T][rot]; in the dtype of the inputs, each product and
    sum rounded to it."""
    a, b = pairs(rot, off, layout)
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if inverse:
        s = -s
    y = x.copy()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def append_block(codes, scale, there, new):
    """One block: codes [page][D] and scale before, `there` tokens in it, new
    values [m][D] (float64) appended.  Returns (codes, scale)."""
    codes = codes.copy()
    old = np.float32(scale) if there > 0 else np.float32(0)
    s = max(old, np.float32(np.abs(new).max() / 448.0))
    if there > 0 and s > old:
        codes[:there] = encode(decode(codes[:there]) * np.float64(old), s)
    codes[there:there + len(new)] = encode(new, s)
    return codes, s


def append(k, v, kc, ks, vc, vs, tab, kv_len, off):
    """The whole cache after the call (k rotated, float64 [T][H][D])."""
    kc, ks, vc, vs = kc.copy(), ks.copy(), vc.copy(), vs.copy()
    page, H = kc.shape[2], kc.shape[1]
    for b in range(len(kv_len)):
        n, m = int(kv_len[b]), int(off[b + 1] - off[b])
        for p in range((n - m) // page, (n + page - 1) // page if m else 0):
            lo, hi = max(n - m, p * page), min(n, (p + 1) * page)
            i = tab[b, p]
            rows = slice(off[b] + lo - (n - m), off[b] + hi - (n - m))
            for h in range(H):
                kc[i, h], ks[i, h] = append_block(kc[i, h], ks[i, h], lo - p * page, k[rows, h])
                vc[i, h], vs[i, h] = append_block(vc[i, h], vs[i, h], lo - p * page, v[rows, h])
    return kc, ks, vc, vs


def attention(q, kc, ks, vc, vs, tab, kv_len, off, scale, causal=True, window=0):
    """binary64 attention; q float64 [T][Hq][D].  Returns out, lse, and what
    the tolerance needs: sum p |v|, and max_j scale sum |q||k| of each row."""
    T, Hq, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out, mag = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    lse, sabs = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for b in range(len(kv_len)):
        n, r0, r1 = int(kv_len[b]), int(off[b]), int(off[b + 1])
        ids = tab[b, :(n + page - 1) // page]
        k = (decode(kc[ids]) * ks[ids][:, :, None, None].astype(np.float64)).swapaxes(0, 1).reshape(Hkv, -1, D)[:, :n]
        v = (decode(vc[ids]) * vs[ids][:, :, None, None].astype(np.float64)).swapaxes(0, 1).reshape(Hkv, -1, D)[:, :n]
        pos = n - (r1 - r0) + np.arange(r1 - r0)
        j = np.arange(n)
        see = np.ones((r1 - r0, n), bool)
        if causal:
            see &= j <= pos[:, None]
        if window:
            see &= j > pos[:, None] - window
        some = see.any(1)
        for h in range(Hq if n else 0):
            kh, vh = k[h // G], v[h // G]
            kf, vf = np.nan_to_num(kh), np.nan_to_num(vh)
            s = np.where(see, q[r0:r1, h] @ kf.T * scale, -np.inf)
            top = np.where(some, s.max(1, initial=-np.inf), 0.0)
            e = np.exp(s - top[:, None])
            l = e.sum(1)
            p = e / np.where(some, l, 1)[:, None]
            out[r0:r1, h], mag[r0:r1, h] = p @ vf, p @ np.abs(vf)
            with np.errstate(divide="ignore"):
                lse[r0:r1, h] = np.where(some, top + np.log(l), -np.inf)
            sabs[r0:r1, h] = np.where(see, np.abs(q[r0:r1, h]) @ np.abs(kf).T * scale, 0).max(1, initial=0)
    return out, lse, mag, sabs
