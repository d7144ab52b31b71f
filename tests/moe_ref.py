"""Plain references in binary64 for the operators around the experts' products,
and the checks that compare the kernels' outputs with them.

An output's allowance is an absolute error for every value, derived in the
tests from the kernels' FP32 operations (U = 2^-24 each, relative); rounding to
BF16 or E4M3 adds half a step."""
import torch

import oracle

U = 2.0 ** -24
E4M3 = torch.tensor(oracle.e4m3_table(), dtype=torch.float64)          # value of every code
_POSITIVE = E4M3[:127]                                                  # 0 .. 448, ascending
_MIDDLE = (_POSITIVE[1:] + _POSITIVE[:-1]) / 2


def randn(*shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * scale


def check_bf16(name, got, want, err):
    """got bf16 within half a BF16 step of a value within err of want (both binary64)."""
    got, want = got.cpu().double(), want.cpu()
    bad = (got - want).abs() > err + (want.abs() + err) * 2.0 ** -8 + 2.0 ** -134
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0].item()!r} against {want[bad][0].item()!r}"


def check_f32(name, got, want, err):
    got, want = got.cpu().double(), want.cpu()
    bad = (got - want).abs() > err + 2.0 ** -149
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}: " \
        f"{got[bad][0].item()!r} against {want[bad][0].item()!r}"


def check_tiles(name, q, s, want, err):
    """Codes and scales of 1x128 tiles of values within err of want: every scale is
    amax / 448 within the error of the largest value, every code the nearest
    one to some value that near, by the scale that was stored."""
    q, s, want = q.cpu().long(), s.cpu().double(), want.cpu()
    err = torch.as_tensor(err, dtype=torch.float64).expand(want.shape)
    tiles, slack = want.abs().unflatten(-1, (-1, 128)), err.unflatten(-1, (-1, 128))
    scale = tiles.amax(-1) / 448
    off = (s - scale).abs() > slack.amax(-1) / 448 + scale * 2 * U + 2.0 ** -149
    assert not off.any(), f"{name}: scales, first at {off.nonzero()[0].tolist()}: {s[off][0].item()!r} " \
        f"against {scale[off][0].item()!r}"
    by = s[..., None].expand(tiles.shape).flatten(-2)
    zero = by == 0
    assert ((q & 127)[zero] == 0).all(), f"{name}: codes of zero tiles"
    code = (q & 127).clamp(max=126)
    assert (code == (q & 127)).all(), f"{name}: NaN codes"
    low = torch.cat([torch.tensor([-float("inf")], dtype=torch.float64), _MIDDLE])[code]
    high = torch.cat([_MIDDLE, torch.tensor([float("inf")], dtype=torch.float64)])[code]
    low = torch.where(code == 0, -high, low)                            # zero of either sign
    y = want * torch.where(q > 127, -1.0, 1.0)
    slack = err + want.abs() * 2 * U
    bad = ((y + slack < low * by) | (y - slack > high * by)) & ~zero
    assert not bad.any(), f"{name}: {int(bad.sum())} codes, first at {bad.nonzero()[0].tolist()}: " \
        f"{(E4M3[q] * by)[bad][0].item()!r} for {want[bad][0].item()!r}"


def sorted_rows(ids, E, first, rows):
    """(offsets, slot) by lists: expert by expert, token by token."""
    of = [[] for _ in range(E)]
    for t, chosen in enumerate(ids.tolist()):
        for j, e in enumerate(chosen):
            if first <= e < first + E:
                of[e - first].append((t, j))
    slot = torch.full(ids.shape, -1, dtype=torch.int32)
    offsets, at = [0], 0
    for one in of:
        for t, j in one:
            if at < rows:
                slot[t, j] = at
            at += 1
        offsets.append(min(at, rows))
    return torch.tensor(offsets, dtype=torch.int32), slot


def norm(h, gamma, eps):
    """(n, rstd) in binary64 of h."""
    h = h.double()
    rstd = (h.square().mean(dim=1) + eps).rsqrt()
    return h * rstd[:, None] * gamma.double(), rstd


def swiglu_grads(dh, g, u):
    """(dg, du, h) in binary64."""
    dh, g, u = dh.double(), g.double(), u.double()
    sig = torch.sigmoid(g)
    return dh * u * (sig + g * sig * torch.sigmoid(-g)), dh * g * sig, g * sig * u
