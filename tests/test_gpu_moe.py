"""Tokens sorted by expert and brought back, with their gradients: the order
against lists, codes and scales bit for bit against the activation quantizer's
oracle, sums against binary64.

Allowances, with U = 2^-24: a combined value is a chain of k + 1 fused sums, so
(k + 1) U of the sum of its terms' magnitudes; a weight's gradient is a lane's
chain of 16 per 16384 columns, 6 levels over the wave and up to 15 over the waves.
"""
import math

import pytest
import torch

import oracle
from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.gpu_common import announce, host, native_loaded
from tests.moe_ref import U, check_bf16, check_f32, randn, sorted_rows

pytestmark = pytest.mark.gpu
NAN = float("nan")


def choices(T, k, of, seed, out_of_range=0.1):
    """Experts of every token, some named twice, some outside 0 .. of - 1."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, of, (T, k), generator=g)
    ids = torch.where(torch.rand((T, k), generator=g) < 0.3, torch.randint(0, 1 + of // 3, (T, k), generator=g), ids)
    odd = torch.randint(-5, 0, (T, k), generator=g)
    return torch.where(torch.rand((T, k), generator=g) < out_of_range, odd, ids)


SORTS = [(1, 1, 1, 1, 0, None), (1, 8, 256, 256, 0, None), (5, 2, 8, 8, 0, None), (37, 6, 60, 13, 20, None),
         (700, 8, 64, 64, 0, None), (512, 8, 16, 16, 0, None), (4097, 1, 1024, 1024, 0, None),
         (3000, 8, 256, 32, 96, 2000), (900, 7, 40, 40, 0, 11), (33, 64, 9, 5, 2, None), (20000, 3, 7, 7, 0, None),
         (64, 8, 8, 8, 0, 0), (1024, 8, 100, 70, 3, None), (1025, 8, 600, 600, 0, None), (40000, 8, 300, 300, 0, None)]


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,k,of,E,first,rows", SORTS)
def test_sort(T, k, of, E, first, rows, wide):
    native_loaded()
    announce(f"sort {T}x{k} of {of}, {first}..{first + E - 1}, rows {rows}, {'int64' if wide else 'int32'}")
    ids = choices(T, k, of, T + k)
    ids[0, 0] = of + 3
    if wide and T > 2:
        ids[1, 0], ids[2, 0] = 2 ** 63 - 1, -2 ** 63
    dev = torch.full((T, k + 3), 1, dtype=torch.int64 if wide else torch.int32, device="cuda")
    dev[:, :k] = ids.cuda()
    offsets, slot = fp8bs.moe_sort(dev[:, :k], E, first, rows)
    want = sorted_rows(ids, E, first, T * k if rows is None else rows)
    assert torch.equal(offsets.cpu(), want[0])
    assert torch.equal(slot.cpu(), want[1])


def test_sort_of_many():
    """More rounds than stretches: workgroups of several rounds."""
    native_loaded()
    T, k, E = 170001, 8, 100   # 1329 rounds, 128 stretches of 11
    announce(f"sort {T}x{k}")
    ids = torch.randint(-3, 130, (T, k), generator=torch.Generator().manual_seed(1))
    offsets, slot = fp8bs.moe_sort(ids.cuda(), E, first=5)
    key = ids.flatten() - 5
    key = torch.where((key >= 0) & (key < E), key, E)
    order = torch.sort(key, stable=True)[1]
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k)
    want = torch.where(key < E, place, -1).view(T, k).int()
    assert torch.equal(slot.cpu(), want)
    assert torch.equal(offsets.cpu().long(), torch.searchsorted(key[order], torch.arange(E + 1)))


def test_sort_of_nothing():
    native_loaded()
    announce("sort of no tokens")
    ids = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    offsets, slot = fp8bs.moe_sort(ids, 300)
    assert (offsets == 0).all() and slot.shape == (0, 4)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    q, s, y, offsets, slot = fp8bs.moe_dispatch(x, ids, 300)
    assert (offsets == 0).all() and q.shape == (0, 256)
    everything_elsewhere = torch.full((7, 4), -1, device="cuda")
    q, s, y, offsets, slot = fp8bs.moe_dispatch(torch.ones((7, 256), dtype=torch.bfloat16, device="cuda"),
                                                everything_elsewhere, 300)
    assert (offsets == 0).all() and (slot == -1).all()


def tokens(T, C, seed):
    x = randn(T, C, seed=seed)
    x[:, ::29] *= 20
    x[T // 2, :128] = 0
    return x.bfloat16()


def codes_of(x):
    q, s = oracle.quant_act_1x128(host(x))
    return torch.from_numpy(q), torch.from_numpy(s)


# around the largest count of one launch (8192), several tokens a workgroup with a short last one,
# widths around a lane's vectors, a wave's and a workgroup's columns
DISPATCHES = [(1, 1, 128, 1, 1, None), (1, 8, 7168, 64, 64, None), (16, 8, 7168, 64, 64, None), (3, 5, 1152, 9, 4, None),
              (256, 8, 256, 32, 32, None), (257, 8, 256, 32, 32, None), (683, 3, 384, 16, 16, 900),
              (2, 64, 640, 16, 16, None), (9, 2, 16512, 4, 4, None), (1500, 2, 1024, 8, 8, None),
              (700, 6, 16512, 160, 20, None), (40, 8, 128, 1024, 1024, None),
              (1025, 8, 128, 256, 256, None), (1024, 8, 512, 256, 256, None), (521, 15, 640, 20, 20, None),
              (1200, 7, 512, 16, 16, None), (3000, 3, 1024, 8, 8, None), (900, 9, 2048, 8, 2, None)]


@pytest.mark.parametrize("T,k,C,of,E,rows", DISPATCHES)
def test_dispatch(T, k, C, of, E, rows):
    native_loaded()
    announce(f"dispatch {T}x{k} of {of}, {E} here, {C} columns, rows {rows}")
    ids, x, first = choices(T, k, of, T + C), tokens(T, C, T), (of - E) // 2
    M = T * k if rows is None else rows
    offsets, slot = sorted_rows(ids, E, first, M)
    q0, s0 = codes_of(x)
    live = slot >= 0
    token = torch.arange(T)[:, None].expand(T, k)[live]
    at = slot[live].long()
    want_q = torch.full((M, C), 0x5A, dtype=torch.uint8)
    want_s = torch.full((M, C // 128), -1.0)
    want_y = torch.full((M, C), 9.0, dtype=torch.bfloat16)
    want_q[at], want_s[at], want_y[at] = q0[token], s0[token], x[token]

    def outputs():
        return [torch.full((M, C + 16), 0x5A, dtype=torch.uint8, device="cuda")[:, :C],
                torch.full((M, C // 128 + 1), -1.0, device="cuda")[:, :C // 128],
                torch.full((M, C + 8), 9.0, dtype=torch.bfloat16, device="cuda")[:, :C]]

    xd = torch.zeros((T, C + 8), dtype=torch.bfloat16, device="cuda")[:, :C]
    xd.copy_(x)
    for made in ("dispatch", "sort and gather"):
        out = outputs()
        if made == "dispatch":
            q, s, y, o, n = fp8bs.moe_dispatch(xd, ids.cuda(), E, first, out=out)
        else:
            o, n = fp8bs.moe_sort(ids.int().cuda(), E, first, M)
            q, s, y = fp8bs.moe_gather(xd, n, out=out)
        assert torch.equal(o.cpu(), offsets) and torch.equal(n.cpu(), slot), made
        assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s) and torch.equal(y.cpu(), want_y), made
        for wide, value in ((q, 0x5A), (s, -1.0), (y, 9.0)):
            assert (wide._base[:, wide.shape[1]:] == value).all(), made
    # rows in BF16 alone, and from codes
    out = outputs()
    fp8bs.moe_dispatch(xd, ids.cuda(), E, first, out=(None, None, out[2]))
    assert torch.equal(out[2].cpu(), want_y)
    out = outputs()
    fp8bs.moe_dispatch(q0.cuda(), ids.int().cuda(), E, first, s_in=s0.cuda(), out=(out[0], out[1], None))
    assert torch.equal(out[0].cpu(), want_q) and torch.equal(out[1].cpu(), want_s)


# larger ones on both sides of each limit between the ways there are: assignments, tokens (of narrow
# and of wide rows), values in and out; most experts, most choices, stretches that end inside a token
LARGER = [(2731, 3, 256, 8, 8, None), (4096, 8, 128, 1024, 1024, None), (4097, 8, 128, 64, 64, None),
          (512, 64, 256, 16, 16, None), (513, 64, 128, 16, 5, None), (8192, 2, 512, 64, 9, 3000), (8193, 2, 512, 64, 9, 3000),
          (16384, 1, 1024, 32, 32, None), (16385, 1, 1024, 32, 32, None), (1100, 8, 15232, 300, 3, 99),
          (1102, 8, 15232, 300, 3, 99), (4369, 7, 640, 20, 20, None), (2000, 15, 1152, 48, 6, None)]


@pytest.mark.parametrize("T,k,C,of,E,rows", LARGER)
def test_dispatch_of_larger_batches(T, k, C, of, E, rows):
    test_dispatch(T, k, C, of, E, rows)


def test_dispatch_of_a_larger_batch_captured():
    native_loaded()
    announce("dispatch 1500x8, two captured graphs")
    T, k, C, E = 1500, 8, 256, 16
    graphs = []
    for seed in (1, 2):
        ids, x = choices(T, k, E, seed).cuda(), tokens(T, C, seed).cuda()
        fp8bs.moe_dispatch(x, ids, E)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            made = fp8bs.moe_dispatch(x, ids, E)
        graphs.append((g, ids, x, made))
    for turn in range(4):
        for i, (g, ids, x, made) in enumerate(graphs):
            ids.copy_(choices(T, k, E, 10 + 2 * turn + i).cuda())
            x.copy_(tokens(T, C, 20 + 2 * turn + i).cuda())
        for g, ids, x, made in graphs:
            g.replay()
        for g, ids, x, made in graphs:
            want = fp8bs.moe_dispatch(x, ids, E)
            rows = int(want[3][-1])
            assert torch.equal(made[3], want[3]) and torch.equal(made[4], want[4])
            assert torch.equal(made[0][:rows], want[0][:rows]) and torch.equal(made[1][:rows], want[1][:rows])


COMBINES = [(1, 1, 128, 1, 1), (50, 3, 512, 8, 8), (600, 9, 128, 8, 8), (16, 8, 7168, 64, 64), (5, 3, 640, 8, 3), (300, 2, 1152, 8, 8), (33, 64, 256, 16, 16),
            (7, 9, 384, 20, 20), (1030, 8, 512, 60, 30)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,N,of,E", COMBINES)
def test_combine(T, k, N, of, E, kind):
    native_loaded()
    announce(f"combine {T}x{k}, {N} columns, {kind}")
    ids = choices(T, k, of, T + N, 0.2)
    if T > 3:
        ids[3] = -1   # a token without rows
    offsets, slot = sorted_rows(ids, E, 0, T * k)
    M = T * k
    y = randn(M, N, seed=1)
    y[int(offsets[-1]):] = NAN   # rows of nobody
    y = y.bfloat16() if kind == "bf16" else y
    w = randn(T, k, seed=2)
    add = randn(T, N, seed=3).bfloat16()
    live = (slot >= 0)[..., None]
    rows = torch.where(live, y.double()[slot.long().clamp(min=0)], 0.0)
    w_there = torch.where(live[..., 0], w.double(), 0.0)[..., None]
    w = torch.where(live[..., 0], w, NAN)   # weights of nothing
    yd = torch.zeros((M, N + 8), dtype=y.dtype, device="cuda")[:, :N]
    yd.copy_(y)
    for weighted in (False, True):
        for added in (False, True):
            terms = rows * w_there if weighted else rows
            want = terms.sum(1) + (add.double() if added else 0)
            size = terms.abs().sum(1) + (add.double().abs() if added else 0)
            out = fp8bs.moe_combine(yd, slot.cuda(), w.cuda() if weighted else None, add.cuda() if added else None)
            check_bf16(f"combine {weighted} {added}", out, want, (k + 1) * U * size)
            if added:   # onto add itself, in wider rows
                wide = torch.full((T + 1, N + 8), 4.0, dtype=torch.bfloat16, device="cuda")
                wide[:T, :N] = add
                part = wide[:T, :N]
                fp8bs.fp8bs_moe_combine(yd, slot.cuda(), w.cuda() if weighted else None, part, part)
                assert torch.equal(part, out)
                assert (wide[T] == 4).all() and (wide[:, N:] == 4).all()


GRADIENTS = [(1, 1, 128, 1, 1), (50, 9, 512, 8, 8), (600, 17, 128, 8, 8), (520, 3, 2176, 8, 8), (512, 2, 16512, 4, 4), (77, 4, 1152, 16, 16), (16, 8, 7168, 64, 40), (5, 64, 640, 8, 8), (9, 2, 16512, 4, 4),
             (700, 3, 1024, 8, 8), (3, 5, 2048, 8, 2)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,N,of,E", GRADIENTS)
def test_combine_gradient(T, k, N, of, E, kind):
    native_loaded()
    announce(f"combine gradient {T}x{k}, {N} columns, {kind}")
    ids = choices(T, k, of, T + N, 0.2)
    offsets, slot = sorted_rows(ids, E, 0, T * k)
    M = T * k
    y = randn(M, N, seed=1)
    y[int(offsets[-1]):] = NAN
    y = y.bfloat16() if kind == "bf16" else y
    dout = tokens(T, N, 2)
    w = randn(T, k, seed=3)
    live = slot >= 0
    at, (t, j) = slot[live].long(), live.nonzero(as_tuple=True)
    w[~live] = NAN
    if at.numel() > 2:
        w[t[0], j[0]] = 0.0
    q0, s0 = codes_of(dout)
    want_q = torch.full((M, N), 0x5A, dtype=torch.uint8)
    want_s = torch.full((M, N // 128), -1.0)
    want_dy = torch.full((M, N), 9.0, dtype=torch.bfloat16)
    weight = w[t, j][:, None]
    want_q[at] = torch.where(weight < 0, q0[t] ^ 0x80, q0[t])
    want_s[at] = s0[t] * weight.abs()
    want_dy[at] = (dout[t].float() * weight).bfloat16()
    want_dw = torch.zeros((T, k), dtype=torch.float64)
    size = torch.zeros((T, k), dtype=torch.float64)
    want_dw[t, j] = (dout[t].double() * y[at].double()).sum(1)
    size[t, j] = (dout[t].double() * y[at].double()).abs().sum(1)

    def outputs():
        return [torch.full((M, N + 16), 0x5A, dtype=torch.uint8, device="cuda")[:, :N],
                torch.full((M, N // 128 + 1), -1.0, device="cuda")[:, :N // 128],
                torch.full((M, N + 8), 9.0, dtype=torch.bfloat16, device="cuda")[:, :N]]

    out = outputs()
    q, s, dy, dw = fp8bs.moe_combine_bwd(dout.cuda(), slot.cuda(), w.cuda(), y.cuda(), out=out)
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s) and torch.equal(dy.cpu(), want_dy)
    check_f32("dw", dw, want_dw, (16 * math.ceil(N / 16384) + 6 + 15) * U * size)
    assert (dw.cpu()[~live] == 0).all()
    for wide, value in ((q, 0x5A), (s, -1.0), (dy, 9.0)):
        assert (wide._base[:, wide.shape[1]:] == value).all()
    # each output alone
    out = outputs()
    assert fp8bs.moe_combine_bwd(dout.cuda(), slot.cuda(), w.cuda(), out=(out[0], out[1], None))[3] is None
    assert torch.equal(out[0].cpu(), want_q) and torch.equal(out[1].cpu(), want_s)
    fp8bs.moe_combine_bwd(dout.cuda(), slot.cuda(), w.cuda(), out=(None, None, out[2]))
    assert torch.equal(out[2].cpu(), want_dy)
    alone = fp8bs.moe_combine_bwd(dout.cuda(), slot.cuda(), w.cuda(), y.cuda(), out=(None, None, None))
    assert torch.equal(alone[3], dw)


def test_slots_outside_are_not_followed():
    """A slot array that no sort gave: in bounds only what is in range."""
    native_loaded()
    announce("slots outside")
    T, k, C, M = 6, 3, 256, 5
    slot = torch.tensor([[-1, 5, 0], [2 ** 31 - 1, -2 ** 31, 6], [1, 7, 2], [3, -9, 100], [5, 5, 5], [4, -1, -1]],
                        dtype=torch.int32)
    x, y, w = tokens(T, C, 1), randn(M, C, seed=2).bfloat16(), randn(T, k, seed=3)
    out = [torch.full((M + 1, C), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((M + 1, 2), -1.0, device="cuda"),
           torch.full((M + 1, C), 9.0, dtype=torch.bfloat16, device="cuda")]
    q, s, z = fp8bs.moe_gather(x.cuda(), slot.cuda(), out=[t[:M] for t in out])
    assert torch.equal(z.cpu(), x[[0, 2, 2, 3, 5]])
    assert (out[0][M] == 0x5A).all() and (out[1][M] == -1).all() and (out[2][M] == 9).all()
    live = ((slot >= 0) & (slot < M))[..., None]
    terms = torch.where(live, y.double()[slot.long().clamp(0, M - 1)] * w.double()[..., None], 0.0)
    check_bf16("combine", fp8bs.moe_combine(y.cuda(), slot.cuda(), w.cuda()), terms.sum(1), 4 * U * terms.abs().sum(1))
    dw = fp8bs.moe_combine_bwd(x.cuda(), slot.cuda(), w.cuda(), y.cuda(), out=[t[:M] for t in out])[3]
    assert (dw.cpu()[~live[..., 0]] == 0).all() and (out[0][M] == 0x5A).all() and (out[2][M] == 9).all()


def test_gradients_of_each_other():
    """<gather(x), z> = <x, combine(z)>, and combine's gradient against differences
    of the binary64 sum along directions of y and w."""
    native_loaded()
    announce("adjoint pair and differences")
    T, k, C, E = 50, 4, 384, 8
    ids = choices(T, k, E, 1)
    offsets, slot = fp8bs.moe_sort(ids.cuda(), E)
    n = int(offsets[-1])
    x, z = tokens(T, C, 1), randn(T * k, C, seed=2).bfloat16()
    moved = fp8bs.moe_gather(x.cuda(), slot, codes=False, with_y=True)[2][:n].cpu().double()
    back = fp8bs.moe_combine(z.cuda(), slot).cpu().double()
    left, right = (moved * z[:n].double()).sum(), (x.double() * back).sum()
    assert abs(left - right) <= 2.0 ** -8 * (x.double() * back).abs().sum() + 1e-4
    w, dout = randn(T, k, seed=3), randn(T, C, seed=4).bfloat16()
    _, _, dy, dw = fp8bs.moe_combine_bwd(dout.cuda(), slot, w.cuda(), z.cuda(), with_dy=True)
    live = (slot >= 0).cpu()[..., None]
    at = slot.cpu().long().clamp(min=0)

    def value(y, w):
        return (dout.double() * torch.where(live, y[at] * w[..., None], 0.0).sum(1)).sum()

    way_y, way_w, step = randn(T * k, C, seed=5).double(), randn(T, k, seed=6).double(), 1e-5
    zd, wd = z.double(), w.double()
    slope = (value(zd + step * way_y, wd) - value(zd - step * way_y, wd)) / (2 * step)
    part = dy[:n].cpu().double() * way_y[:n]
    assert abs(part.sum() - slope) <= (2.0 ** -8 + 1e-6) * part.abs().sum()
    slope = (value(zd, wd + step * way_w) - value(zd, wd - step * way_w)) / (2 * step)
    part = dw.cpu().double() * way_w
    assert abs(part.sum() - slope) <= 1e-5 * part.abs().sum()


def test_past_32_bits():
    """Rows past 2^31 values and 4 GiB, in every array that has them."""
    native_loaded()
    C = 7168
    M = 2 ** 31 // C + 100
    announce(f"rows past 32 bits, {M}x{C}")
    T, k = 40, 3
    slot = torch.randperm(2 * T * k, generator=torch.Generator().manual_seed(1))[:T * k].view(T, k).int()
    slot = torch.where(slot % 2 == 0, M - 1 - slot, slot)
    x, w = tokens(T, C, 1), randn(T, k, seed=2)
    q = torch.zeros((M, C), dtype=torch.uint8, device="cuda")
    s = torch.zeros((M, C // 128), device="cuda")
    y = torch.zeros((M, C), dtype=torch.bfloat16, device="cuda")
    fp8bs.moe_gather(x.cuda(), slot.cuda(), out=(q, s, y))
    at = slot.long().flatten()
    token = torch.arange(T)[:, None].expand(T, k).flatten()
    q0, s0 = codes_of(x)
    rows = at.cuda()
    assert torch.equal(q[rows].cpu(), q0[token]) and torch.equal(s[rows].cpu(), s0[token])
    assert torch.equal(y[rows].cpu(), x[token])
    terms = x.double()[:, None] * w.double()[..., None]
    check_bf16("combine", fp8bs.moe_combine(y, slot.cuda(), w.cuda()), terms.sum(1), (k + 1) * U * terms.abs().sum(1))
    dout = tokens(T, C, 3)
    _, _, dy, dw = fp8bs.moe_combine_bwd(dout.cuda(), slot.cuda(), w.cuda(), y, out=(q, s, torch.zeros_like(y)))
    want = (dout.double() * x.double()).sum(1)[:, None].expand(T, k)
    check_f32("dw", dw, want, 37 * U * (dout.double() * x.double()).abs().sum(1)[:, None])
    assert torch.equal(dy[rows].cpu(), (dout[token].float() * w.flatten()[:, None]).bfloat16())
    # many tokens: sources and outputs by token past 4 GiB
    del q, s, y, dy
    many = torch.zeros((M, C), dtype=torch.bfloat16, device="cuda")
    many[-T:] = x.cuda()
    ids = torch.full((M, 1), -1, dtype=torch.int32, device="cuda")
    ids[-T:, 0] = torch.arange(T, device="cuda") % 3
    q, s, _, offsets, slot = fp8bs.moe_dispatch(many, ids, 3, rows=T)
    want_o, want_slot = sorted_rows(ids[-T:].cpu(), 3, 0, T)
    assert torch.equal(slot[-T:].cpu(), want_slot) and (slot[:-T] == -1).all() and torch.equal(offsets.cpu(), want_o)
    assert torch.equal(q.cpu()[want_slot[:, 0].long()], q0)
    out = fp8bs.moe_combine(x.cuda()[:1].expand(T, C).contiguous(), slot, add=many)
    assert torch.equal(out[-T:], (x.cuda()[:1].float() + x.cuda().float()).bfloat16())
    assert (out[:-T] == 0).all()
