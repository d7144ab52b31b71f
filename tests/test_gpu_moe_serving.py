"""GPU: the operators around the experts' products as programs call them: on
other streams, from two streams at once, captured two at a time, by the compiled
short way and by the long one, and with poisoned LDS."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import build, fp8bs
from tests import test_gpu_moe as tm
from tests import test_gpu_norm as tn
from tests import test_gpu_swiglu_bwd as ts
from tests.gpu_common import announce
from tests.moe_ref import randn

pytestmark = pytest.mark.gpu


def calls(T=300, k=4, C=512, E=12, seed=0):
    """Every helper as a function of a stream, with its arguments."""
    x, r = tm.tokens(T, C, seed).cuda(), tm.tokens(T, C, seed + 1).cuda()
    dout = randn(T, C, seed=seed + 2, scale=0.01).bfloat16().cuda()
    gamma = tn.gamma_of(C, "f32", seed).cuda()
    ids = tm.choices(T, k, E, seed).cuda()
    w = torch.rand((T, k), generator=torch.Generator().manual_seed(seed)).cuda()
    offsets, slot = fp8bs.moe_sort(ids, E)
    y = randn(T * k, C, seed=seed + 3).bfloat16().cuda()
    rstd = tn.norm(x.cpu(), gamma.cpu(), 1e-6)[1].float().cuda()
    q, s, _ = fp8bs.moe_gather(x, slot, out=(torch.zeros((T * k, C), dtype=torch.uint8, device="cuda"),
                                             torch.zeros((T * k, C // 128), device="cuda"), None))

    def rows(with_y=True):
        """Zeros to write into: rows past the last stay as they are."""
        return (torch.zeros_like(q), torch.zeros_like(s),
                torch.zeros((T * k, C), dtype=torch.bfloat16, device="cuda") if with_y else None)

    torch.cuda.synchronize()
    return {
        "norm": lambda **kw: fp8bs.rmsnorm_quant_1x128(x, gamma, r, with_y=True, with_rstd=True, **kw),
        "norm gradient": lambda **kw: fp8bs.rmsnorm_bwd(dout, x, gamma, rstd, r, **kw),
        "sort": lambda **kw: fp8bs.moe_sort(ids, E, **kw),
        "gather": lambda out=None, **kw: fp8bs.moe_gather(x, slot, out=out or rows(), **kw),
        "dispatch": lambda out=None, **kw: fp8bs.moe_dispatch(x, ids, E, out=out or rows(), **kw),
        "dispatch codes": lambda out=None, **kw: fp8bs.moe_dispatch(q[:T], ids, E, s_in=s[:T], out=out or rows(False), **kw),
        "combine": lambda **kw: fp8bs.moe_combine(y, slot, w, r, **kw),
        "combine gradient": lambda out=None, **kw: fp8bs.moe_combine_bwd(dout, slot, w, y, out=out or rows(), **kw),
        "swiglu gradient": lambda **kw: fp8bs.swiglu_bwd_quant_1x128(dout, x, r, with_d=True, with_h=True, **kw),
    }, rows


SIZES = [dict(T=300), dict(T=1500), dict(T=3000, C=256)]   # the sort's three forms, few rows and many


def flat(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


def same(a, b, name):
    a, b = flat(a), flat(b)
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b)), name


@pytest.mark.parametrize("size", SIZES)
def test_on_another_stream(size):
    """With the current stream busy: the working memory that the call allocates
    belongs to the stream it runs on, and what is allocated right after on the current
    one does not get it."""
    ops, rows = calls(**size)
    st = torch.cuda.Stream()
    for name, op in ops.items():
        announce(f"{name} on another stream {size}")
        want = op()
        torch.cuda.synchronize()
        for stream in (st, st.cuda_stream):
            kw = dict(out=rows("codes" not in name)) if name in ("gather", "dispatch", "dispatch codes", "combine gradient") else {}
            torch.cuda.synchronize()
            torch.cuda._sleep(1000000)
            got = op(stream=stream, **kw)
            over = [torch.full((1 << 18,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
            st.synchronize()
            same(got, want, name)
            torch.cuda.synchronize()
            del over


def test_two_streams_at_once():
    """Interleaved calls from two streams, each under torch's stream context."""
    announce("two streams at once")
    a, b = calls(T=1500, seed=1), calls(T=1500, seed=2)
    want = [{n: f() for n, f in ops.items()} for ops, _ in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for name in a[0]:
            for i, ops in enumerate((a[0], b[0])):
                with torch.cuda.stream(streams[i]):
                    got[i].append((name, ops[name]()))
    torch.cuda.synchronize()
    for i in range(2):
        for name, out in got[i]:
            same(out, want[i][name], name)


@pytest.mark.parametrize("size", SIZES)
def test_two_graphs(size):
    """Two graphs of the same calls on other inputs, captured one after the other
    and replayed in turn, with eager calls between."""
    announce(f"two graphs {size}")
    both = [calls(seed=s, **size)[0] for s in (1, 2)]
    graphs, captured = [], []
    for ops in both:
        for op in ops.values():
            op()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            captured.append({n: op() for n, op in ops.items()})
        graphs.append(g)
    for turn in range(3):
        want = [{n: op() for n, op in ops.items()} for ops in both]
        torch.cuda.synchronize()
        for i in ((0, 1), (1, 0), (0, 1))[turn]:
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for n in want[i]:
                same(captured[i][n], want[i][n], n)


@pytest.mark.parametrize("size", SIZES)
def test_both_ways_give_the_same_bits(size, monkeypatch):
    """The compiled short way and the checks in Python, on the same tensors."""
    announce(f"short and long way {size}")
    ops, _ = calls(**size)
    short = {n: op() for n, op in ops.items()}
    assert any(w is not fp8bs._no_way for w in fp8bs._ways.values()), "no compiled short way"
    monkeypatch.setattr(fp8bs, "_ways", dict.fromkeys(fp8bs._ways, fp8bs._no_way))
    for n, op in ops.items():
        same(op(), short[n], n)


def test_statuses_of_the_short_way():
    """Refusals of the library come back as errors, also by the short way."""
    announce("refusals by the short way")
    x = torch.zeros((4, 192), dtype=torch.bfloat16, device="cuda")
    gamma, ids = torch.ones(192, device="cuda"), torch.zeros((4, 2), dtype=torch.int32, device="cuda")
    slot, w = ids.clone(), torch.ones((4, 2), device="cuda")
    for call in (lambda: fp8bs.rmsnorm_quant_1x128(x, gamma), lambda: fp8bs.rmsnorm_bwd(x, x, gamma, gamma[:4].contiguous()),
                 lambda: fp8bs.moe_dispatch(x, ids, 4), lambda: fp8bs.moe_combine(x, slot, w),
                 lambda: fp8bs.moe_combine_bwd(x, slot, w, x), lambda: fp8bs.swiglu_bwd_quant_1x128(x, x, x),
                 lambda: fp8bs.moe_gather(x, slot)):
        with pytest.raises(fp8bs.Fp8bsError) as e:
            call()
        assert e.value.status == fp8bs.ERR_UNSUPPORTED_SHAPE
    for eps in (0.0, -1.0, float("nan")):
        with pytest.raises(fp8bs.Fp8bsError):
            fp8bs.rmsnorm_quant_1x128(x[:, :128], gamma[:128], eps=eps)
    for call in (lambda: fp8bs.moe_sort(ids, 0), lambda: fp8bs.moe_sort(ids, 2000), lambda: fp8bs.moe_sort(ids, 4, first=-1)):
        with pytest.raises((fp8bs.Fp8bsError, ValueError)):
            call()


def test_a_single_row_of_any_stride():
    """One token as a slice of rows whose stride breaks the alignment rules."""
    announce("single rows")
    C = 256
    wide = randn(3, C + 3, seed=1).bfloat16().cuda()
    x = torch.cat([wide[:, :C].flatten(), wide.flatten()]).as_strided((1, C), (C + 3, 1))
    gamma, ids = torch.ones(C, device="cuda"), torch.zeros((1, 1), dtype=torch.int64, device="cuda")
    dense = x.contiguous()
    same(fp8bs.rmsnorm_quant_1x128(x, gamma, x), fp8bs.rmsnorm_quant_1x128(dense, gamma, dense), "norm")
    same(fp8bs.moe_dispatch(x, ids, 1), fp8bs.moe_dispatch(dense, ids, 1), "dispatch")
    same(fp8bs.moe_gather(x, ids.int()), fp8bs.moe_gather(dense, ids.int()), "gather")
    same(fp8bs.swiglu_bwd_quant_1x128(x, x, x), fp8bs.swiglu_bwd_quant_1x128(dense, dense, dense), "swiglu gradient")


def test_misfits_are_turned_back():
    """Arguments that do not fit are refused, whichever way sees them first."""
    announce("misfits")
    T, k, C = 4, 2, 256
    x, gamma = torch.zeros((T, C), dtype=torch.bfloat16, device="cuda"), torch.ones(C, device="cuda")
    f, ids = torch.ones((T, k), device="cuda"), torch.zeros((T, k), dtype=torch.int32, device="cuda")
    rstd, y = torch.ones(T, device="cuda"), torch.zeros((T * k, C), dtype=torch.bfloat16, device="cuda")
    good = [(fp8bs.rmsnorm_quant_1x128, [x, gamma, x]), (fp8bs.rmsnorm_bwd, [x, x, gamma, rstd, x]),
            (fp8bs.moe_dispatch, [x, ids, 4]), (fp8bs.moe_combine, [y, ids, f, x]),
            (fp8bs.moe_combine_bwd, [x, ids, f, y]), (fp8bs.swiglu_bwd_quant_1x128, [x, x, x])]
    for call, args in good:
        call(*args)
        for i, a in enumerate(args):
            if not isinstance(a, torch.Tensor):
                continue
            for bad in (a.double(), a[:-1], a.unsqueeze(0), a.cpu(), torch.cat([a, a], dim=-1)[..., ::2]):
                if bad.shape == a.shape and bad.dtype == a.dtype and bad.is_cuda and bad.is_contiguous():
                    continue
                if call is fp8bs.moe_combine and i == 0 and bad.dim() == 2 and bad.is_cuda and bad.dtype == a.dtype and \
                        bad.stride(-1) == 1:
                    continue   # fewer rows are rows too: slots past them are not followed
                if call is fp8bs.moe_combine_bwd and i == 3 and bad.dim() == 2 and bad.is_cuda and bad.dtype == a.dtype and \
                        bad.stride(-1) == 1:
                    continue
                with pytest.raises(ValueError):
                    call(*args[:i], bad, *args[i + 1:])


def test_poisoned_lds():
    """With LDS filled with NaN bytes before a kernel's first use: the library
    build's bits."""
    for size in SIZES + [dict(T=3, k=3, C=8448), dict(T=2, k=64, C=128, E=1000)]:
        announce(f"poisoned LDS {size}")
        ops, _ = calls(**size)
        want = {n: op() for n, op in ops.items()}
        torch.cuda.synchronize()
        prev = fp8bs.use_library(build.POISON_LIB)
        try:
            for n, op in ops.items():
                same(op(), want[n], n)
            torch.cuda.synchronize()
        finally:
            fp8bs.use_library(prev)
    ts.test_edge_gates()


def wide(t, extra, value):
    """The tensor as a part of wider rows."""
    w = torch.full((t.shape[0], t.shape[1] + extra), value, dtype=t.dtype, device="cuda")
    w[:, :t.shape[1]] = t
    return w[:, :t.shape[1]]


def test_every_input_in_wider_rows():
    announce("inputs in wider rows")
    T, k, C, E = 130, 3, 640, 7
    x, dout = tm.tokens(T, C, 1).cuda(), tm.tokens(T, C, 2).cuda()
    ids, w = tm.choices(T, k, E, 1).cuda(), torch.rand((T, k), device="cuda")
    offsets, slot = fp8bs.moe_sort(wide(ids, 5, 3), E)
    same((offsets, slot), fp8bs.moe_sort(ids, E), "sort")
    n = int(offsets[-1])
    y = randn(T * k, C, seed=3).cuda()
    cut = lambda out: tuple(t if t is None or t.shape[0] != T * k else t[:n] for t in out)  # noqa: E731
    q, s, _ = fp8bs.moe_gather(x, slot)
    q, s = q[:T].clone(), s[:T].clone()
    same(cut(fp8bs.moe_gather(wide(q, 32, 1), slot, s_in=wide(s, 3, 9.0))), cut(fp8bs.moe_gather(q, slot, s_in=s)), "gather")
    same(cut(fp8bs.moe_dispatch(wide(q, 32, 1), ids, E, s_in=wide(s, 3, 9.0))), cut(fp8bs.moe_dispatch(q, ids, E, s_in=s)),
         "dispatch")
    for rows in (y, y.bfloat16()):
        same(fp8bs.moe_combine(wide(rows, 8, 1.0), slot, wide(w, 5, 7.0), wide(x, 24, 1.0)),
             fp8bs.moe_combine(rows, slot, w, x), "combine")
        same(cut(fp8bs.moe_combine_bwd(wide(dout, 8, 1.0), slot, wide(w, 1, 7.0), wide(rows, 16, 1.0), with_dy=True)),
             cut(fp8bs.moe_combine_bwd(dout, slot, w, rows, with_dy=True)), "combine gradient")
    same(fp8bs.swiglu_bwd_quant_1x128(wide(dout, 40, 1.0), wide(x, 8, 1.0), wide(y.bfloat16()[:T], 16, 1.0), with_d=True),
         fp8bs.swiglu_bwd_quant_1x128(dout, x, y.bfloat16()[:T], with_d=True), "swiglu gradient")


@pytest.mark.parametrize("T", [3, 400, 1500])
def test_more_rows_than_assignments(T):
    """Buffers larger than every case needs: the rows behind the last stay."""
    announce(f"more rows than assignments, T {T}")
    k, C, E = 4, 256, 9
    x, ids = tm.tokens(T, C, 1).cuda(), tm.choices(T, k, E, 2).cuda()
    few = fp8bs.moe_dispatch(x, ids, E)
    n = int(few[3][-1])
    out = (torch.full((T * k + 50, C), 0x5A, dtype=torch.uint8, device="cuda"), torch.full((T * k + 50, C // 128), -1.0, device="cuda"),
           None)
    q, s, _, offsets, slot = fp8bs.moe_dispatch(x, ids, E, out=out)
    assert torch.equal(offsets, few[3]) and torch.equal(slot, few[4])
    assert torch.equal(q[:n], few[0][:n]) and torch.equal(s[:n], few[1][:n])
    assert (q[n:] == 0x5A).all() and (s[n:] == -1).all()
