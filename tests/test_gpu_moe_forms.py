"""GPU: what the operators around the experts' products are called with by
programs (other streams, two graphs, the short and the long way, poisoned LDS), at
the sizes of each form that they have:
- 8300 x 4 of 256 or 1152 columns: dispatch in three launches that share a working
  memory (past 8192 tokens of narrow rows, and past 32768 assignments);
- 2000 x 5 of 1280 columns: dispatch behind the counting kernel, wide rows;
- 600 x 4 of 1280 columns: dispatch in one launch; the norm's gradient with its
  parts of dgamma in a working memory, three waves a row; the gradient of the
  way back with four vectors a lane.
And the parts of the example's layer that are torch's."""
import functools

import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests import test_gpu_expert_layer as layer_tests
from tests import test_gpu_moe_serving as serving
from tests.gpu_common import announce, native_loaded
from tests.moe_ref import U, check_f32
from tests.test_gpu_moe_serving import calls, same

pytestmark = pytest.mark.gpu
SIZES = [dict(T=8300, k=4, C=256), dict(T=8300, k=4, C=1152), dict(T=2000, k=5, C=1280), dict(T=600, k=4, C=1280)]


def test_which_have_a_working_memory():
    for size in SIZES:
        T, k, C = size["T"], size["k"], size["C"]
        assert (fp8bs.fp8bs_moe_sort_ws(T, k, 12) > 0) == (T > 600) and fp8bs.fp8bs_rmsnorm_bwd_ws(T, C) > 0


@pytest.mark.parametrize("size", SIZES)
def test_on_another_stream(size):
    native_loaded()
    serving.test_on_another_stream(size)


@pytest.mark.parametrize("size", SIZES)
def test_two_streams_at_once(size, monkeypatch):
    announce(f"two streams at once {size}")
    monkeypatch.setattr(serving, "calls", lambda T, seed: calls(seed=seed, **size))
    serving.test_two_streams_at_once()


@pytest.mark.parametrize("size", SIZES)
def test_two_graphs(size):
    serving.test_two_graphs(size)


def test_poisoned_lds(monkeypatch):
    monkeypatch.setattr(serving, "SIZES", SIZES)
    serving.test_poisoned_lds()


# above 32768 assignments: the sort's two kernels and the rows' own
def test_layer_captured():
    layer_tests.test_captured(4200)


SHORT = ("rmsnorm_quant_1x128", "rmsnorm_bwd", "moe_dispatch", "moe_combine", "moe_combine_bwd", "swiglu_bwd_quant_1x128")


@pytest.mark.parametrize("size", serving.SIZES + SIZES)
def test_the_short_way_is_taken(size, monkeypatch):
    """Every helper that has a compiled short way goes by it, with the bits of the
    long one."""
    announce(f"short way taken {size}")
    taken = []

    def watched(name, way, *args):
        result = way(*args)
        taken.append((name, result is not None and result.__class__ is not int))
        return result

    ops, _ = calls(**size)
    for op in ops.values():      # looks the ways up
        op()
    ways = dict(fp8bs._ways)
    assert set(ways) == {"fp8bs_" + n for n in SHORT}
    monkeypatch.setattr(fp8bs, "_ways", {n: functools.partial(watched, n, w) for n, w in ways.items()})
    short = {n: op() for n, op in ops.items()}
    assert all(ok for _, ok in taken) and {n for n, _ in taken} == set(ways), taken
    count = len(taken)
    monkeypatch.setattr(fp8bs, "_ways", dict.fromkeys(ways, fp8bs._no_way))
    for n, op in ops.items():
        same(op(), short[n], n)
    assert len(taken) == count


def test_outputs_made_by_both_ways(monkeypatch):
    """The same where the helpers make the rows' outputs: the rows that have a token."""
    announce("outputs made by the short and the long way")
    T, k, C, E = 700, 3, 640, 9
    ids = torch.randint(-1, E, (T, k), generator=torch.Generator().manual_seed(1)).cuda()
    x, y = torch.randn((T, C), device="cuda").bfloat16(), torch.randn((T * k, C), device="cuda")
    w = torch.rand((T, k), device="cuda")
    got = []
    for way in ("short", "long"):
        if way == "long":
            monkeypatch.setattr(fp8bs, "_ways", dict.fromkeys(fp8bs._ways, fp8bs._no_way))
        q, s, rows, offsets, slot = fp8bs.moe_dispatch(x, ids, E, with_y=True)
        n = int(offsets[-1])
        q2, s2, dy, dw = fp8bs.moe_combine_bwd(x, slot, w, y, with_dy=True)
        assert fp8bs.moe_combine_bwd(x, slot, w)[3] is None and fp8bs.moe_dispatch(x, ids, E, rows=50)[0].shape[0] == 50
        got.append((q[:n], s[:n], rows[:n], offsets, slot, q2[:n], s2[:n], dy[:n], dw))
    same(*got, "made")


@pytest.mark.parametrize("tokens,hidden,inner,experts,choices", [(37, 256, 128, 5, 2), (300, 384, 256, 8, 3)])
def test_router_of_the_layer(tokens, hidden, inner, experts, choices):
    """The choice, its weights and their gradients, which torch computes: FP32 sums in
    any order, n U of their terms' sizes (products of two BF16 values are exact); the
    softmax's exponents are off by twice a score's error, its sum and quotient by few U."""
    announce(f"router of {tokens} tokens, {choices} of {experts}")
    layer, x, residual, _, _, kept, (_, _, drouter, t) = layer_tests.example().run(tokens, hidden, inner, experts, choices,
                                                                                verbose=False)
    n = fp8bs.rmsnorm_quant_1x128(x, layer.gamma, residual, with_y=True)[3].cpu().double()
    router, ids = layer.router.cpu().double(), kept["ids"].cpu()
    scores, off = n @ router.t(), hidden * U * (n.abs() @ router.abs().t()).amax()
    top = scores.gather(1, ids)
    assert all(len(set(row)) == choices for row in ids.tolist())
    rest = scores.scatter(1, ids, -float("inf"))
    assert (top.amin(1) >= rest.amax(1) - 2 * off).all()
    w = top.softmax(1)
    check_f32("w", kept["w"], w, w * (torch.expm1(2 * off) + (choices + 16) * U))
    w, dw = kept["w"].cpu().double(), t["dw"].cpu().double()
    mean, size = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
    zeros = torch.zeros((tokens, experts), dtype=torch.float64)
    check_f32("dlogits", t["dlogits"], zeros.scatter(1, ids, w * (dw - mean)),
              zeros.scatter(1, ids, (choices + 3) * U * w * (dw.abs() + size)))
    f = kept["h"].cpu().double() * kept["rstd"].cpu().double()[:, None] * layer.gamma.cpu().double()
    d = t["dlogits"].cpu().double()
    check_f32("drouter", drouter, d.t() @ f, (tokens + 3) * U * (d.abs().t() @ f.abs()))
