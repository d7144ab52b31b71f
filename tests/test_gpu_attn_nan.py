"""GPU: a NaN among a row's queries makes that row's outputs and its lse NaN, and
nothing else: minus infinity is the lse of a row that sees no key."""
import numpy as np
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests import test_gpu_attn as ta
from tests.gpu_common import announce, dev, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new", [([700, 0, 33], [1, 1, 1]), ([20000], [1]), ([500, 4, 90], [5, 6, 2]),
                                      ([300, 40], [300, 70]), ([9000], [70])])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_a_row_of_nan(lens, new, d, page):
    hq, hkv = 4, 2
    c = ta.make(len(lens) + d, lens, new, hq, hkv, d, page)
    T = sum(new)
    bad = np.random.default_rng(T).random((T, hq)) < 0.3
    bad[-1, 1] = True
    c["q"][bad, 7] = 0x7FC0
    announce(f"attn with NaN queries: lens {lens} rows {new} heads of {d}")
    a = [ta.u8_dev(c["kc"]), ta.f32_dev(c["ks"]), ta.u8_dev(c["vc"]), ta.f32_dev(c["vs"])]
    rest = [torch.from_numpy(c[n]).to(dev()) for n in ("tab", "kv_len", "off")]
    out, lse = fp8bs.attn_paged(ta.bf16_dev(c["q"]), *a, *rest, max_q=max(new), with_lse=True)
    clean = dict(c, q=np.where(bad[..., None], 0x3F80, c["q"]).astype(np.uint16))
    want, want_lse = fp8bs.attn_paged(ta.bf16_dev(clean["q"]), *a, *rest, max_q=max(new), with_lse=True)
    out, lse, want, want_lse = out.float().cpu().numpy(), host(lse), want.float().cpu().numpy(), host(want_lse)
    # a row that sees no key has zeros and minus infinity whatever its query is
    none = np.isneginf(want_lse)
    gone = bad & ~none
    assert gone.any()
    assert np.isnan(out[gone]).all() and np.isnan(lse[gone]).all()
    assert np.array_equal(out[~gone], want[~gone]) and np.array_equal(lse[~gone], want_lse[~gone])
