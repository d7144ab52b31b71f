"""Race check of the attention kernels: the LDS-poisoning debug build fills
each kernel's LDS with NaN bytes before its first use; results must be those of
the library build, bit for bit."""
import numpy as np
import pytest

from fp8_fine_grained_fp8bs_amd import build, fp8bs
from tests import test_gpu_attn as ta
from tests import test_gpu_kv_append as tk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def poisoned_library():
    prev = fp8bs.use_library(build.POISON_LIB)
    try:
        yield
    finally:
        fp8bs.use_library(prev)


@pytest.mark.parametrize("d", [64, 128])
def test_few_rows(d):
    ta.check(ta.make(1, [1, 17, 700, 0, 333], [1] * 5, 8, 2, d, 16), no_off=True)
    ta.check(ta.make(2, [4000, 90], [1, 3], 8, 1, d, 64))


@pytest.mark.parametrize("d,page", [(64, 16), (64, 64), (128, 32), (128, 128)])
def test_many_rows(d, page):
    ta.check(ta.make(3, [130, 1, 400, 900], [130, 1, 400, 70], 8, 2, d, page))
    ta.check(ta.make(4, [260] * 8, [260] * 8, 64, 8, d, page), window=50)


def test_append():
    tk.check(tk.setup(5, [1, 130, 64, 20], [1, 130, 64, 3], 4, 2, 128, 64))
    tk.check(tk.setup(6, [33, 17], [1, 1], 4, 2, 64, 16), no_off=True)


def test_the_library_build_gives_the_same_bits():
    c = ta.make(7, [300, 1200, 40], [300, 2, 40], 16, 2, 128, 64)
    args = [ta.u8_dev(c["kc"]), ta.f32_dev(c["ks"]), ta.u8_dev(c["vc"]), ta.f32_dev(c["vs"])]
    rest = [ta.torch.from_numpy(c[n]).to(ta.dev()) for n in ("tab", "kv_len", "off")]
    x = ta.host(fp8bs.attn_paged(ta.bf16_dev(c["q"]), *args, *rest, max_q=300))
    fp8bs.use_library(fp8bs.LIB_PATH)
    y = ta.host(fp8bs.attn_paged(ta.bf16_dev(c["q"]), *args, *rest, max_q=300))
    assert np.array_equal(x, y)
