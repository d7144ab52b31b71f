"""CPU: in the LDS-poisoning build every shared array of every kernel is filled."""
import os
import re

import pytest

from fp8_fine_grained_fp8bs_amd import build


@pytest.mark.parametrize("src", sorted(f for f in os.listdir(build.CSRC) if f.endswith(".hip")))
def test_every_array_is_filled(src):
    with open(os.path.join(build.CSRC, src)) as f:
        kernels = f.read().split("__global__")[1:]
    arrays = 0
    for text in kernels:
        declared = re.findall(r"__shared__[^;]*?(\w+)(?:\[[^;]*)?;", text)
        filled = re.findall(r"poison_lds<[^;]*>\((\w+)\);", text)
        assert sorted(declared) == sorted(filled), text[:120]
        arrays += len(declared)
    assert (arrays > 0) == (src in build.LDS_SOURCES)
