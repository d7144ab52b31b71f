"""Build invariants of the attention kernels (CPU only): the workgroups that a
launch counts on as resident fit a compute unit's registers and LDS."""
import functools
import os
import re
import shutil

import pytest

from fp8_fine_grained_fp8bs_amd import build

pytestmark = pytest.mark.skipif(shutil.which("hipcc") is None and not os.path.exists("/opt/rocm/bin/hipcc"),
                                reason="hipcc not available")

LDS = 160 * 1024


@functools.lru_cache(maxsize=None)
def kernels(src):
    """Demangled-enough name -> (VGPRs, LDS bytes)."""
    out = {}
    for m in re.finditer(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", build.asm(src), re.S):
        field = lambda f: int(re.search(rf"\.amdhsa_{f}\s+(\d+)", m.group(2)).group(1))  # noqa: E731
        out[m.group(1)] = (field("next_free_vgpr"), field("group_segment_fixed_size"))
    return out


# (source, name, template arguments, workgroups of 256 threads a compute unit)
RESIDENT = [("attn.hip", "attn_rows_kernel", d, n, 2) for d in (64, 128) for n in (1, 2)]
RESIDENT += [("attn_prompt.hip", "attn_prompt_kernel", 128, g, 2) for g in (16, 32, 64)]
RESIDENT += [("attn_prompt.hip", "attn_prompt_kernel", 64, g, 3 if g >= 32 else 2) for g in (16, 32, 64)]


@pytest.mark.parametrize("src,name,d,n,groups", RESIDENT)
def test_workers_are_resident(src, name, d, n, groups):
    found = [v for k, v in kernels(src).items() if f"{name}ILi{d}ELi{n}E" in k]
    assert len(found) == 1
    vgpr, lds = found[0]
    assert 512 // (-(-vgpr // 8) * 8) >= groups, f"{vgpr} registers"
    assert groups * lds <= LDS, f"{lds} bytes of LDS"
