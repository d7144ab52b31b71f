"""CPU: an append that rotates queries in place takes one row stride: with two,
a row's result would land on rows that other workgroups have yet to read."""
import pytest

from fp8_fine_grained_fp8bs_amd import fp8bs
from tests.test_attn_abi import A, append


@pytest.mark.parametrize("ldq,ldqo", [(512, 640), (768, 512)])
def test_in_place_queries_keep_their_stride(ldq, ldqo):
    assert append(q=A, qo=A, ldq=ldq, ldqo=ldqo) == fp8bs.ERR_INVALID_ARG

