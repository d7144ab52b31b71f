"""Dispatch and gather without an output to write are refused, whichever way they
are called: without rows to count, a sort into none would leave every
assignment without a row."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs


def operands(device, T=6, k=2, C=128, E=4):
    x = torch.zeros((T, C), dtype=torch.bfloat16, device=device)
    ids, slot = (torch.zeros((T, k), dtype=torch.int32, device=device) for _ in range(2))
    return x, ids, slot, torch.zeros(E + 1, dtype=torch.int32, device=device)


def test_entry_points():
    x, ids, slot, offsets = operands("cpu")
    with pytest.raises(ValueError, match="no output"):
        fp8bs.fp8bs_moe_gather(fp8bs.SRC_BF16, x, None, slot, None, None, None)
    with pytest.raises(ValueError, match="no output"):
        fp8bs.fp8bs_moe_dispatch(fp8bs.SRC_BF16, x, None, ids, 0, offsets, slot, None, None, None, None)


def test_only_codes_or_only_scales():
    x, ids, slot, offsets = operands("cpu")
    q, s = torch.zeros((12, 128), dtype=torch.uint8), torch.zeros((12, 1))
    for given in ((q, None), (None, s)):
        with pytest.raises(ValueError, match="both or neither|no output"):
            fp8bs.fp8bs_moe_gather(fp8bs.SRC_BF16, x, None, slot, *given, None)
        with pytest.raises(ValueError, match="both or neither|no output"):
            fp8bs.fp8bs_moe_dispatch(fp8bs.SRC_BF16, x, None, ids, 0, offsets, slot, *given, None, None)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [None, (None, None, None)])
def test_helpers(out):
    x, ids, slot, _ = operands("cuda")
    for stream in (None, torch.cuda.current_stream()):
        with pytest.raises((ValueError, fp8bs.Fp8bsError)):
            fp8bs.moe_dispatch(x, ids, 4, codes=False, out=out, stream=stream)
        with pytest.raises((ValueError, fp8bs.Fp8bsError)):
            fp8bs.moe_gather(x, slot, codes=False, out=out, stream=stream)


@pytest.mark.gpu
def test_outputs_of_no_rows():
    """Buffers without rows are outputs: every assignment is without one."""
    x, ids, _, _ = operands("cuda")
    q, s, _, offsets, slot = fp8bs.moe_dispatch(x, ids, 4, rows=0)
    assert q.shape == (0, 128) and not offsets.any() and (slot == -1).all()
    q, s, _, offsets, slot = fp8bs.moe_dispatch(x, ids, 4, out=(q, s, None), stream=torch.cuda.current_stream())
    assert not offsets.any() and (slot == -1).all()
