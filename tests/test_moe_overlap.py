"""CPU: the sort's outputs and working memory must not lie on its ids: of few
assignments every workgroup reads all of them, while others already write their
rows."""
import pytest
import torch

from fp8_fine_grained_fp8bs_amd import fp8bs


def sort(ids, offsets, slot, ws=None):
    fp8bs.fp8bs_moe_sort(ids, 0, slot.numel(), offsets, slot, ws)


def dispatch(ids, offsets, slot, ws=None):
    rows = slot.numel()
    fp8bs.fp8bs_moe_dispatch(fp8bs.SRC_BF16, torch.zeros((len(slot), 128), dtype=torch.bfloat16), None, ids, 0, offsets,
                             slot, torch.zeros((rows, 128), dtype=torch.uint8), torch.zeros((rows, 1)), None, ws)


def buffer():
    return torch.zeros(64, dtype=torch.int32)


def refused(call, *args):
    with pytest.raises(ValueError, match="must not overlap ids"):
        call(*args)


def taken(call, *args):
    """As far as host tensors are."""
    with pytest.raises(ValueError, match="on the GPU|cuda|device"):
        call(*args)


@pytest.mark.parametrize("call", [sort, dispatch])
def test_outputs_on_the_ids(call):
    b = buffer()
    ids, offsets, slot = b[:8].view(4, 2), torch.zeros(9, dtype=torch.int32), torch.zeros((4, 2), dtype=torch.int32)
    refused(call, ids, offsets, ids)
    refused(call, ids, offsets, b[7:15].view(4, 2))
    refused(call, ids, b[:9], slot)
    refused(call, ids, offsets, slot, b[4:].view(torch.uint8))
    refused(call, b[:16].view(torch.int64).view(4, 2), offsets, b[8:16].view(4, 2))


@pytest.mark.parametrize("call", [sort, dispatch])
def test_outputs_beside_the_ids(call):
    b = buffer()
    taken(call, b[:8].view(4, 2), b[16:25], b[8:16].view(4, 2), b[25:].view(torch.uint8))
    taken(call, b[8:16].view(4, 2), b[16:25], b[:8].view(4, 2))


@pytest.mark.parametrize("call", [sort, dispatch])
def test_wider_rows_of_ids(call):
    """Between two rows of ids there is room; on one there is none."""
    b = buffer()
    ids, offsets = b.view(2, 32)[:, :2], torch.zeros(3, dtype=torch.int32)
    for at in (0, 1, 29, 32, 33):
        refused(call, ids, offsets, b[at:at + 4].view(2, 2))
    for at in (2, 10, 28, 34, 60):
        taken(call, ids, offsets, b[at:at + 4].view(2, 2))
