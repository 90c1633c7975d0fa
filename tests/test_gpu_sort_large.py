"""The stable sort of slots by expert where many workgroups share it, against torch's stable sort."""
import pytest
import torch

import microscaling_weight_quantization_amd as mxq

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("slots", [2048 * 32 - 5, 2048 * 32, 2048 * 32 + 1, 2048 * 256, 2048 * 256 + 1, 2048 * 1031 + 77, 1 << 24])
@pytest.mark.parametrize("n", [1, 63, 64, 511, 512])
def test_sort_by_many_workgroups(slots, n):
    """Workgroups of 2048 slots add up each other's counts of n + 1 experts up to 16384 of them; beyond, a launch does."""
    ids = torch.randint(-1, n + 1, (slots, 1), generator=torch.Generator().manual_seed(n), dtype=torch.int32).to(DEV)
    offsets, order, position = mxq.mxq_sort_experts(ids, n)
    key = torch.where((ids >= 0) & (ids < n), ids, n).view(-1)
    sorted_key, want = key.sort(stable=True)
    assert torch.equal(offsets.long(), torch.searchsorted(sorted_key, torch.arange(n + 1, dtype=torch.int32, device=DEV)))
    kept = sorted_key < n
    assert torch.equal(order.long(), torch.where(kept, want, ~want))
    place = torch.empty_like(want)
    place[want] = torch.where(kept, torch.arange(slots, device=DEV), ~torch.arange(slots, device=DEV))
    assert torch.equal(position.view(-1).long(), place)
