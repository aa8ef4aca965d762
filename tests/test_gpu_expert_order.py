"""expert_order of more received rows than the small cases reach."""
import pytest
import torch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

import combine_get_dispatch_histogram_amd as miep  # noqa: E402
from test_gpu_experts import DEV, i32, say  # noqa: E402


@pytest.mark.parametrize("K", [1, 3])
def test_rows_from_two_to_the_24_on(K):
    """2^24 + 100 received rows: their numbers come out of a division of entries by K."""
    say("order past 2^24 rows", K)
    rows, R, L = 2 ** 24 + 100, 2, 3
    split = 2 ** 23 + 17
    g = torch.Generator(device=DEV).manual_seed(K)
    topk = torch.randint(-1, L, (rows, K), generator=g, device=DEV)
    order = miep.expert_order(topk, i32([0, split, rows]), R * L)
    expert = torch.where(topk >= 0, topk, R * L)
    expert[split:] = torch.where(topk[split:] >= 0, topk[split:] + L, R * L)
    by, at = torch.sort(expert.reshape(-1), stable=True)
    live = int((by < R * L).sum())
    count = torch.bincount(by[:live], minlength=R * L)
    assert torch.equal(order.group_rows.long(), count)
    assert torch.equal(order.group_begin.long(), count.cumsum(0) - count)
    assert torch.equal(order.slot_row[:live].long(), at[:live] // K)
    assert bool((order.slot_row[live:] == -1).all())
    slot = torch.full((rows * K,), -1, dtype=torch.int64, device=DEV)
    slot[at[:live]] = torch.arange(live, device=DEV)
    assert torch.equal(order.row_slot.long(), slot.view(rows, K))
