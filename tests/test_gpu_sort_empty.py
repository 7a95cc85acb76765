"""A batch without tokens: the plan is empty and nothing is read."""
import pytest
import torch

import mixture_experts_forward_moe_amd as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("order", [moe.ROUTE_ORDER_AUTO, moe.ROUTE_ORDER_SINGLE, moe.ROUTE_ORDER_SPAN])
def test_empty_batch(order):
    print("sort of an empty batch", order, flush=True)
    ids = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    plan = moe.moe_sort(ids, 4, 4, 0, 16, route_order=order)
    torch.cuda.synchronize()
    assert plan.route_slots == 0 and int(plan.num_tiles) == 0
    assert plan.expert_counts.tolist() == [0] * 4 and plan.expert_offsets.tolist() == [0] * 5
