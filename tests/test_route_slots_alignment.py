"""moe_route_slots refuses int32 pointers that are not 4-byte aligned, before any launch (CPU), as the calls beside it do."""
import pytest

import mixture_experts_ffn_planner_b200 as moe

ALIGNMENT = -3
P = 1 << 20


@pytest.mark.parametrize("ids,total,slots", [(P + 2, P, P), (P, P + 1, P), (P, P, P + 2)])
def test_misaligned(ids, total, slots):
    lib = moe.load()
    assert lib.moe_route_slots(ids, total, 64, 4, 2, slots, None) == ALIGNMENT
    assert lib.moe_last_error().startswith(b"moe_route_slots")
