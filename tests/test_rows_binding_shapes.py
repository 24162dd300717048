"""Tensors without dimensions where the row operators expect two: refused as every other wrong shape is (CPU)."""
import pytest
import torch

import mixture_experts_ffn_planner_b200 as moe

SCALAR = torch.zeros((), dtype=torch.int32)
SLOTS = torch.zeros((4, 2), dtype=torch.int32)
IDS, TOTAL = torch.zeros(16, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
X, ROWS, W = torch.zeros(4, 8), torch.zeros(16, 8), torch.zeros(4, 2)


@pytest.mark.parametrize("call", [
    lambda: moe.moe_permute(X, IDS, TOTAL, SCALAR, out=ROWS),
    lambda: moe.moe_permute(X, IDS, TOTAL, SLOTS, out=torch.zeros(())),
    lambda: moe.moe_permute(torch.zeros(()), IDS, TOTAL, SLOTS, out=ROWS),
    lambda: moe.moe_permute_backward(ROWS, SCALAR, out=X),
    lambda: moe.moe_permute_backward(torch.zeros(()), SLOTS, out=X),
    lambda: moe.moe_unpermute(ROWS, SCALAR, W, out=X),
    lambda: moe.moe_unpermute(torch.zeros(()), SLOTS, W, out=X),
    lambda: moe.moe_unpermute_backward(X, ROWS, IDS, TOTAL, SCALAR, W),
    lambda: moe.moe_expert_down(torch.zeros(()), torch.zeros((2, 8, 8), dtype=torch.bfloat16), SCALAR, IDS, TOTAL, 16),
])
def test_no_dimensions(call):
    with pytest.raises((ValueError, TypeError)):
        call()
