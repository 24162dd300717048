"""What the row operators refuse, before any launch (CPU): the C ABI by status, the binding by exception."""
import pytest
import torch

import mixture_experts_ffn_planner_b200 as moe

OK, INVALID, UNSUPPORTED, ALIGNMENT = 0, -1, -2, -3
P = 1 << 20  # a well-aligned stand-in for a device pointer: these calls return before it is used


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def test_sizes_and_types(lib):
    assert lib.moe_permute(P, 0, P, P, P, 64, -1, 2, 8, P, None) == INVALID
    assert lib.moe_permute(P, 0, P, P, P, 64, 4, 0, 8, P, None) == INVALID
    assert lib.moe_permute(P, 0, P, P, P, 64, 4, 2, 0, P, None) == INVALID
    assert lib.moe_permute(P, 0, P, P, P, -1, 4, 2, 8, P, None) == INVALID
    assert lib.moe_permute(P, 2, P, P, P, 64, 4, 2, 8, P, None) == UNSUPPORTED
    assert b"bf16 or fp32" in lib.moe_last_error()
    assert lib.moe_permute_backward(P, 0, P, 64, 1 << 30, 2, 8, P, None) == UNSUPPORTED
    assert lib.moe_unpermute(P, 0, P, P, 1 << 31, 4, 2, 8, P, None) == UNSUPPORTED
    assert lib.moe_route_slots(P, P, -1, 4, 2, P, None) == INVALID


def test_null_pointers(lib):
    assert lib.moe_permute(None, 0, P, P, P, 64, 4, 2, 8, P, None) == INVALID
    assert lib.moe_permute(P, 0, P, None, P, 64, 4, 2, 8, P, None) == INVALID
    assert lib.moe_permute(P, 0, P, P, P, 64, 4, 2, 8, None, None) == INVALID
    assert lib.moe_permute_backward(P, 0, None, 64, 4, 2, 8, P, None) == INVALID
    assert lib.moe_unpermute(P, 0, P, None, 64, 4, 2, 8, P, None) == INVALID
    assert lib.moe_unpermute_backward(P, None, 0, P, P, P, P, 64, 4, 2, 8, P, P, None) == INVALID
    assert lib.moe_unpermute_backward(P, P, 0, P, P, P, P, 64, 4, 2, 8, P, None, None) == INVALID
    assert lib.moe_route_slots(P, P, 64, 4, 2, None, None) == INVALID


def test_alignment(lib):
    assert lib.moe_permute(P + 1, 0, P, P, P, 64, 4, 2, 8, P, None) == ALIGNMENT
    assert lib.moe_permute(P, 1, P, P, P, 64, 4, 2, 8, P + 2, None) == ALIGNMENT
    assert lib.moe_unpermute(P, 0, P + 2, P, 64, 4, 2, 8, P, None) == ALIGNMENT


def test_nothing_to_do(lib):
    assert lib.moe_permute(None, 0, None, None, None, 0, 0, 2, 8, None, None) == OK
    assert lib.moe_permute_backward(None, 0, None, 64, 0, 2, 8, None, None) == OK
    assert lib.moe_unpermute(None, 0, None, None, 64, 0, 2, 8, None, None) == OK
    assert lib.moe_route_slots(None, None, 64, 0, 2, None, None) == OK


def test_binding_refuses():
    slots = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_unpermute(torch.zeros(8, 16), slots, torch.zeros(4, 2))
    with pytest.raises(TypeError, match="y: dtype"):
        moe.moe_unpermute(torch.zeros(8, 16, dtype=torch.float16), slots, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="two dimensions"):
        moe.moe_permute_backward(torch.zeros(8), slots)
    with pytest.raises(ValueError, match="slots must be"):
        moe.moe_permute_backward(torch.zeros(8, 16), slots.view(-1))
    with pytest.raises(TypeError, match="slots: dtype"):
        moe.moe_permute_backward(torch.zeros(8, 16), slots.long())
    with pytest.raises(ValueError, match="sorted_token_ids is required"):
        moe.moe_route_slots(None, torch.zeros(1, dtype=torch.int32), 4, 2)
