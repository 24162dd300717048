"""Rows next to 2^31 elements, the longest that the row operators take: one token of two routes, whose rows lie in the
order [route 1, route 0, padding].  Odd, so that every element is an access of its own and indices go as far as they can."""
import pytest

pytestmark = pytest.mark.gpu

K = 2 ** 31 - 1
AT = (0, 1, 2 ** 20 + 7, 2 ** 30 + 1, 2145386496, K - 1000, K - 600, K - 513, K - 512, K - 257, K - 33, K - 2, K - 1)


@pytest.fixture
def plan():
    import torch

    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    yield i32([1, 0, -1]), i32([3]), i32([[1, 0]])
    torch.cuda.empty_cache()


def _row(dtype):
    import torch

    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty((1, K), dtype=dtype, device="cuda")
    return x.random_(-120, 120, generator=g)  # whole numbers: every sum below is exact


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_copies_and_sums(plan, dtype):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    ids, total, slots = plan
    x = _row(getattr(torch, dtype))
    rows = torch.full((3, K), 7.0, dtype=x.dtype, device="cuda")
    moe.moe_permute(x, ids, total, slots, out=rows)
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[1], x[0])
    assert int(torch.count_nonzero(rows[2])) == 0
    rows[2] = float("nan")
    out = torch.full_like(x, 7.0)
    moe.moe_permute_backward(rows, slots, out=out)
    assert torch.equal(out, x + x)
    out.fill_(7.0)
    moe.moe_unpermute(rows, slots, torch.tensor([[2.0, -1.0]], device="cuda"), out=out)
    assert torch.equal(out, x)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_weighted_sum_backward(plan, dtype):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    ids, total, slots = plan
    x = _row(getattr(torch, dtype))
    y = torch.zeros((3, K), dtype=x.dtype, device="cuda")
    at = torch.tensor(AT, device="cuda")
    y[1, at] = 1.0
    y[0, at] = torch.arange(1, len(AT) + 1, device="cuda").to(x.dtype)
    y[2] = float("nan")
    grad_y = torch.full_like(y, 7.0)
    w = torch.tensor([[2.0, -1.0]], device="cuda")
    _, gw = moe.moe_unpermute_backward(x, y, ids, total, slots, w, grad_y=grad_y)
    assert torch.equal(grad_y[1], x[0] * 2) and torch.equal(grad_y[0], -x[0])
    assert int(torch.count_nonzero(grad_y[2])) == 0
    picked = x[0, at].double()
    want = [float(picked.sum()), float((picked * torch.arange(1, len(AT) + 1, device="cuda")).sum())]
    assert gw[0].tolist() == want
