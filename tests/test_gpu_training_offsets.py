"""Row buffers of more than 2^31 elements: what lies behind that offset is read and written where it belongs."""
import pytest

pytestmark = pytest.mark.gpu


def _plan(T, k, E, bm):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.int()
    plan = moe.moe_align(ids, E, bm)
    return g, ids, plan, moe.moe_route_slots(plan[0], plan[2], T, k)


def test_rows_behind_2_31_elements():
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, E, bm, K = 66000, 8, 16, 128, 4096
    g, ids, plan, slots = _plan(T, k, E, bm)
    assert plan[0].numel() * K > 2 ** 31
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    rows = moe.moe_permute(x, plan[0], plan[2], slots)
    at = torch.cat((slots[-40:].flatten(), slots[:40].flatten())).long()
    tok = torch.cat((torch.arange(T - 40, T), torch.arange(40))).repeat_interleave(k).cuda()
    assert int(at.max()) * K > 2 ** 31 and torch.equal(rows[at], x[tok])
    # every token's rows are its own: the sum is k times x, exactly; with weights 1 the same, and the dot products
    assert torch.equal(moe.moe_permute_backward(rows, slots), (x.float() * k).bfloat16())
    tw = torch.ones((T, k), device="cuda")
    assert torch.equal(moe.moe_unpermute(rows, slots, tw), (x.float() * k).bfloat16())
    gy, gw = moe.moe_unpermute_backward(x, rows, plan[0], plan[2], slots, tw)
    n = int(plan[2])
    assert torch.equal(gy[:n], rows[:n])
    ref = (x.double() ** 2).sum(1, keepdim=True)  # 4096 squares summed in fp32: 4096 * 2^-23 of the sum
    assert bool(((gw.double() - ref).abs() <= 4096 * 2.0 ** -23 * ref).all())


@pytest.mark.parametrize("bm", [16, 128])
def test_products_behind_2_31_elements(bm):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, E, K, N = 66000, 8, 16, 64, 4096
    g, ids, plan, slots = _plan(T, k, E, bm)
    cap, n = plan[0].numel(), int(plan[2])
    assert (n - 1) * N > 2 ** 31
    rows = torch.randn((cap, K), generator=g, device="cuda").bfloat16()
    w1 = (torch.randn((E, N, K), generator=g, device="cuda") * K ** -0.5).bfloat16()
    h, act = moe.moe_expert_up(rows, w1, *plan, bm)
    last = torch.arange(n - 256, n, device="cuda")
    live = last[plan[0][n - 256:n] >= 0]
    ref = rows[live].double() @ w1[E - 1].double().T
    slack = K * 2.0 ** -23 * (rows[live].double().abs() @ w1[E - 1].double().abs().T)
    assert bool(((h[live].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + slack).all())
    # the rows' gradient and the last expert's weights' gradient, from h as a gradient
    grows, gw1 = moe.moe_expert_up_backward(h, rows, w1, *plan, bm)
    moe.moe_device_status()
    hd = h[live].double()
    ref = hd @ w1[E - 1].double()
    slack = N * 2.0 ** -23 * (hd.abs() @ w1[E - 1].double().abs())
    assert bool(((grows[live].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + slack).all())
    expert = plan[1].long().repeat_interleave(bm)[:cap]
    at = torch.nonzero((plan[0] >= 0) & (expert == E - 1)).squeeze(1)
    hd, xd = h[at].double(), rows[at].double()
    ref = hd.T @ xd
    slack = len(at) * 2.0 ** -23 * (hd.abs().T @ xd.abs())
    assert bool(((gw1[E - 1].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + slack).all())
