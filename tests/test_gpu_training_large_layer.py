"""A layer whose weights hold far more than 2^31 elements: 384 experts of 4096 x 7168 and 7168 x 2048.  Few tokens, on the
first expert, one in the middle and the last; every other expert has no rows and gets a gradient of zeros.  Tolerances as
in test_gpu_expert_gemm.py and test_gpu_orthogonalize.py."""
import pytest

from test_gpu_expert_gemm import U, FAST, check
from test_gpu_orthogonalize import check as check_orthogonal, matrices, reference

pytestmark = pytest.mark.gpu

E, K, N, BM = 384, 7168, 4096, 64
EXPERTS = (0, 211, 383)


@pytest.fixture
def plan():
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    ids = torch.tensor([[EXPERTS[t % 3], EXPERTS[(t + 1) % 3]] for t in range(70)], dtype=torch.int32, device="cuda")
    s_ids, e_ids, total = moe.moe_align(ids, E, BM)
    expert = e_ids.long().repeat_interleave(BM)[: s_ids.numel()]
    at = {e: torch.nonzero((s_ids >= 0) & (expert == e)).squeeze(1) for e in EXPERTS}
    assert all(len(p) >= 46 for p in at.values())
    yield (s_ids, e_ids, total, BM), at, torch.Generator(device="cuda").manual_seed(8)
    torch.cuda.empty_cache()


def _weights(shape, g):
    import torch

    w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for e in range(shape[0]):  # by expert: the fp32 normals of a whole layer would not fit beside it
        w[e] = torch.randn(shape[1:], generator=g, device="cuda") * shape[-1] ** -0.5
    return w


def test_up_and_its_gradient(plan):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    p, at, g = plan
    cap = p[0].numel()
    w1 = _weights((E, N, K), g)
    rows = torch.randn((cap, K), generator=g, device="cuda").bfloat16()
    gh = torch.randn((cap, N), generator=g, device="cuda").bfloat16()
    h, act = moe.moe_expert_up(rows, w1, *p)
    gx, gw = moe.moe_expert_up_backward(gh, rows, w1, *p)
    moe.moe_device_status()
    for e, i in at.items():
        x, w, q = rows[i].double(), w1[e].double(), gh[i].double()
        rh, sh = x @ w.T, K * U * (x.abs() @ w.abs().T)
        gate, up = rh.chunk(2, 1)
        sg, su = sh.chunk(2, 1)
        silu = gate * torch.sigmoid(gate)
        check(h[i], rh, sh)
        check(act[i], silu * up, 1.1 * up.abs() * sg + silu.abs() * su + sg * su + FAST * (silu * up).abs())
        check(gx[i], q @ w, N * U * (q.abs() @ w.abs()))
        check(gw[e], q.T @ x, len(i) * U * (q.abs().T @ x.abs()))
    for e in range(E):
        assert e in at or int(torch.count_nonzero(gw[e])) == 0


def test_down_and_its_gradient(plan):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    p, at, g = plan
    cap, half = p[0].numel(), N // 2
    w2 = _weights((E, K, half), g)
    h = torch.randn((cap, N), generator=g, device="cuda").bfloat16()
    act = torch.randn((cap, half), generator=g, device="cuda").bfloat16()
    gy = torch.randn((cap, K), generator=g, device="cuda").bfloat16()
    y = moe.moe_expert_down(act, w2, *p)
    gw = torch.full((E, K, half), 2.0, device="cuda")
    gh, _ = moe.moe_expert_down_backward(gy, h, act, w2, *p, grad_w2=gw, accumulate=True)
    moe.moe_device_status()
    for e, i in at.items():
        a, w, q = act[i].double(), w2[e].double(), gy[i].double()
        check(y[i], a @ w.T, half * U * (a.abs() @ w.abs().T))
        ga, sga = q @ w, K * U * (q.abs() @ w.abs())
        gate, up = h[i].double().chunk(2, 1)
        s = torch.sigmoid(gate)
        check(gh[i], torch.cat((ga * up * s * (1 + gate * (1 - s)), ga * gate * s), 1),
              torch.cat((1.1 * up.abs() * sga + FAST * 2.6 * (ga * up).abs(),
                         (gate * s).abs() * sga + FAST * (ga * gate * s).abs()), 1))
        ref = q.T @ a
        err = (gw[e].double() - 2 - ref).abs()
        assert bool((err <= len(i) * U * (q.abs().T @ a.abs()) + U * (ref.abs() + 2)).all())
    for e in range(E):
        assert e in at or bool((gw[e] == 2).all())


@pytest.mark.parametrize("M,N", [(4096, 7168), (7168, 2048)])
def test_update(M, N):
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(1, M, N, "lowrank", "bfloat16")
    check_orthogonal(moe.moe_orthogonalize(g), reference(g))
    moe.moe_device_status()
