"""The training operators at the ends of what they take: the largest number of experts, a token routed to one expert more
than once, in-place updates of large matrices, and many shapes drawn by chance.  Checks and tolerances are those of the
operators' own tests."""
import random

import pytest

import test_gpu_expert_gemm as products
import test_gpu_orthogonalize as updates
import test_gpu_permute as rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,bm,K,N", [(600, 3, 16, 64, 64), (40, 2, 128, 24, 32), (2100, 8, 32, 8, 16)])
def test_most_experts(T, k, bm, K, N):
    products.test_forward(T, k, 1024, bm, K, N)
    products.test_backward(T, k, 1024, bm, K, N)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("K", [8, 33, 640])
def test_one_expert_more_than_once(K, dtype):
    """Whole numbers, so that every sum is exact."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    dt = getattr(torch, dtype)
    T, k, E, bm = 75, 5, 4, 16
    g = torch.Generator(device="cuda").manual_seed(K)
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[0] = 2                                      # all routes of a token to one expert
    s_ids, _, total = moe.moe_align(ids, E, bm)
    slots = moe.moe_route_slots(s_ids, total, T, k)
    assert len(set(slots.flatten().tolist())) == T * k and int(slots.min()) >= 0
    x = torch.randint(-9, 10, (T, K), generator=g, device="cuda").to(dt)
    r = moe.moe_permute(x, s_ids, total, slots)
    assert torch.equal(r[slots.long()], x.unsqueeze(1).expand(T, k, K))
    assert torch.equal(moe.moe_permute_backward(r, slots), x * k)
    w = torch.randint(-2, 3, (T, k), generator=g, device="cuda").float()
    assert torch.equal(moe.moe_unpermute(r, slots, w), (x.float() * w.sum(1, keepdim=True)).to(dt))
    gy, gw = moe.moe_unpermute_backward(x, r, s_ids, total, slots, w)
    assert torch.equal(gy[slots.long()], (x.float().unsqueeze(1) * w.unsqueeze(2)).to(dt))
    assert torch.equal(gw, (x.double() ** 2).sum(1, keepdim=True).float().expand(T, k))


@pytest.mark.parametrize("M,N", [(300, 520), (520, 300), (777, 513), (260, 264)])
def test_large_updates_in_place(M, N):
    updates.test_in_place_unaligned_stream_and_graph(M, N)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_products(seed):
    rng = random.Random(seed)
    bm, E = rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 5, 13, 40, 90))
    k = rng.randint(1, max(1, min(4, E // 2)))
    T, K, N = rng.choice((1, 7, 60, 333, 1500, 4000)), 8 * rng.randint(1, 130), 16 * rng.randint(1, 70)
    products.test_forward(T, k, E, bm, K, N)
    products.test_backward(T, k, E, bm, K, N)


@pytest.mark.parametrize("seed", range(8))
def test_drawn_rows(seed):
    rng = random.Random(100 + seed)
    E = rng.randint(1, 300)
    k = rng.randint(1, min(12, E))
    T, K = rng.choice((1, 2, 17, 200, 900)), rng.choice((1, 3, 64, 100, 511, 2050, 5000))
    for dtype in ("bfloat16", "float32"):
        rows.test_rows_by_expert_and_back(T, k, E, rng.choice((16, 32, 64, 128)), K, dtype)


@pytest.mark.parametrize("seed", range(10))
def test_drawn_updates(seed):
    rng = random.Random(200 + seed)
    E, M, N = rng.choice((1, 3, 20)), rng.randint(1, 700), rng.randint(1, 700)
    updates.test_matches_the_iteration(E, M, N, rng.choice(("gauss", "lowrank", "decades")), rng.choice(("bfloat16", "float32")))
