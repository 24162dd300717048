"""Token rows in expert order and back (moe_permute, moe_unpermute) and their gradients, against the formulas in
64 bits.

Tolerances.  A copy is exact.  A sum over a token's k routes is formed in fp32 (one fma a route, each off by at
most 2^-24 of the partial sum, which sum |w y| bounds) and rounded once to the row type: |error| <= half a step of
the row type relative to the value + k * 2^-24 * sum |w y|, taken twice to cover the rounding of the bound's own
terms.  A product w * g has one fp32 rounding and one to the row type.  A dot product over K elements runs as a chain
of at most K / 32 + 8 fmas a thread (a token has at least 32 threads and vectors of at most 8), 5 additions between
lanes and at most 8 between warps: |error| <= (K / 32 + 21) * 2^-24 * sum |g y|.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SENTINEL = 7.0


def _plan(T, k, E, bm, seed, drop=0.2):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    rng = np.random.default_rng(seed)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[rng.random((T, k)) < drop] = -1
    if T > 2:
        ids[1, :] = E + 3          # a token that keeps no route
    w = torch.from_numpy((rng.random((T, k)) - 0.3).astype(np.float32)).cuda()
    s_ids, e_ids, ntpp = moe.moe_align(torch.from_numpy(ids).cuda(), E, bm)
    slots = moe.moe_route_slots(s_ids, ntpp, T, k)
    return s_ids, ntpp, slots, w


def _check(got, ref, slack):
    import torch

    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    lim = half * ref.abs() + slack
    assert bool(torch.isfinite(got).all())
    assert bool((err <= lim).all()), f"worst {float((err - lim).max()):.3e} over its bound"


SHAPES = [
    # T, k, E, bm, K
    (1, 1, 1, 16, 1), (1, 8, 16, 128, 4096), (3, 2, 4, 64, 33), (64, 2, 8, 64, 1024), (300, 6, 48, 32, 1001),
    (257, 8, 64, 16, 72), (129, 11, 40, 16, 264), (31, 3, 300, 128, 7168), (500, 4, 5, 128, 30),
]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("T,k,E,bm,K", SHAPES)
def test_rows_by_expert_and_back(T, k, E, bm, K, dtype):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    dt = getattr(torch, dtype)
    s_ids, ntpp, slots, w = _plan(T, k, E, bm, seed=T * 7 + K)
    g = torch.Generator(device="cuda").manual_seed(T + K)
    cap, n = s_ids.numel(), int(ntpp)
    ids = s_ids.long()
    # the slots invert the planner's order
    flat = slots.reshape(-1).long()
    have = flat >= 0
    assert torch.equal(ids[flat[have]], torch.nonzero(have).squeeze(1))
    assert int(have.sum()) == int((ids >= 0).sum())

    x = torch.randn((T, K), generator=g, device="cuda").to(dt)
    rows = torch.full((cap, K), SENTINEL, dtype=dt, device="cuda")
    assert moe.moe_permute(x, s_ids, ntpp, slots, out=rows) is rows
    want = torch.where((ids >= 0).unsqueeze(1), x[ids.clamp(min=0) // k], torch.zeros((), dtype=dt, device="cuda"))
    assert torch.equal(rows[:n], want[:n])
    assert bool((rows[n:] == SENTINEL).all())

    # padding and tail rows of y hold NaN: nothing may read them
    y = torch.randn((cap, K), generator=g, device="cuda").to(dt)
    y[ids < 0] = float("nan")
    yd = torch.where((flat >= 0).view(T, k, 1), y[flat.clamp(min=0)].view(T, k, K).double(), 0.0)
    out = moe.moe_unpermute(y, slots, w)
    wd = w.double().unsqueeze(2)
    _check(out, (wd * yd).sum(1), 2 * k * 2.0 ** -24 * (wd * yd).abs().sum(1))
    gx = moe.moe_permute_backward(y, slots)
    _check(gx, yd.sum(1), 2 * k * 2.0 ** -24 * yd.abs().sum(1))

    go = torch.randn((T, K), generator=g, device="cuda").to(dt)
    gy = torch.full((cap, K), SENTINEL, dtype=dt, device="cuda")
    gy2, gw = moe.moe_unpermute_backward(go, y, s_ids, ntpp, slots, w, grad_y=gy)
    assert gy2 is gy and bool((gy[n:] == SENTINEL).all())
    wr = torch.where(ids >= 0, w.reshape(-1).double()[ids.clamp(min=0)], 0.0).unsqueeze(1)
    ref = wr * go.double()[ids.clamp(min=0) // k]
    _check(gy[:n], ref[:n], 2.0 ** -23 * ref[:n].abs())
    terms = yd * go.double().unsqueeze(1)
    err = (gw.double() - terms.sum(2)).abs()
    assert bool((err <= (K / 32 + 21) * 2.0 ** -24 * terms.abs().sum(2)).all())
    assert bool((gw[slots < 0] == 0).all())


def test_gradients_against_differences():
    """unpermute(permute(x) * c) is linear in x and in the weights: a central difference of the loss is the
    gradient's product with the direction up to fp32 rounding (|loss terms| * 2^-22 / h, h = 1/4)."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, E, bm, K = 37, 3, 6, 16, 40
    s_ids, ntpp, slots, w = _plan(T, k, E, bm, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    n = int(ntpp)
    x, dx, co = (torch.randn((T, K), generator=g, device="cuda") for _ in range(3))
    dw = torch.randn((T, k), generator=g, device="cuda")
    c = torch.randn((s_ids.numel(), K), generator=g, device="cuda")
    zeros = lambda: torch.zeros((s_ids.numel(), K), device="cuda")  # noqa: E731

    def loss(x_, w_):
        y = moe.moe_permute(x_, s_ids, ntpp, slots, out=zeros()) * c
        return float((moe.moe_unpermute(y, slots, w_).double() * co.double()).sum())

    y = moe.moe_permute(x, s_ids, ntpp, slots, out=zeros()) * c
    gy, gw = moe.moe_unpermute_backward(co, y, s_ids, ntpp, slots, w, grad_y=zeros())
    gx = moe.moe_permute_backward(gy * c, slots)
    h = 0.25
    scale = float((y[:n].double().abs().sum() + 1) * co.abs().max())
    tol = scale * 2.0 ** -22 / h
    assert abs((loss(x + h * dx, w) - loss(x - h * dx, w)) / (2 * h) - float((gx.double() * dx.double()).sum())) < tol
    assert abs((loss(x, w + h * dw) - loss(x, w - h * dw)) / (2 * h) - float((gw.double() * dw.double()).sum())) < tol


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_unaligned_views_and_no_tokens(dtype):
    """Contiguous views that start off a 16-byte boundary take narrower accesses; no tokens is a valid call."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    dt = getattr(torch, dtype)
    T, k, E, bm, K = 50, 4, 8, 32, 64
    s_ids, ntpp, slots, w = _plan(T, k, E, bm, seed=5)
    n, cap = int(ntpp), s_ids.numel()
    for off in (1, 2, 4):
        x = torch.randn(T * K + off, device="cuda").to(dt)[off:].view(T, K)
        y = torch.randn(cap * K + off, device="cuda").to(dt)[off:].view(cap, K)
        assert torch.equal(moe.moe_permute(x, s_ids, ntpp, slots)[:n],
                           moe.moe_permute(x.clone(), s_ids, ntpp, slots)[:n])
        assert torch.equal(moe.moe_unpermute(y, slots, w), moe.moe_unpermute(y.clone(), slots, w))
        a, b = moe.moe_unpermute_backward(x, y, s_ids, ntpp, slots, w), \
            moe.moe_unpermute_backward(x.clone(), y.clone(), s_ids, ntpp, slots, w)
        assert torch.equal(a[0][:n], b[0][:n])
        torch.testing.assert_close(a[1], b[1], rtol=0, atol=K * 2.0 ** -20)  # the sums' order follows the vector width
    s_ids, ntpp, slots, w = _plan(0, k, E, bm, seed=5)
    x = torch.empty((0, K), dtype=dt, device="cuda")
    rows = torch.full((s_ids.numel(), K), SENTINEL, dtype=dt, device="cuda")
    moe.moe_permute(x, s_ids, ntpp, slots, out=rows)
    assert bool((rows == SENTINEL).all())
    assert moe.moe_unpermute(rows, slots, w).shape == (0, K)
    assert moe.moe_permute_backward(rows, slots).shape == (0, K)


def test_bad_slots_and_ids_are_skipped():
    """Slots outside the row buffer count as none and ids outside the routes as padding: no access leaves the
    buffers (the kernels check both)."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, K = 4, 2, 16
    s_ids = torch.tensor([0, 99, -5, 3], dtype=torch.int32, device="cuda")
    ntpp = torch.tensor([1000], dtype=torch.int32, device="cuda")
    assert moe.moe_route_slots(s_ids, ntpp, T, k).tolist() == [[0, -1], [-1, 3], [-1, -1], [-1, -1]]
    slots = torch.tensor([[0, 4], [2 ** 31 - 1, 3], [-7, -1], [-1, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn((T, K), device="cuda")
    rows = moe.moe_permute(x, s_ids, ntpp, slots)
    assert torch.equal(rows[[0, 3]], x[[0, 1]]) and bool((rows[1:3] == 0).all())
    w = torch.ones((T, k), device="cuda")
    out = moe.moe_unpermute(rows, slots, w)
    assert torch.equal(out[:2], x[:2]) and bool((out[2:] == 0).all())


def test_other_stream_and_graph_replay():
    """On a stream of its own, and captured once and replayed on new values: the same results."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, E, bm, K = 200, 4, 16, 64, 512
    s_ids, ntpp, slots, w = _plan(T, k, E, bm, seed=9)
    cap, n = s_ids.numel(), int(ntpp)
    x = torch.randn((T, K), device="cuda").bfloat16()
    want_rows = moe.moe_permute(x, s_ids, ntpp, slots)[:n].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_permute(x, s_ids, ntpp, slots, stream=side)
    raw = moe.moe_permute(x, s_ids, ntpp, slots, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got[:n], want_rows) and torch.equal(raw[:n], want_rows)

    rows = torch.zeros((cap, K), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros((T, K), dtype=torch.bfloat16, device="cuda")
    gy, gw = torch.zeros_like(rows), torch.zeros((T, k), device="cuda")
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            moe.moe_permute(x, s_ids, ntpp, slots, out=rows)
            moe.moe_unpermute(rows, slots, w, out=out)
            moe.moe_unpermute_backward(out, rows, s_ids, ntpp, slots, w, grad_y=gy, grad_weights=gw)
    x.copy_(torch.randn((T, K), device="cuda"))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    rows2 = moe.moe_permute(x, s_ids, ntpp, slots)
    assert torch.equal(rows[:n], rows2[:n]) and torch.equal(out, moe.moe_unpermute(rows2, slots, w))
    gy2, gw2 = moe.moe_unpermute_backward(out, rows2, s_ids, ntpp, slots, w)
    assert torch.equal(gy[:n], gy2[:n]) and torch.equal(gw, gw2)
