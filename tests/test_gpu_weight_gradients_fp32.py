"""fp32 weight gradients, written and added to, at sizes whose products run on pairs of CTAs (and, for comparison, on single
ones): tails in both directions, experts without rows, NaN in all padding, nothing written beside the buffer.

Tolerance: products of bf16 values are exact in fp32, and a sum of n of them is off by at most n * 2^-23 * sum |a b|,
whatever its order and whether an addition rounds or truncates.  It is stored as it is; adding it to a buffer rounds once
more, by at most 2^-24 of the result, which the sum's own error moves too: 2^-23 of |start| + |sum| covers both."""
import pytest

from test_gpu_expert_gemm import U, Case

pytestmark = pytest.mark.gpu

SHAPES = [
    # T, k, E, bm, K, N: E * N * K and E * K * N / 2 of at least 24 tiles of 256 x 256, or fewer
    (900, 3, 24, 128, 264, 1040),
    (900, 3, 24, 16, 264, 1040),
    (2500, 4, 30, 64, 520, 528),
    (4, 2, 200, 32, 136, 272),       # nearly all experts without rows
    (1500, 1, 3, 128, 1032, 1040),   # many chunks an expert
    (70, 2, 5, 16, 72, 48),          # single CTAs
]


def _guarded(shape, start):
    """A buffer of `shape` between two stretches of sentinels: (all of it, the view)."""
    import torch

    n = start.numel()
    whole = torch.full((n + 512,), -7.0, device="cuda")
    view = whole[256:256 + n].view(shape)
    view.copy_(start)
    return whole, view


@pytest.mark.parametrize("T,k,E,bm,K,N", SHAPES)
def test_written_and_added(T, k, E, bm, K, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Case(T, k, E, bm, K, N, drop=0.05, skip=True, seed=T + N)
    rows, w1, w2 = c.rows(K), c.weights(E, N, K), c.weights(E, K, N // 2)
    gy, h, act, gh = c.rows(K), c.rows(N), c.rows(c.half), c.rows(N)
    calls = (((E, N, K), gh, rows, lambda **kw: moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, **kw)[1], "grad_w1"),
             ((E, K, N // 2), gy, act, lambda **kw: moe.moe_expert_down_backward(gy, h, act, w2, *c.plan, bm, **kw)[1],
              "grad_w2"))
    for shape, a, b, call, name in calls:
        start = torch.randn(shape, generator=c.g, device="cuda")
        whole, new = _guarded(shape, start)
        assert call(**{name: new}) is new
        whole2, add = _guarded(shape, start)
        call(**{name: add, "accumulate": True})
        moe.moe_device_status()
        for w in (whole, whole2):
            assert bool((w[:256] == -7).all()) and bool((w[-256:] == -7).all())
        once = add.clone()
        call(**{name: add, "accumulate": True})
        for e, p in c.by_expert():
            x, y = a[p].double(), b[p].double()
            ref, slack = x.T @ y, len(p) * U * (x.abs().T @ y.abs())
            assert bool(((new[e].double() - ref).abs() <= slack).all())
            first = start[e].double()
            assert bool(((once[e].double() - first - ref).abs() <= slack + U * (first.abs() + ref.abs())).all())
            # a second time from what the first left: the same sum, rounded once more
            err = (add[e].double() - once[e].double() - ref).abs()
            assert bool((err <= slack + U * (once[e].double().abs() + ref.abs())).all())
            if len(p) == 0:
                assert bool((new[e] == 0).all()) and torch.equal(once[e], start[e]) and torch.equal(add[e], start[e])
        # the bf16 gradient is the fp32 one, rounded
        assert torch.equal(call(), new.bfloat16())
        for _ in range(10):
            again = torch.full_like(new, 3.0)
            call(**{name: again})
            assert torch.equal(again, new)


def test_captured_and_on_streams_of_their_own():
    """A captured accumulation adds once a replay; two streams with buffers of their own do not meet."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    T, k, E, bm, K, N = 900, 3, 24, 64, 264, 1040
    c = Case(T, k, E, bm, K, N, seed=3)
    gh, rows, w1 = c.rows(N), c.rows(K), c.weights(E, N, K)
    gx = c.out(K)
    total = torch.zeros((E, N, K), device="cuda")
    one = moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, grad_rows=gx, grad_w1=torch.empty_like(total))[1]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, grad_rows=gx, grad_w1=total, accumulate=True)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(total, one + one)  # 0 + g is exact, g + g too
    streams = [torch.cuda.Stream() for _ in range(2)]
    sums = [torch.zeros_like(total) for _ in streams]
    outs = [c.out(K) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(2):
        for s, buf, o in zip(streams, sums, outs):
            moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, grad_rows=o, grad_w1=buf, accumulate=True, stream=s)
    torch.cuda.synchronize()
    for buf, o in zip(sums, outs):
        assert torch.equal(buf, total) and torch.equal(o[: c.n], gx[: c.n])
