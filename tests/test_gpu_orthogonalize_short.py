"""moe_orthogonalize with a side of at most 64, value by value against the iteration in 64 bits.

Tolerances.  The result is rounded to bf16: half a step, 2^-8 of the value.
A longer side up to 5120 is iterated in fp32.  An emulation of that on the CPU (sums in fp32, in two orders; 20 to 200
matrices of each of 11 sizes from 1 x 7 to 64 x 200 and each kind below) was at most 2.0e-4 of the largest value off, on
matrices of rank one and noise, whose weak directions the steps raise together with the rounding of the strong one.
Asserted: 2^-11 (4.9e-4) of the largest value beside the rounding.
A longer side above 5120 is iterated in 64 bits on S x S matrices and stored by way of fp32: 2^-24 of the value, and the
squared condition of at most 10^10 leaves 10^-6 of the largest: 2^-20 of it is asserted."""
import pytest

from test_gpu_orthogonalize import matrices, reference

pytestmark = pytest.mark.gpu

FP32 = [(1, 1, 7), (2, 3, 5), (3, 9, 1), (2, 16, 40), (1, 64, 64), (3, 64, 2000), (2, 5000, 33), (1, 5120, 64), (1, 64, 5120),
        (2, 1, 5120)]
FP64 = [(2, 9000, 63), (1, 5121, 1), (1, 1, 5121), (3, 64, 5121), (2, 5200, 64), (1, 6000, 17), (1, 20011, 64)]


def _matrices(E, M, N, kind, dtype):
    import torch

    if kind != "rank1":
        return matrices(E, M, N, kind, dtype)
    gen = torch.Generator(device="cuda").manual_seed(M * 31 + N)
    g = torch.randn((E, M, 1), generator=gen, device="cuda") @ torch.randn((E, 1, N), generator=gen, device="cuda")
    return ((g + 1e-4 * torch.randn((E, M, N), generator=gen, device="cuda")) * 1e-3).to(getattr(torch, dtype))


def _check(got, ref, part):
    import torch

    assert got.dtype == torch.bfloat16 and bool(torch.isfinite(got).all())
    top = ref.abs().amax((1, 2), keepdim=True)
    over = (got.double() - ref).abs() - 2.0 ** -8 * ref.abs() - part * top
    assert float(over.max()) <= 0, f"worst {float((over / top).max()):.3e} of the largest value over its bound"


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", ["gauss", "lowrank", "decades", "rank1"])
@pytest.mark.parametrize("E,M,N", FP32 + FP64)
def test_values(E, M, N, kind, dtype):
    import mixture_experts_ffn_planner_b200 as moe

    g = _matrices(E, M, N, kind, dtype)
    _check(moe.moe_orthogonalize(g), reference(g), 2.0 ** (-11 if max(M, N) <= 5120 else -20))
    moe.moe_device_status()


@pytest.mark.parametrize("M,N", [(9000, 40), (40, 9000), (5125, 64), (7, 5123), (3000, 21), (64, 5120)])
def test_in_place_unaligned_stream_and_graph(M, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    E = 2
    g = matrices(E, M, N, "lowrank", "bfloat16")
    want = moe.moe_orthogonalize(g)
    assert torch.equal(moe.moe_orthogonalize(g), want)
    same = g.clone()
    assert moe.moe_orthogonalize(same, out=same) is same and torch.equal(same, want)
    odd_in = torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:].view(E, M, N).copy_(g)
    guarded = torch.full((g.numel() + 130,), 3.0, dtype=g.dtype, device="cuda")
    odd_out = guarded[65:65 + g.numel()].view(E, M, N)
    assert torch.equal(moe.moe_orthogonalize(odd_in, out=odd_out), want)
    assert bool((guarded[:65] == 3).all()) and bool((guarded[65 + g.numel():] == 3).all())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = moe.moe_orthogonalize(g, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    ws = torch.full((moe.moe_orthogonalize_workspace_bytes(E, M, N),), 0xFF, dtype=torch.uint8, device="cuda")  # NaNs
    assert torch.equal(moe.moe_orthogonalize(g, workspace=ws), want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        moe.moe_orthogonalize(g, out=out)
    g.copy_(matrices(E, M, N, "gauss", "bfloat16", seed=4))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, moe.moe_orthogonalize(g))


@pytest.mark.parametrize("M,N", [(9000, 40), (6, 5500)])
def test_zero_matrices_and_neighbours(M, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(3, M, N, "gauss", "bfloat16")
    g[1] = 0
    out = moe.moe_orthogonalize(g)
    assert bool((out[1] == 0).all())
    _check(out[::2], reference(g[::2]), 2.0 ** -20)
    g[1, 0, 0] = float("nan")
    out = moe.moe_orthogonalize(g)
    _check(out[::2], reference(g[::2]), 2.0 ** -20)
    assert bool(torch.isnan(out[1]).any())
