"""moe_orthogonalize against the iteration in 64 bits.

Tolerance: the 2-norm of the error, relative.  The bf16 result is off by at most half a step, 2^-8, of each value
(1.7e-3 of the 2-norm: a rounding error is uniform over the step and values over the binade).  The fp16 operands of
sides above 64 add, in an emulation of every rounding in 64 bits over 200 matrices a size (sides 65 to 1024; Gaussian,
near-low-rank, singular values over four decades), at most 1.8e-3; together at most 2.5e-3.  Asserted: 2^-8.
Sides up to 64 run in 64 bits: only the rounding is left, and 2^-8 bounds it rigorously.
"""
import pytest

pytestmark = pytest.mark.gpu

NS = (3.4445, -4.7750, 2.0315)


def reference(g, steps=5, coefficients=NS, eps=1e-7):
    import torch

    a, b, c = coefficients
    x = g.double()
    x = x / (torch.linalg.matrix_norm(x).view(-1, 1, 1) + eps)
    tall = x.shape[1] > x.shape[2]
    x = x.mT if tall else x
    for _ in range(steps):
        m = x @ x.mT
        x = a * x + (b * m + c * m @ m) @ x
    return x.mT if tall else x


def matrices(E, M, N, kind, dtype, seed=0):
    import torch

    gen = torch.Generator(device="cuda").manual_seed(seed + M * 31 + N)
    g = torch.randn((E, M, N), generator=gen, device="cuda")
    s = min(M, N)
    if kind == "lowrank":
        r = max(1, s // 6)
        g = torch.randn((E, M, r), generator=gen, device="cuda") @ torch.randn((E, r, N), generator=gen, device="cuda") \
            + 0.05 * g
    if kind == "decades":
        u, _, v = torch.linalg.svd(g, full_matrices=False)
        g = u * torch.logspace(0, -4, s, device="cuda") @ v
    return (g * 1e-3).to(getattr(torch, dtype))


def check(got, ref):
    import torch

    assert got.dtype == torch.bfloat16 and got.shape == ref.shape
    assert bool(torch.isfinite(got).all())
    err = torch.linalg.matrix_norm(got.double() - ref) / torch.linalg.matrix_norm(ref)
    assert float(err.max()) <= 2.0 ** -8, err.tolist()


SIZES = [(1, 1, 1), (2, 1, 7), (3, 9, 1), (4, 3, 5), (2, 16, 40), (1, 64, 64), (3, 64, 2000), (2, 5000, 33),
         (1, 65, 65), (2, 66, 129), (3, 129, 66), (1, 256, 256), (2, 257, 1000), (1, 1000, 257), (5, 128, 384),
         (1, 511, 512), (2, 1024, 640)]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("kind", ["gauss", "lowrank", "decades"])
@pytest.mark.parametrize("E,M,N", SIZES)
def test_matches_the_iteration(E, M, N, kind, dtype):
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(E, M, N, kind, dtype)
    check(moe.moe_orthogonalize(g), reference(g))
    moe.moe_device_status()


def test_larger_matrices():
    import mixture_experts_ffn_planner_b200 as moe

    for E, M, N in ((2, 1024, 2048), (1, 2304, 1152), (40, 256, 512)):
        g = matrices(E, M, N, "lowrank", "bfloat16")
        check(moe.moe_orthogonalize(g), reference(g))


@pytest.mark.parametrize("E,M,N", [(1, 64, 65), (3, 33, 520), (1, 32, 513), (3, 17, 130), (2, 256, 61), (4, 64, 257), (2, 2, 640), (1, 5120, 64), (1, 4608, 31), (1, 64, 4609),
                                   (1, 64, 5121), (2, 63, 9000), (150, 40, 500)])
def test_short_sides(E, M, N):
    """Every way of a side of at most 64: one CTA a matrix, clusters of 2, 4 and 8, and a side too long for them."""
    import mixture_experts_ffn_planner_b200 as moe

    for kind in ("lowrank", "decades"):
        g = matrices(E, M, N, kind, "float32")
        check(moe.moe_orthogonalize(g), reference(g))
    moe.moe_device_status()


@pytest.mark.parametrize("E,M,N", [(1, 65, 512), (2, 512, 65), (5, 96, 97), (3, 127, 500), (1, 129, 129), (2, 255, 256),
                                   (2, 256, 449), (1, 511, 192), (4, 200, 320), (56, 128, 65), (57, 128, 65),
                                   (1, 256, 513), (1, 257, 512), (2, 128, 513), (1, 1024, 70), (2, 101, 1000), (1, 128, 1025),
                                   (14, 90, 700), (15, 90, 1024)])
def test_middle_sides(E, M, N):
    """One launch for shorter sides of 65 to 256 and few matrices, and the sizes next to where it begins and ends."""
    import mixture_experts_ffn_planner_b200 as moe

    for kind, dtype in (("lowrank", "bfloat16"), ("decades", "float32")):
        g = matrices(E, M, N, kind, dtype)
        check(moe.moe_orthogonalize(g), reference(g))
    moe.moe_device_status()


@pytest.mark.parametrize("E,M,N", [(80, 100, 300), (75, 300, 72), (20, 520, 700), (19, 777, 513)])
def test_many_matrices(E, M, N):
    """Enough tiles for every pair of SMs, with tails on both sides."""
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(E, M, N, "lowrank", "bfloat16")
    check(moe.moe_orthogonalize(g), reference(g))
    moe.moe_device_status()


@pytest.mark.parametrize("M,N", [(40, 96), (96, 40), (200, 136), (136, 200)])
def test_steps_coefficients_and_eps(M, N):
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(2, M, N, "gauss", "float32")
    for steps in (1, 2, 4, 7):
        check(moe.moe_orthogonalize(g, steps=steps), reference(g, steps))
    cubic = (1.5, -0.5, 0.0)
    check(moe.moe_orthogonalize(g, steps=6, coefficients=cubic), reference(g, 6, cubic))
    eps = 0.05
    check(moe.moe_orthogonalize(g, eps=eps), reference(g, eps=eps))


@pytest.mark.parametrize("M,N", [(8, 24), (100, 72), (72, 100)])
def test_zero_matrices_and_neighbours(M, N):
    """A zero matrix (an expert without tokens) gives zeros; one with a NaN harms no other of the batch."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    g = matrices(3, M, N, "gauss", "bfloat16")
    g[1] = 0
    out = moe.moe_orthogonalize(g)
    assert bool((out[1] == 0).all())
    check(out[::2], reference(g[::2]))
    g[1, 0, 0] = float("nan")
    out = moe.moe_orthogonalize(g)
    check(out[::2], reference(g[::2]))
    assert bool(torch.isnan(out[1]).any())


@pytest.mark.parametrize("M,N", [(48, 80), (80, 48), (200, 96), (96, 200), (131, 97)])
def test_in_place_unaligned_stream_and_graph(M, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    E = 2
    g = matrices(E, M, N, "lowrank", "bfloat16")
    want = moe.moe_orthogonalize(g)
    same = g.clone()
    assert moe.moe_orthogonalize(same, out=same) is same and torch.equal(same, want)
    odd_in = torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:].view(E, M, N).copy_(g)
    odd_out = torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:].view(E, M, N)
    assert torch.equal(moe.moe_orthogonalize(odd_in, out=odd_out), want)
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
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, moe.moe_orthogonalize(g))


def test_nothing_to_do():
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    for shape in ((0, 8, 8), (2, 0, 8), (2, 8, 0)):
        assert moe.moe_orthogonalize(torch.empty(shape, device="cuda")).shape == shape
