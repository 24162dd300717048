"""moe_orthogonalize where 1 / (|g| + eps) lies beyond fp32: zero matrices under a tiny eps give zeros, and matrices of
tiny norm (subnormal entries) the iteration's result.  Sizes of every way: short sides in shared memory, short sides on
S x S matrices, middle sides in one launch, launches on single CTAs and on pairs.

Tolerance as in test_gpu_orthogonalize.py: 2^-8 of the 2-norm, for the bf16 result and the fp16 operands.  The entries
are exact in the reference, and a product with a power of two is exact, so a tiny norm adds one fp32 rounding (2^-24)."""
import pytest

from test_gpu_orthogonalize import check, reference

pytestmark = pytest.mark.gpu

SIZES = [(2, 8, 24), (1, 60, 5200), (2, 100, 72), (1, 256, 200), (2, 300, 520), (30, 300, 320)]


@pytest.mark.parametrize("eps", [1e-36, 1e-38, 1e-45])
@pytest.mark.parametrize("E,M,N", SIZES)
def test_zero_matrices(E, M, N, eps):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    assert bool((moe.moe_orthogonalize(torch.zeros((E, M, N), device="cuda"), eps=eps) == 0).all())
    assert bool((moe.moe_orthogonalize(torch.zeros((E, M, N), device="cuda").bfloat16(), eps=eps) == 0).all())


@pytest.mark.parametrize("scale", [2.0 ** -110, 2.0 ** -126, 2.0 ** -136])
@pytest.mark.parametrize("E,M,N", SIZES)
def test_tiny_matrices(E, M, N, scale):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    gen = torch.Generator().manual_seed(M)
    # whole numbers up to 64 times a power of two: exact in fp32, subnormal at the smallest scales
    whole = torch.randint(-64, 65, (E, M, N), generator=gen).double()
    g = (whole * scale).float().cuda()
    assert torch.equal(g.double().cpu(), whole * scale)
    check(moe.moe_orthogonalize(g, eps=0.0), reference(g, eps=0.0))
    moe.moe_device_status()
