"""moe_orthogonalize next to the longest side that it takes, 2^31 - 2048: its kernels walk the longer side in steps of up
to 2048 places with 32-bit indices.  Longer ones are refused before any launch, and workspaces are never negative (CPU);
the longest comes out right (GPU)."""
import pytest

import mixture_experts_ffn_planner_b200 as moe

UNSUPPORTED, WORKSPACE = -2, -4
P = 1 << 20
LONGEST = 2 ** 31 - 2048


@pytest.fixture(scope="module")
def lib():
    return moe.load()


@pytest.mark.parametrize("length", [LONGEST + 1, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 1])
@pytest.mark.parametrize("side", [1, 64, 65])
@pytest.mark.parametrize("tall", [False, True])
def test_too_long(lib, length, side, tall):
    M, N = (length, side) if tall else (side, length)
    assert lib.moe_orthogonalize_workspace_bytes(1, M, N) == -1
    # null pointers: refused for its size before anything is looked at
    assert lib.moe_orthogonalize(None, 0, 1, M, N, 5, 3.4, -4.7, 2.0, 1e-7, None, None, 0, None) == UNSUPPORTED
    assert b"2^31 - 2048" in lib.moe_last_error()


@pytest.mark.parametrize("side", [1, 64, 65])
@pytest.mark.parametrize("tall", [False, True])
def test_longest(lib, side, tall):
    M, N = (LONGEST, side) if tall else (side, LONGEST)
    n = lib.moe_orthogonalize_workspace_bytes(1, M, N)
    if side <= 64:
        assert n == (1 + 32) * 64 * 64 * 8  # Q and at most 32 shares of G G^T, in 64 bits
    else:
        assert n >= 4 * 2 * side * LONGEST  # two iterates, each two halves of 16 bits
    assert lib.moe_orthogonalize(P, 0, 1, M, N, 5, 3.4, -4.7, 2.0, 1e-7, P, P, n - 1, None) == WORKSPACE


@pytest.mark.gpu
@pytest.mark.parametrize("tall", [False, True])
def test_longest_row(tall):
    """One row: X stays a multiple of G, so each value is G's times p^steps(1) / |G|, in 64 bits but for the result's own
    rounding, half a step of bf16 (2^-8), and the way by fp32 (2^-24)."""
    import torch

    g = torch.empty((1, LONGEST, 1) if tall else (1, 1, LONGEST), dtype=torch.bfloat16, device="cuda")
    g.random_(-120, 120, generator=torch.Generator(device="cuda").manual_seed(2))
    out = moe.moe_orthogonalize(g)
    moe.moe_device_status()
    flat, got = g.view(-1), out.view(-1)
    parts = range(0, LONGEST, 1 << 27)
    norm = sum(float((flat[i:i + (1 << 27)].double() ** 2).sum()) for i in parts) ** 0.5
    x = 1.0
    for _ in range(5):
        x = 3.4445 * x - 4.7750 * x ** 3 + 2.0315 * x ** 5
    for i in parts:
        ref = flat[i:i + (1 << 27)].double() * (x / norm)
        assert bool(((got[i:i + (1 << 27)].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -22) * ref.abs()).all())
    del out, got
    torch.cuda.empty_cache()
