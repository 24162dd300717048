"""moe_orthogonalize next to the longest side that it takes, 2^31 - 2048: its kernels walk the longer side in steps of up
to 2048 places with 32-bit indices.  Longer ones are refused before any launch, and workspaces are never negative (CPU)."""
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
