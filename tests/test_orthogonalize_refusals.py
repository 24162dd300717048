"""What moe_orthogonalize refuses, before any launch (CPU)."""
import pytest
import torch

import mixture_experts_ffn_planner_b200 as moe

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, -1, -2, -3, -4
P = 1 << 20


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def call(lib, g=P, dt=0, E=2, M=128, N=96, steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7, out=P, ws=P, n=1 << 30):
    return lib.moe_orthogonalize(g, dt, E, M, N, steps, a, b, c, eps, out, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(E=-1), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(steps=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(dt=2), UNSUPPORTED), (dict(a=65.0), UNSUPPORTED),
    (dict(b=float("nan")), UNSUPPORTED), (dict(c=float("-inf")), UNSUPPORTED), (dict(E=65536), UNSUPPORTED),
    (dict(E=60000, M=100000, N=100000), UNSUPPORTED), (dict(g=None), INVALID), (dict(out=None), INVALID),
    (dict(ws=None), INVALID), (dict(g=P + 1), ALIGNMENT), (dict(g=P + 2, dt=1), ALIGNMENT), (dict(out=P + 1), ALIGNMENT),
    (dict(ws=P + 128), ALIGNMENT), (dict(n=1000), WORKSPACE), (dict(M=8, n=1000), WORKSPACE),
    (dict(E=0, g=None), OK), (dict(M=0, g=None, out=None, ws=None), OK),
])
def test_status(lib, kw, code):
    assert call(lib, **kw) == code


def test_workspace_sizes(lib):
    assert lib.moe_orthogonalize_workspace_bytes(0, 8, 8) == -1
    assert lib.moe_orthogonalize_workspace_bytes(2, 0, 8) == -1
    small, large = lib.moe_orthogonalize_workspace_bytes(3, 64, 512), lib.moe_orthogonalize_workspace_bytes(3, 65, 512)
    assert small >= 3 * 64 * 64 * 4 and large >= 3 * 65 * 512 * 8
    with pytest.raises(moe.MoeError):
        moe.moe_orthogonalize_workspace_bytes(0, 8, 8)


def test_binding_refuses():
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        moe.moe_orthogonalize(torch.zeros(2, 8, 8))
    with pytest.raises(ValueError, match="dimensions"):
        moe.moe_orthogonalize(torch.zeros(8, 8))
    with pytest.raises(TypeError, match="g: dtype"):
        moe.moe_orthogonalize(torch.zeros(2, 8, 8, dtype=torch.float64))
    with pytest.raises(ValueError, match="g is required"):
        moe.moe_orthogonalize(None)
