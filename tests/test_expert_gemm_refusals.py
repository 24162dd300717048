"""What the experts' products refuse, before any launch (CPU): the C ABI by status, the binding by exception."""
import pytest
import torch

import mixture_experts_ffn_planner_b200 as moe

INVALID, UNSUPPORTED, ALIGNMENT = -1, -2, -3
P = 1 << 20  # a well-aligned stand-in for a device pointer: these calls return before it is used


@pytest.fixture(scope="module")
def lib():
    return moe.load()


def up(lib, rows=P, w=P, ids=P, experts=P, total=P, cap=512, K=64, N=64, E=4, bm=64, h=P, act=P):
    return lib.moe_expert_up(rows, w, ids, experts, total, cap, K, N, E, bm, h, act, None)


def up_backward(lib, gh=P, rows=P, w=P, cap=512, K=64, N=64, E=4, bm=64, gx=P, gw=P, dt=0, acc=0):
    return lib.moe_expert_up_backward(gh, rows, w, P, P, P, cap, K, N, E, bm, gx, gw, dt, acc, None)


def down_backward(lib, gy=P, h=P, act=P, w=P, cap=512, K=64, N=64, E=4, bm=64, gh=P, gw=P, dt=0, acc=0):
    return lib.moe_expert_down_backward(gy, h, act, w, P, P, P, cap, K, N, E, bm, gh, gw, dt, acc, None)


@pytest.mark.parametrize("call", [up, up_backward, down_backward])
@pytest.mark.parametrize("kw,code", [
    (dict(K=0), INVALID), (dict(N=-16), INVALID), (dict(E=0), INVALID), (dict(cap=-1), INVALID),
    (dict(bm=48), UNSUPPORTED), (dict(bm=256), UNSUPPORTED), (dict(K=60), UNSUPPORTED), (dict(N=72), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED), (dict(cap=1 << 31), UNSUPPORTED), (dict(cap=(1 << 31) - 1, N=1 << 20, bm=16), UNSUPPORTED),
    (dict(w=None), INVALID), (dict(rows=None), INVALID), (dict(h=None), INVALID), (dict(gw=None), INVALID),
    (dict(gx=None), INVALID), (dict(w=P + 2), ALIGNMENT), (dict(rows=P + 8), ALIGNMENT), (dict(act=P + 4), ALIGNMENT),
    (dict(dt=2), UNSUPPORTED), (dict(acc=1), UNSUPPORTED),
])
def test_rejects(lib, call, kw, code):
    takes = call.__code__.co_varnames[1:call.__code__.co_argcount]
    if all(k in takes for k in kw):
        assert call(lib, **kw) == code
        assert lib.moe_last_error().startswith(b"moe_expert_")


def test_down_rejects(lib):
    f = lambda act=P, w=P, cap=512, K=64, N=64, E=4, bm=64, y=P: lib.moe_expert_down(  # noqa: E731
        act, w, P, P, P, cap, K, N, E, bm, y, None)
    assert f(K=12) == UNSUPPORTED and f(bm=8) == UNSUPPORTED and f(act=None) == INVALID and f(y=P + 8) == ALIGNMENT
    assert up(lib, ids=None) == INVALID and up(lib, experts=None) == INVALID and up(lib, total=None) == INVALID
    assert up(lib, ids=P + 2) == ALIGNMENT


def test_binding_refuses():
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    plan = (i32(128), i32(2), i32(1), 64)
    with pytest.raises(ValueError, match="w1 must be a CUDA tensor"):
        moe.moe_expert_up(bf(128, 64), bf(2, 64, 64), *plan)
    with pytest.raises(TypeError, match="w2: dtype"):
        moe.moe_expert_down(bf(128, 32), torch.zeros(2, 64, 32), *plan)
    with pytest.raises(ValueError, match="three dimensions"):
        moe.moe_expert_down(bf(128, 32), bf(64, 32), *plan)
    with pytest.raises(ValueError, match="w1 is required"):
        moe.moe_expert_up_backward(bf(128, 64), bf(128, 64), None, *plan)
