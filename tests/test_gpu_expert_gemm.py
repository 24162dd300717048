"""The experts' products (moe_expert_up, moe_expert_down) and their gradients against the formulas in 64 bits.

Tolerances.  Products of bf16 values are exact in fp32.  A sum of n of them in fp32 is off by at most n * 2^-23 *
sum |a b| whatever its order and whether each addition rounds or truncates (S below), and is then rounded once: half
a step of the output type, relative.  On top of that:
  act    silu(g) u: |silu'| <= 1.1, so 1.1 |u| S(g) + |silu(g)| S(u), + S(g) S(u); the fast exponential and
         division: 2^-18 relative.
  grad_h 1.1 |u| S(ga) and |silu(g)| S(ga); the factors s (1 + g (1 - s)) and g s are sums of terms below 1.3 and |g|
         computed with relative errors below 2^-18.
The elementwise bound of a long sum is loose, so the whole is held to rounding too: the 2-norm of the error is at most
half a step of the 2-norm of the result, + 2^-14 of it for the sums (fp32 rounding accumulates far below that).
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

SENTINEL = 5.0
U = 2.0 ** -23
FAST = 2.0 ** -18


def _plan(T, k, E, bm, seed, drop, skip):
    """A plan with dropped routes and, with skip, experts that no token routes to."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    rng = np.random.default_rng(seed)
    pool = np.arange(E) if not skip else np.array([e for e in range(E) if e % 3 != 1])
    ids = np.stack([rng.permutation(pool)[:k] for _ in range(T)]).astype(np.int32) if T else np.zeros((0, k), np.int32)
    ids[rng.random((T, k)) < drop] = -1
    s_ids, e_ids, ntpp = moe.moe_align(torch.from_numpy(ids).cuda(), E, bm)
    return s_ids, e_ids, ntpp


class Case:
    def __init__(self, T, k, E, bm, K, N, drop=0.1, skip=True, seed=0):
        import torch

        self.E, self.bm, self.K, self.N, self.half = E, bm, K, N, N // 2
        self.plan = s_ids, e_ids, ntpp = _plan(T, k, E, bm, seed, drop, skip)
        self.cap, self.n = s_ids.numel(), int(ntpp)
        self.routed = s_ids >= 0
        self.expert = e_ids.long().repeat_interleave(bm)[: self.cap]
        self.g = torch.Generator(device="cuda").manual_seed(seed + 1)

    def rows(self, width, std=1.0):
        """Rows whose padding holds NaN: what is there must not matter."""
        import torch

        v = (torch.randn((self.cap, width), generator=self.g, device="cuda") * std).bfloat16()
        v[~self.routed] = float("nan")
        return v

    def weights(self, *shape):
        import torch

        return (torch.randn(shape, generator=self.g, device="cuda") * shape[-1] ** -0.5).bfloat16()

    def out(self, width):
        import torch

        return torch.full((self.cap, width), SENTINEL, dtype=torch.bfloat16, device="cuda")

    def by_expert(self):
        import torch

        for e in range(self.E):
            yield e, torch.nonzero(self.routed & (self.expert == e)).squeeze(1)

    def check_rows(self, got, ref, slack):
        """ref, slack (cap, width): values at routed rows."""
        import torch

        assert bool((got[self.n:] == SENTINEL).all()), "rows past the padded total were written"
        pad = ~self.routed
        pad[self.n:] = False
        assert bool((got[pad] == 0).all()), "padding rows are not zero"
        check(got[self.routed], ref[self.routed], slack[self.routed])


def check(got, ref, slack):
    import torch

    assert bool(torch.isfinite(got).all())
    half = torch.finfo(got.dtype).eps / 2
    err = (got.double() - ref).abs()
    over = err - half * ref.abs() - slack
    assert got.numel() == 0 or float(over.max()) <= 0, f"worst {float(over.max()):.3e} over its bound"
    norm = float(ref.norm())
    assert float((got.double() - ref).norm()) <= (half + 2.0 ** -14) * norm + 1e-30


SHAPES = [
    # T, k, E, bm, K, N
    (1, 1, 1, 16, 8, 16),              # one token, the smallest sizes
    (1, 2, 4, 128, 64, 32),
    (5, 2, 8, 16, 128, 128),
    (64, 2, 8, 64, 1024, 1024),
    (100, 3, 7, 32, 200, 272),         # tails in every direction
    (300, 4, 10, 64, 392, 336),
    (257, 2, 3, 128, 512, 624),        # several blocks an expert
    (1000, 8, 24, 128, 264, 1040),
    (77, 1, 200, 16, 136, 48),         # most experts empty
    (2000, 2, 2, 16, 72, 80),          # very many small blocks
    (3000, 4, 24, 16, 520, 1040),      # tiles enough for every pair of SMs, tails in every direction
    (2100, 3, 20, 128, 456, 528),
]


@pytest.mark.parametrize("T,k,E,bm,K,N", SHAPES)
def test_forward(T, k, E, bm, K, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Case(T, k, E, bm, K, N, drop=0.1 if T > 1 else 0.0, skip=E > 4, seed=T + K)
    rows, w1, w2 = c.rows(K), c.weights(E, N, K), c.weights(E, K, N // 2)
    h, act = c.out(N), c.out(c.half)
    got = moe.moe_expert_up(rows, w1, *c.plan, bm, h=h, act=act)
    assert got[0] is h and got[1] is act
    a_in = c.rows(c.half)
    y = moe.moe_expert_down(a_in, w2, *c.plan, bm, out=c.out(K))
    moe.moe_device_status()
    z = lambda w: torch.zeros((c.cap, w), dtype=torch.float64, device="cuda")  # noqa: E731
    rh, sh, ra, sa, ry, sy = z(N), z(N), z(c.half), z(c.half), z(K), z(K)
    for e, p in c.by_expert():
        x, w = rows[p].double(), w1[e].double()
        rh[p] = x @ w.T
        sh[p] = K * U * (x.abs() @ w.abs().T)
        g, u = rh[p].chunk(2, 1)
        sg, su = sh[p].chunk(2, 1)
        silu = g * torch.sigmoid(g)
        ra[p] = silu * u
        sa[p] = 1.1 * u.abs() * sg + silu.abs() * su + sg * su + FAST * (silu * u).abs()
        x, w = a_in[p].double(), w2[e].double()
        ry[p] = x @ w.T
        sy[p] = c.half * U * (x.abs() @ w.abs().T)
    c.check_rows(h, rh, sh)
    c.check_rows(act, ra, sa)
    c.check_rows(y, ry, sy)


@pytest.mark.parametrize("T,k,E,bm,K,N", SHAPES)
def test_backward(T, k, E, bm, K, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Case(T, k, E, bm, K, N, drop=0.1 if T > 1 else 0.0, skip=E > 4, seed=T + N)
    rows, w1, w2 = c.rows(K), c.weights(E, N, K), c.weights(E, K, N // 2)
    gy, h, act, gh_in = c.rows(K), c.rows(N), c.rows(c.half, 0.6), c.rows(N)
    gh, gw2 = moe.moe_expert_down_backward(gy, h, act, w2, *c.plan, bm, grad_h=c.out(N))
    gx, gw1 = moe.moe_expert_up_backward(gh_in, rows, w1, *c.plan, bm, grad_rows=c.out(K))
    moe.moe_device_status()
    d = torch.float64
    z = lambda *s: torch.zeros(s, dtype=d, device="cuda")  # noqa: E731
    rh, sh, rx, sx = z(c.cap, N), z(c.cap, N), z(c.cap, K), z(c.cap, K)
    r1, s1, r2, s2 = z(E, N, K), z(E, N, K), z(E, K, c.half), z(E, K, c.half)
    for e, p in c.by_expert():
        y, w, a = gy[p].double(), w2[e].double(), act[p].double()
        ga, sga = y @ w, K * U * (y.abs() @ w.abs())
        g, u = h[p].double().chunk(2, 1)
        s = torch.sigmoid(g)
        rh[p] = torch.cat((ga * u * s * (1 + g * (1 - s)), ga * g * s), 1)
        sh[p] = torch.cat((1.1 * u.abs() * sga + FAST * 2.6 * (ga * u).abs(),
                           (g * s).abs() * sga + FAST * (ga * g * s).abs()), 1)
        r2[e], s2[e] = y.T @ a, len(p) * U * (y.abs().T @ a.abs())
        q, w, x = gh_in[p].double(), w1[e].double(), rows[p].double()
        rx[p], sx[p] = q @ w, N * U * (q.abs() @ w.abs())
        r1[e], s1[e] = q.T @ x, len(p) * U * (q.abs().T @ x.abs())
    c.check_rows(gh, rh, sh)
    c.check_rows(gx, rx, sx)
    check(gw2, r2, s2)
    check(gw1, r1, s1)


@pytest.mark.parametrize("T,E,bm", [(200, 5, 64), (3, 6, 16), (0, 3, 32)])
def test_fp32_weight_gradients_accumulate(T, E, bm):
    """fp32 buffers: written in full (empty experts: zeros), or added to: one fp32 rounding of the sum more."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    K, N = 136, 112
    c = Case(T, 2, E, bm, K, N, drop=0.0, skip=True, seed=11)
    rows, w1, w2 = c.rows(K), c.weights(E, N, K), c.weights(E, K, N // 2)
    gy, h, act, gh = c.rows(K), c.rows(N), c.rows(c.half), c.rows(N)
    f = lambda *s: torch.full(s, 3.0, device="cuda")  # noqa: E731
    new = (moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, grad_w1=f(E, N, K))[1],
           moe.moe_expert_down_backward(gy, h, act, w2, *c.plan, bm, grad_w2=f(E, K, N // 2))[1])
    add = (moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm, grad_w1=f(E, N, K), accumulate=True)[1],
           moe.moe_expert_down_backward(gy, h, act, w2, *c.plan, bm, grad_w2=f(E, K, N // 2), accumulate=True)[1])
    moe.moe_device_status()
    ref = [torch.zeros((E, N, K), dtype=torch.float64, device="cuda"),
           torch.zeros((E, K, N // 2), dtype=torch.float64, device="cuda")]
    mag = [r.clone() for r in ref]
    for e, p in c.by_expert():
        for i, (a, b) in enumerate(((gh, rows), (gy, act))):
            ref[i][e] = a[p].double().T @ b[p].double()
            mag[i][e] = len(p) * U * (a[p].double().abs().T @ b[p].double().abs())
        if len(p) == 0:
            assert bool((new[0][e] == 0).all()) and bool((new[1][e] == 0).all())
            assert bool((add[0][e] == 3).all()) and bool((add[1][e] == 3).all())
    for i in range(2):
        assert bool(((new[i].double() - ref[i]).abs() <= mag[i] + U * ref[i].abs()).all())
        assert bool(((add[i].double() - 3 - ref[i]).abs() <= mag[i] + U * (ref[i].abs() + 3)).all())


def test_no_tokens():
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Case(0, 2, 4, 64, 64, 64)
    w1, w2 = c.weights(4, 64, 64), c.weights(4, 64, 32)
    h, act = moe.moe_expert_up(c.rows(64), w1, *c.plan, 64, h=c.out(64), act=c.out(32))
    assert bool((h == SENTINEL).all()) and bool((act == SENTINEL).all())
    gx, gw = moe.moe_expert_up_backward(c.rows(64), c.rows(64), w1, *c.plan, 64, grad_rows=c.out(64))
    assert bool((gx == SENTINEL).all()) and bool((gw == 0).all())
    # a plan without any capacity
    s = torch.empty(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    e = lambda w: torch.empty((0, w), dtype=torch.bfloat16, device="cuda")  # noqa: E731
    gx, gw = moe.moe_expert_up_backward(e(64), e(64), w1, s, s, zero, 64)
    assert gx.shape == (0, 64) and bool((gw == 0).all())
    assert moe.moe_expert_down(e(32), w2, s, s, zero, 64).shape == (0, 64)
    moe.moe_device_status()


def test_repeat_is_bitwise_and_streams_and_graphs():
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Case(500, 4, 12, 64, 256, 320, seed=2)
    rows, w1, w2 = c.rows(256), c.weights(12, 320, 256), c.weights(12, 256, 160)

    def step(**kw):
        h, act = moe.moe_expert_up(rows, w1, *c.plan, 64, **kw)
        y = moe.moe_expert_down(act, w2, *c.plan, 64, **kw)
        gh, gw2 = moe.moe_expert_down_backward(y, h, act, w2, *c.plan, 64, **kw)
        gx, gw1 = moe.moe_expert_up_backward(gh, rows, w1, *c.plan, 64, **kw)
        return [t[: c.n] for t in (h, act, y, gh, gx)] + [gw1, gw2]

    first = step()
    assert all(torch.equal(a, b) for a, b in zip(first, step()))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    keep = rows.clone()
    rows.copy_(torch.where(c.routed.unsqueeze(1), torch.randn_like(rows), rows))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    rows.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, first))


def test_padding_is_cleared_every_time():
    """Weight gradients of many experts with ragged ends, NaN in all padding: finite and the same bits, run after run."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    for T, E, bm, K, N in ((9000, 32, 128, 512, 512), (5000, 100, 16, 264, 144)):  # pairs of CTAs, and single ones
        c = Case(T, 4, E, bm, K, N, drop=0.05, skip=True, seed=7)
        gh, rows, w1 = c.rows(N), c.rows(K), c.weights(E, N, K)
        first = moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm)
        assert bool(torch.isfinite(first[1]).all()) and bool(torch.isfinite(first[0][: c.n]).all())
        for _ in range(40):
            again = moe.moe_expert_up_backward(gh, rows, w1, *c.plan, bm)
            assert torch.equal(again[1], first[1]) and torch.equal(again[0][: c.n], first[0][: c.n])
    moe.moe_device_status()
