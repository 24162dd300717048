"""A training step of the expert FFN as its calls are used together: router and planner, rows by expert, the products,
the weighted sum back, every gradient, and the weights' update; against the layer's formula in 64 bits.

Tolerances, elementwise, from the operands' magnitudes.  A rounding to bf16 is off by at most H = 2^-8 of the value, a
sum of n products in fp32 by at most n * 2^-23 * sum |a b|; an operand that is off by e adds e times the others'
magnitudes (products of several: with every magnitude enlarged by its error).  silu and its derivative change by at
most 1.1 and 0.5 times their argument's error, and are computed to 2^-18.  bounds() carries these through the step.
"""
import pytest

pytestmark = pytest.mark.gpu

H = 2.0 ** -8
U = 2.0 ** -23
FAST = 2.0 ** -18


class Layer:
    def __init__(self, T, k, E, bm, K, N, seed):
        import torch
        import mixture_experts_ffn_planner_b200 as moe

        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, std=1.0: torch.randn(s, generator=g, device="cuda") * std  # noqa: E731
        self.T, self.k, self.E, self.bm, self.K, self.N, self.half = T, k, E, bm, K, N, N // 2
        self.x, self.go = r(T, K).bfloat16(), r(T, K).bfloat16()
        self.w1, self.w2 = r(E, N, K, std=K ** -0.5).bfloat16(), r(E, K, N // 2, std=(N // 2) ** -0.5).bfloat16()
        self.ids, self.tw, *self.plan = moe.moe_route_align(r(T, E), k, bm)
        self.slots = moe.moe_route_slots(self.plan[0], self.plan[2], T, k)

    def step(self, **kw):
        """The calls of one step; gradients by x, w1, w2 and the routing weights of <out, go>."""
        import mixture_experts_ffn_planner_b200 as moe

        s_ids, _, ntpp = self.plan
        rows = moe.moe_permute(self.x, s_ids, ntpp, self.slots, **kw)
        h, act = moe.moe_expert_up(rows, self.w1, *self.plan, self.bm, **kw)
        y = moe.moe_expert_down(act, self.w2, *self.plan, self.bm, **kw)
        out = moe.moe_unpermute(y, self.slots, self.tw, **kw)
        gy, gtw = moe.moe_unpermute_backward(self.go, y, s_ids, ntpp, self.slots, self.tw, **kw)
        gh, gw2 = moe.moe_expert_down_backward(gy, h, act, self.w2, *self.plan, self.bm, **kw)
        grows, gw1 = moe.moe_expert_up_backward(gh, rows, self.w1, *self.plan, self.bm, **kw)
        gx = moe.moe_permute_backward(grows, self.slots, **kw)
        up1, up2 = moe.moe_orthogonalize(gw1, **kw), moe.moe_orthogonalize(gw2, **kw)
        return dict(out=out, gx=gx, gw1=gw1, gw2=gw2, gtw=gtw), (up1, up2)

    def loss(self, x, w1, w2, tw):
        """<out, go> from the definition, route by route."""
        import torch

        out = torch.zeros((self.T, self.K), dtype=torch.float64, device="cuda")
        for e in range(self.E):
            t, j = torch.nonzero(self.ids == e, as_tuple=True)
            g, u = (x[t] @ w1[e].T).chunk(2, 1)
            out = out.index_add(0, t, tw[t, j].unsqueeze(1) * ((g * torch.sigmoid(g) * u) @ w2[e].T))
        return out, (out * self.go.double()).sum()

    def bounds(self):
        """What every result may be off by (see above)."""
        import torch

        z = lambda *s: torch.zeros(s, dtype=torch.float64, device="cuda")  # noqa: E731
        b = dict(out=z(self.T, self.K), gx=z(self.T, self.K), gw1=z(self.E, self.N, self.K),
                 gw2=z(self.E, self.K, self.half), gtw=z(self.T, self.k))
        mag = dict(out=z(self.T, self.K), gx=z(self.T, self.K))  # sums of the routes' magnitudes

        def product(*ab):  # |a' b' ...| - |a b ...| for |a' - a| <= e
            p, q = 1.0, 1.0
            for a, e in ab:
                p, q = p * (a + e), q * a
            return p - q

        def rounded(a, e):
            return e + H * (a + e)

        for e in range(self.E):
            t, j = torch.nonzero(self.ids == e, as_tuple=True)
            x, w1, w2, go = self.x[t].double(), self.w1[e].double(), self.w2[e].double(), self.go[t].double()
            w = self.tw[t, j].double().unsqueeze(1)
            h, eh = x @ w1.T, self.K * U * (x.abs() @ w1.abs().T)
            (g, u), (eg, eu) = h.chunk(2, 1), eh.chunk(2, 1)
            s = torch.sigmoid(g)
            silu, d = g * s, s * (1 + g * (1 - s))
            act = (silu * u).abs()
            ea = rounded(act, product((silu.abs(), 1.1 * eg + FAST * silu.abs()), (u.abs(), eu)) + FAST * act)
            y = ((silu * u) @ w2.T).abs()
            ey = ea @ w2.abs().T + self.half * U * ((act + ea) @ w2.abs().T)
            ey = rounded(y, ey)
            gy = (w * go).abs()
            egy = H * gy + U * gy
            ga = ((w * go) @ w2).abs()
            ega = egy @ w2.abs() + self.K * U * ((gy + egy) @ w2.abs())
            rg, ru = rounded(g.abs(), eg), rounded(u.abs(), eu)  # h as it is stored
            egg = product((ga, ega), (u.abs(), ru), (d.abs(), 0.5 * rg + FAST))
            egu = product((ga, ega), (silu.abs(), 1.1 * rg + FAST * silu.abs()))
            gh = torch.cat((ga * (u * d).abs(), ga * silu.abs()), 1)
            egh = rounded(gh, torch.cat((egg, egu), 1) + FAST * gh)
            gr = (torch.cat(((w * go) @ w2 * u * d, (w * go) @ w2 * silu), 1) @ w1).abs()
            egr = rounded(gr, egh @ w1.abs() + self.N * U * ((gh + egh) @ w1.abs()))
            n = max(len(t), 1)
            b["gw1"][e] = egh.T @ x.abs() + n * U * ((gh + egh).T @ x.abs())
            b["gw2"][e] = (gy + egy).T @ (act + ea) * (1 + n * U) - gy.T @ act
            b["out"].index_add_(0, t, w * ey)
            mag["out"].index_add_(0, t, w * (y + ey))
            b["gx"].index_add_(0, t, egr)
            mag["gx"].index_add_(0, t, gr + egr)
            b["gtw"][t, j] = (go.abs() * ey).sum(1) + self.K * U * (go.abs() * (y + ey)).sum(1)
        for n in mag:
            b[n] += (self.k + 1) * U * mag[n]
        return b


CASES = [
    # T, k, E, bm, K, N
    (1, 2, 4, 16, 64, 64),
    (33, 3, 9, 16, 136, 80),
    (300, 4, 16, 64, 256, 320),
    (700, 2, 3, 128, 384, 208),
    (1500, 8, 24, 32, 272, 560),
]


@pytest.mark.parametrize("T,k,E,bm,K,N", CASES)
def test_step_against_the_formula_and_differences(T, k, E, bm, K, N):
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Layer(T, k, E, bm, K, N, seed=T + E)
    got, _ = c.step()
    moe.moe_device_status()
    leaves = [v.double().requires_grad_(True) for v in (c.x, c.w1, c.w2, c.tw)]
    out, loss = c.loss(*leaves)
    ref = dict(zip(("gx", "gw1", "gw2", "gtw"), torch.autograd.grad(loss, leaves)), out=out.detach())
    bound = c.bounds()
    for name, r in ref.items():
        half = 0.0 if name == "gtw" else H  # the result's own rounding
        err = (got[name].double() - r).abs()
        over = err - bound[name] - half * (r.abs() + bound[name]) - 1e-30
        assert float(over.max()) <= 0, f"{name}: {float(over.max()):.3e} over its bound"
    # against differences: along one direction, in 64 bits, a central difference is off by the third derivative's
    # share, (1e-4)^2, and by the cancellation, 2^-52 |loss| / 1e-4
    gen = torch.Generator(device="cuda").manual_seed(5)
    step = 1e-4
    direction = [torch.randn(v.shape, generator=gen, device="cuda", dtype=torch.float64) for v in leaves]
    with torch.no_grad():
        scale = [1.0, K ** -0.5, (N // 2) ** -0.5, 1.0]
        moved = [c.loss(*[v + sign * step * s * d for v, s, d in zip(leaves, scale, direction)])[1] for sign in (1, -1)]
        difference = float(moved[0] - moved[1]) / (2 * step)
        along, slack, total = 0.0, 0.0, 0.0
        for name, s, d in zip(("gx", "gw1", "gw2", "gtw"), scale, direction):
            half = 0.0 if name == "gtw" else H
            along += float((got[name].double() * s * d).sum())
            slack += float(((bound[name] + half * (ref[name].abs() + bound[name])) * (s * d).abs()).sum())
            total += float((ref[name] * s * d).abs().sum())
    assert abs(along - difference) <= slack + 1e-4 * total


def test_step_captured_on_another_stream_and_repeated():
    """Eagerly, on a side stream, and captured and replayed on new inputs: the same bits."""
    import torch

    c = Layer(200, 4, 12, 32, 264, 208, seed=3)

    def flat(result):
        d, ups = result
        return [d[n] for n in ("out", "gx", "gw1", "gw2", "gtw")] + list(ups)

    first = flat(c.step())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = flat(c.step(stream=side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = flat(c.step())
    keep = c.x.clone()
    c.x.copy_(torch.randn_like(c.x))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, flat(c.step())))
    c.x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(captured, first))


def test_forward_agrees_with_the_fused_call():
    """The unfused forward and fused_moe_bf16 on the same plan: both within their roundings of the formula, so of
    each other within the two bounds' sum (the fused call rounds act to bf16 and sums in fp32, as this one does, but
    keeps y in fp32)."""
    import torch
    import mixture_experts_ffn_planner_b200 as moe

    c = Layer(256, 4, 8, 64, 256, 512, seed=9)
    got = c.step()[0]["out"]
    fused = torch.empty_like(got)
    moe.fused_moe_bf16(c.x, c.w1, c.w2, *c.plan, c.tw, fused, c.bm)
    ref = c.loss(c.x.double(), c.w1.double(), c.w2.double(), c.tw.double())[0]
    b = c.bounds()["out"]
    assert bool(((got.double() - fused.double()).abs() <= 2 * (b + H * (ref.abs() + b))).all())


def test_two_steps_at_once():
    """Two layers' steps on two streams, neither waiting for the other."""
    import torch

    layers = [Layer(400, 4, 16, 64, 256, 256, seed=1), Layer(250, 2, 5, 128, 520, 144, seed=2)]
    alone = [c.step() for c in layers]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        both = [c.step(stream=s) for c, s in zip(layers, streams)]
        torch.cuda.synchronize()
        for (a, ups_a), (b, ups_b) in zip(alone, both):
            assert all(torch.equal(a[n], b[n]) for n in a) and all(torch.equal(p, q) for p, q in zip(ups_a, ups_b))
