"""The operators of training a mixture-of-experts feed-forward layer, as cases that can be timed and compared.

Three families, in the order a training step meets them:

* rows by expert: ``permute`` copies every token's row to the places its routes have in the planner's order,
  ``unpermute`` brings the experts' rows back as the weighted sum over a token's routes; each with its gradient.
* the experts' products on those rows: ``up`` (gate/up product with SwiGLU, keeping what the gradient needs) and
  ``down``; each with its gradients by rows and by weights.
* ``orthogonalize``: an expert's update made orthogonal by five Newton-Schulz steps.

``run`` takes a state of ``prepare`` through one operator: with ``own`` through the framework's kernels, otherwise
through elementary torch operations in fp32, rounded once.  ``exact`` gives the same outputs in 64 bits.

All row buffers have the planner's capacity.  Rows of a segment's padding come out as zeros; rows past the padded
total are left as they were, which the buffers of ``prepare`` make zeros.
"""
import math

import torch

own = False

NS = (3.4445, -4.7750, 2.0315)   # Newton-Schulz coefficients a, b, c of X <- a X + (b A + c A^2) X, A = X X^T
NS_EPS = 1e-7
ROW_OPS = ("permute", "permute_backward", "unpermute", "unpermute_backward")
EXPERT_OPS = ("up", "up_backward", "down", "down_backward")
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of tokens, as a latency-bound call meets them: 64 rows of 8 KB
        dict(name="permute T8", op="permute", T=8, K=4096, E=128, top_k=8, block_m=16, zipf=1.2, drop=0.0, dtype="bf16"),
        # the gradient of permute over a full training batch: every row read once, summed per token
        dict(name="permute_backward T8192", op="permute_backward", T=8192, K=4096, E=128, top_k=8, block_m=128,
             zipf=1.2, drop=0.0, dtype="bf16"),
        # an odd row length in fp32 (no 16-byte vectors), with dropped routes and tokens that keep none
        dict(name="unpermute T777 fp32 odd", op="unpermute", T=777, K=1001, E=48, top_k=6, block_m=32, zipf=0.0,
             drop=0.3, dtype="fp32"),
        # the weighted sum's gradient over a full batch: rows and routing weights
        dict(name="unpermute_backward T8192", op="unpermute_backward", T=8192, K=4096, E=128, top_k=8, block_m=128,
             zipf=1.2, drop=0.0, dtype="bf16"),
        # few tokens over few experts: the weights' bytes and the launch are what counts
        dict(name="up T64", op="up", T=64, K=1024, N=1024, E=8, top_k=2, block_m=64, zipf=0.0, drop=0.0),
        # a training batch, balanced: large products
        dict(name="up T8192", op="up", T=8192, K=2048, N=2048, E=64, top_k=8, block_m=128, zipf=0.0, drop=0.0),
        # skewed experts, some with very many rows and some with none
        dict(name="up_backward T4096 skewed", op="up_backward", T=4096, K=4096, N=512, E=128, top_k=8, block_m=128,
             zipf=1.2, drop=0.0),
        # odd tails in every direction and dropped routes
        dict(name="down T1000 ragged", op="down", T=1000, K=1992, N=1360, E=20, top_k=4, block_m=64, zipf=0.6,
             drop=0.1),
        # a training batch, balanced: SwiGLU's gradient behind the product, and the weights' gradient
        dict(name="down_backward T8192", op="down_backward", T=8192, K=2048, N=2048, E=64, top_k=8, block_m=128,
             zipf=0.0, drop=0.0),
        # one small matrix: fifteen dependent products, latency only
        dict(name="orthogonalize 1x256x256", op="orthogonalize", E=1, M=256, N=256, dtype="fp32"),
        # odd sides, taller than wide
        dict(name="orthogonalize 3x1537x1000", op="orthogonalize", E=3, M=1537, N=1000, dtype="bf16"),
        # a layer's experts together
        dict(name="orthogonalize 16x2048x2048", op="orthogonalize", E=16, M=2048, N=2048, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6e12, w["flops"] / 1.5e15)


def draw(rng):
    op = rng.choice(ROW_OPS + EXPERT_OPS + ("orthogonalize",) * 2)
    while True:
        if op == "orthogonalize":
            case = dict(op=op, E=_log(rng, 1, 16), M=_log(rng, 32, 2048), N=_log(rng, 32, 2048),
                        dtype=rng.choice(("bf16", "fp32")))
            if _cost(case) <= _cost(dict(op=op, E=16, M=2048, N=2048, dtype="bf16")):
                return case
            continue
        E, top_k = _log(rng, 2, 256 if op in ROW_OPS else 64), rng.randint(1, 8)
        case = dict(op=op, T=_log(rng, 1, 8192), E=max(E, top_k), top_k=top_k, block_m=rng.choice((16, 32, 64, 128)),
                    zipf=rng.choice((0.0, 0.6, 1.2)))
        case["drop"] = rng.choice((0.0, 0.0, 0.1, 0.5)) if case["T"] * top_k >= 16 else 0.0
        if op in ROW_OPS:
            K = _log(rng, 32, 8192)
            case.update(K=K if rng.random() < 0.4 else max(8, K // 8 * 8), dtype=rng.choice(("bf16", "fp32")))
            if case["T"] * top_k * case["K"] * (4 if case["dtype"] == "fp32" else 2) <= 8192 * 8 * 4096 * 2:
                return case
            continue
        case.update(K=max(1, _log(rng, 128, 4096) // 8) * 8, N=max(1, _log(rng, 128, 4096) // 16) * 16)
        blocks = (case["T"] * top_k + case["E"] * (case["block_m"] - 1)) // case["block_m"]
        top = dict(op=op, T=8192, K=2048, N=2048, E=64, top_k=8, drop=0.0)
        if _cost(case) <= _cost(top) and blocks * case["N"] * case["K"] * 4 <= 10e9:  # the plain form's weights, by block
            return case


def work(case):
    """Bytes and operations of one pass: every input once, every output once."""
    op = case["op"]
    if op == "orthogonalize":
        E, s, l = case["E"], min(case["M"], case["N"]), max(case["M"], case["N"])
        size = 4 if case["dtype"] == "fp32" else 2
        # X X^T and A A are symmetric: half of each
        return {"bytes": E * s * l * (size + 2.0), "flops": 5.0 * E * (3.0 * s * s * l + 1.0 * s * s * s)}
    T, K, E, k = case["T"], case["K"], case["E"], case["top_k"]
    R = T * k * (1.0 - case["drop"])
    if op in ROW_OPS:
        size = 4 if case["dtype"] == "fp32" else 2
        moved = {"permute": T + R, "permute_backward": T + R, "unpermute": T + R, "unpermute_backward": T + 2 * R}[op]
        ids = T * k * 4.0 + (T * k * (4.0 if op == "unpermute" else 8.0) if op.startswith("unpermute") else 0.0)
        flops = {"permute": 0.0, "permute_backward": R * K, "unpermute": 2.0 * R * K, "unpermute_backward": 3.0 * R * K}[op]
        return {"bytes": moved * K * size + ids, "flops": flops}
    N, half = case["N"], case["N"] // 2
    touched = min(float(E), R)
    if op == "up":
        return {"bytes": 2.0 * (R * (K + N + half) + touched * N * K), "flops": 2.0 * R * N * K}
    if op == "down":
        return {"bytes": 2.0 * (R * (K + half) + touched * half * K), "flops": 2.0 * R * half * K}
    if op == "up_backward":  # reads the gradient of h, the rows and w1; writes the gradients of the rows and of w1
        return {"bytes": 2.0 * (R * (N + 2 * K) + (touched + E) * N * K), "flops": 4.0 * R * N * K}
    # reads the gradient of y, h, act and w2; writes the gradients of h and of w2
    return {"bytes": 2.0 * (R * (K + 2 * N + half) + (touched + E) * half * K), "flops": 4.0 * R * half * K}


# ---------------------------------------------------------------------------------------------------- inputs
def _routes(case, g):
    """Routing as a gate makes it (softmax over logits, top-k, renormalised) and the planner's outputs for it."""
    T, E, k, bm = case["T"], case["E"], case["top_k"], case["block_m"]
    dev = "cuda"
    logits = torch.randn((T, E), generator=g, device=dev)
    rank = torch.randperm(E, generator=g, device=dev).float() + 1.0
    top, ids = torch.topk(logits - case["zipf"] * torch.log(rank), k, dim=1)
    weights = torch.softmax(top, dim=1)
    gone = torch.rand((T, k), generator=g, device=dev) < case["drop"]
    ids = torch.where(gone, torch.full_like(ids, -1), ids)

    capacity = T * k + E * (bm - 1)
    flat = ids.reshape(-1)
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.bincount(key, minlength=E + 1)[:E]
    padded = (counts + bm - 1) // bm * bm
    ends = torch.cumsum(padded, 0)
    n = int(counts.sum())
    order = order[:n]
    e = key[order]
    place = (ends - padded)[e] + torch.arange(n, device=dev) - (torch.cumsum(counts, 0) - counts)[e]
    sorted_ids = torch.full((capacity,), -1, dtype=torch.int32, device=dev)
    sorted_ids[place] = order.int()
    slots = torch.full((T * k,), -1, dtype=torch.int32, device=dev)
    slots[order] = place.int()
    blocks = torch.arange((capacity + bm - 1) // bm, device=dev)
    expert = torch.searchsorted(ends // bm, blocks, right=True)
    expert = torch.where(blocks < ends[-1] // bm, expert, torch.full_like(expert, -1))
    return dict(sorted_ids=sorted_ids, expert_ids=expert.int(), total=ends[-1:].int(), slots=slots.view(T, k),
                weights=weights, block_m=bm)


def prepare(case, seed):
    op, dev = case["op"], "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, generator=g, device=dev) * std).to(dtype)

    if op == "orthogonalize":
        # a gradient's moving average: a few strong directions above noise
        E, M, N = case["E"], case["M"], case["N"]
        r = max(1, min(M, N) // 8)
        strong = torch.bmm(normal(E, M, r, dtype=torch.float32), normal(E, r, N, dtype=torch.float32)) / math.sqrt(r)
        return dict(op=op, g=((strong + 0.5 * normal(E, M, N, dtype=torch.float32)) * 1e-3).to(DTYPES[case["dtype"]]),
                    out=torch.zeros((E, M, N), dtype=torch.bfloat16, device=dev))
    s = dict(_routes(case, g), op=op)
    T, K, E = case["T"], case["K"], case["E"]
    capacity = s["sorted_ids"].numel()
    live = (s["sorted_ids"] >= 0).unsqueeze(1)

    def rows(width, dtype=torch.bfloat16, std=1.0):
        """A row buffer of the planner's capacity: values at routed rows, zeros elsewhere."""
        return torch.where(live, normal(capacity, width, dtype=dtype, std=std), torch.zeros((), dtype=dtype, device=dev))

    def empty(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device=dev)

    if op in ROW_OPS:
        dt = DTYPES[case["dtype"]]
        if op in ("permute", "unpermute_backward"):
            s.update(token=normal(T, K, dtype=dt), row_out=empty(capacity, K, dtype=dt))
        if op != "permute":
            s.update(rows=rows(K, dtype=dt))
        if op in ("permute_backward", "unpermute"):
            s.update(token_out=empty(T, K, dtype=dt))
        return s
    N, half = case["N"], case["N"] // 2
    if op in ("up", "up_backward"):
        s.update(rows=rows(K), w1=normal(E, N, K, std=K ** -0.5))
    else:
        s.update(w2=normal(E, K, half, std=half ** -0.5))
    if op == "up":
        s.update(h_out=empty(capacity, N), act_out=empty(capacity, half))
    elif op == "down":
        s.update(act=rows(half, std=0.6), y_out=empty(capacity, K))
    elif op == "up_backward":
        s.update(grad_h=rows(N), grad_rows_out=empty(capacity, K), grad_w1_out=empty(E, N, K))
    else:
        h = rows(N)
        act = (torch.nn.functional.silu(h[:, :half].float()) * h[:, half:].float()).to(torch.bfloat16)
        s.update(grad_y=rows(K), h=h, act=act, grad_h_out=empty(capacity, N), grad_w2_out=empty(E, K, half))
    return s


# ---------------------------------------------------------------------------------------------------- the operators
def run(s):
    return _kernels(s) if own else _plain(s)


def _kernels(s):
    import mixture_experts_ffn_planner_b200 as moe

    op = s["op"]
    if op == "orthogonalize":
        return dict(out=moe.moe_orthogonalize(s["g"], out=s["out"]))
    if op == "permute":
        return dict(rows=moe.moe_permute(s["token"], s["sorted_ids"], s["total"], s["slots"], out=s["row_out"]))
    if op == "permute_backward":
        return dict(grad_x=moe.moe_permute_backward(s["rows"], s["slots"], out=s["token_out"]))
    if op == "unpermute":
        return dict(out=moe.moe_unpermute(s["rows"], s["slots"], s["weights"], out=s["token_out"]))
    if op == "unpermute_backward":
        gy, gw = moe.moe_unpermute_backward(s["token"], s["rows"], s["sorted_ids"], s["total"], s["slots"], s["weights"],
                                            grad_y=s["row_out"])
        return dict(grad_y=gy, grad_weights=gw)
    plan = (s["sorted_ids"], s["expert_ids"], s["total"], s["block_m"])
    if op == "up":
        h, act = moe.moe_expert_up(s["rows"], s["w1"], *plan, h=s["h_out"], act=s["act_out"])
        return dict(h=h, act=act)
    if op == "down":
        return dict(y=moe.moe_expert_down(s["act"], s["w2"], *plan, out=s["y_out"]))
    if op == "up_backward":
        gx, gw = moe.moe_expert_up_backward(s["grad_h"], s["rows"], s["w1"], *plan, grad_rows=s["grad_rows_out"],
                                            grad_w1=s["grad_w1_out"])
        return dict(grad_rows=gx, grad_w1=gw)
    gh, gw = moe.moe_expert_down_backward(s["grad_y"], s["h"], s["act"], s["w2"], *plan, grad_h=s["grad_h_out"],
                                          grad_w2=s["grad_w2_out"])
    return dict(grad_h=gh, grad_w2=gw)


def _newton_schulz(x):
    a, b, c = NS
    gram = torch.bmm(x, x.transpose(1, 2))
    return a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)


def _plain(s):
    op = s["op"]
    if op == "orthogonalize":
        x = s["g"].float()
        x = x / ((x * x).sum(dim=(1, 2), keepdim=True).sqrt() + NS_EPS)
        tall = x.shape[1] > x.shape[2]
        x = x.transpose(1, 2) if tall else x
        x = _newton_schulz(_newton_schulz(_newton_schulz(_newton_schulz(_newton_schulz(x)))))
        return dict(out=(x.transpose(1, 2) if tall else x).to(torch.bfloat16))
    ids, slots = s["sorted_ids"].long(), s["slots"].long()
    k = slots.shape[1]
    routed, kept = (ids >= 0).unsqueeze(1), (slots >= 0).unsqueeze(2)
    ids, slots = ids.clamp(min=0), slots.clamp(min=0)
    if op == "permute":
        return dict(rows=torch.where(routed, s["token"][ids // k], 0.0))
    if op in ("permute_backward", "unpermute"):
        picked = torch.where(kept, s["rows"][slots].float(), 0.0)
        if op == "permute_backward":
            return dict(grad_x=picked.sum(1).to(s["rows"].dtype))
        return dict(out=(picked * s["weights"].unsqueeze(2)).sum(1).to(s["rows"].dtype))
    if op == "unpermute_backward":
        grad = s["token"].float()
        weighted = grad[ids // k] * s["weights"].reshape(-1)[ids].unsqueeze(1)
        dots = (s["rows"][slots].float() * grad.unsqueeze(1)).sum(2, keepdim=True)
        return dict(grad_y=torch.where(routed, weighted, 0.0).to(s["token"].dtype),
                    grad_weights=torch.where(kept, dots, 0.0).squeeze(2))
    bm, half = s["block_m"], None
    n = ids.numel() // bm * bm                     # whole blocks; the padded total is a multiple of block_m
    expert = s["expert_ids"].long()[: n // bm]
    used = (expert >= 0).view(-1, 1, 1)
    expert = expert.clamp(min=0)
    behind = ids.numel() - n

    def blocks(t):
        return t[:n].float().view(n // bm, bm, t.shape[1])

    def flat(t):
        t = torch.where(routed[:n], t.reshape(n, t.shape[2]), 0.0)
        return torch.nn.functional.pad(t, (0, 0, 0, behind)).to(torch.bfloat16)

    def by_expert(grad, row, count):
        per_block = torch.where(used, torch.bmm(grad.transpose(1, 2), row), 0.0)
        total = torch.zeros((count,) + per_block.shape[1:], device=per_block.device)
        return total.index_add_(0, expert, per_block).to(torch.bfloat16)

    if op == "up":
        h = torch.bmm(blocks(s["rows"]), s["w1"].float()[expert].transpose(1, 2))
        half = h.shape[2] // 2
        gate, up = h[..., :half], h[..., half:]
        return dict(h=flat(h), act=flat(gate / (1.0 + torch.exp(-gate)) * up))
    if op == "down":
        return dict(y=flat(torch.bmm(blocks(s["act"]), s["w2"].float()[expert].transpose(1, 2))))
    if op == "up_backward":
        grad_h = blocks(s["grad_h"])
        grad_rows = flat(torch.bmm(grad_h, s["w1"].float()[expert]))
        return dict(grad_rows=grad_rows, grad_w1=by_expert(grad_h, blocks(s["rows"]), s["w1"].shape[0]))
    grad_y, h = blocks(s["grad_y"]), blocks(s["h"])
    half = h.shape[2] // 2
    gate, up = h[..., :half], h[..., half:]
    sig = 1.0 / (1.0 + torch.exp(-gate))
    grad_act = torch.bmm(grad_y, s["w2"].float()[expert])
    grad_h = torch.cat((grad_act * up * sig * (1.0 + gate * (1.0 - sig)), grad_act * gate * sig), dim=2)
    return dict(grad_h=flat(grad_h), grad_w2=by_expert(grad_y, blocks(s["act"]), s["w2"].shape[0]))


# ---------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """The outputs from the definitions, token by token's routes and expert by expert, in 64 bits."""
    s, op = prepare(case, seed), case["op"]
    if op == "orthogonalize":
        a, b, c = NS
        out = []
        for g in s["g"].double().unbind(0):
            x = g / (torch.linalg.matrix_norm(g) + NS_EPS)
            for _ in range(5):  # on the side that is shorter: (x x^T) x = x (x^T x)
                if x.shape[0] <= x.shape[1]:
                    m = x @ x.mT
                    x = a * x + b * (m @ x) + c * (m @ (m @ x))
                else:
                    m = x.mT @ x
                    x = a * x + b * (x @ m) + c * ((x @ m) @ m)
            out.append(x)
        return dict(out=torch.stack(out))
    T, k, bm = case["T"], case["top_k"], case["block_m"]
    slots, weights = s["slots"].long(), s["weights"].double()
    capacity = s["sorted_ids"].numel()
    if op in ROW_OPS:
        K, dev = case["K"], "cuda"
        row_out = torch.zeros((capacity, K), dtype=torch.float64, device=dev)
        token_out = torch.zeros((T, K), dtype=torch.float64, device=dev)
        grad_w = torch.zeros((T, k), dtype=torch.float64, device=dev)
        for j in range(k):
            t = torch.nonzero(slots[:, j] >= 0).squeeze(1)
            at = slots[t, j]
            if op == "permute":
                row_out[at] = s["token"][t].double()
            elif op == "permute_backward":
                token_out[t] += s["rows"][at].double()
            elif op == "unpermute":
                token_out[t] += weights[t, j, None] * s["rows"][at].double()
            else:
                row_out[at] = weights[t, j, None] * s["token"][t].double()
                grad_w[t, j] = (s["token"][t].double() * s["rows"][at].double()).sum(1)
        if op == "permute":
            return dict(rows=row_out)
        if op == "permute_backward":
            return dict(grad_x=token_out)
        return dict(out=token_out) if op == "unpermute" else dict(grad_y=row_out, grad_weights=grad_w)
    expert = s["expert_ids"].long().repeat_interleave(bm)[:capacity]
    routed = s["sorted_ids"] >= 0
    names = {"up": ("h", "act"), "down": ("y",), "up_backward": ("grad_rows", "grad_w1"),
             "down_backward": ("grad_h", "grad_w2")}[op]
    res = {n: torch.zeros(s[n + "_out"].shape, dtype=torch.float64, device="cuda") for n in names}
    for e in range(case["E"]):
        p = torch.nonzero(routed & (expert == e)).squeeze(1)
        if op == "up":
            gate, up = (s["rows"][p].double() @ s["w1"][e].double().mT).chunk(2, dim=1)
            res["h"][p] = torch.cat((gate, up), dim=1)
            res["act"][p] = gate * torch.sigmoid(gate) * up
        elif op == "down":
            res["y"][p] = s["act"][p].double() @ s["w2"][e].double().mT
        elif op == "up_backward":
            gh = s["grad_h"][p].double()
            res["grad_rows"][p] = gh @ s["w1"][e].double()
            res["grad_w1"][e] = gh.mT @ s["rows"][p].double()
        else:
            gy = s["grad_y"][p].double()
            gate, up = s["h"][p].double().chunk(2, dim=1)
            ga, sig = gy @ s["w2"][e].double(), torch.sigmoid(gate)
            res["grad_h"][p] = torch.cat((ga * up * (sig + gate * sig * (1 - sig)), ga * gate * sig), dim=1)
            res["grad_w2"][e] = gy.mT @ s["act"][p].double()
    return res
