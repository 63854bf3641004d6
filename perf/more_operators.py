"""Cases, plain forms and exact values of the router's selection rules and of the adapters beside the 4-bit products.

select        a token's experts and their weights from the router's logits: softmax or sigmoid scores, a bias on the
              scores, groups, top-k, renormalised weights; with ``step`` also the gradient of the weights to the logits
bias          one step of the bias that balances the experts' picks, for every layer of a stack
lora          y = base + scale * B (A x), each token with its request's adapter

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, calls this repository's
entry points on the same state.
"""
import math

import torch

own = False

MAX_ROUTER = 65537 * 512                 # T * E
MAX_LORA = 16384 * (4096 + 4096)         # T * (N + K)
MAX_POOL = 16 * 16 * (131072 + 4096)     # n * r * (N + K), adapter values in use


def listed():
    return [
        # one request's token through a 128-expert router, the softmax renormalised over the picks: latency counts
        dict(name="select_1x128", op="select", T=1, E=128, k=8, z="f32", score="softmax", bias=False, groups=1, kept=1,
             top=1, renorm=True, scale=1.0, masked=False, step=False, add=False),
        # a decode batch through a 288-expert router with a balance bias and groups
        dict(name="select_64x288_groups", op="select", T=64, E=288, k=8, z="f32", score="sigmoid", bias=True, groups=8,
             kept=4, top=2, renorm=True, scale=2.5, masked=False, step=False, add=False),
        # a prompt through a 512-expert router, raw softmax scores, bf16 logits with many ties
        dict(name="select_4096x512_bf16", op="select", T=4096, E=512, k=10, z="bf16", score="softmax", bias=False,
             groups=1, kept=1, top=1, renorm=False, scale=1.0, masked=False, step=False, add=False),
        # a padded training batch: sigmoid scores, bias and groups, the gradient added to that of the balance loss
        dict(name="select_16384x288_step", op="select", T=16384, E=288, k=8, z="f32", score="sigmoid", bias=True,
             groups=8, kept=4, top=2, renorm=True, scale=2.5, masked=True, step=True, add=True),
        # a large training batch of bf16 logits, one token over a round number; the raw softmax's gradient is dense
        dict(name="select_65537x512_step", op="select", T=65537, E=512, k=10, z="bf16", score="softmax", bias=True,
             groups=1, kept=1, top=1, renorm=False, scale=1.0, masked=False, step=True, add=False),
        # one layer's balance bias: the smallest call
        dict(name="bias_1x288", op="bias", L=1, E=288),
        # the biases of a whole stack
        dict(name="bias_48x512", op="bias", L=48, E=512),
        # one request's token beside a square projection of a 2048-wide layer: latency counts
        dict(name="lora_1x2048x2048", op="lora", T=1, N=2048, K=2048, n=4, r=16, x="bf16", y="f32", order="mixed",
             ranks=False, idle=False),
        # a small decode batch, fp32 activations, odd row and token counts, adapters of several ranks, some requests
        # without one
        dict(name="lora_7x5001x1536_f32", op="lora", T=7, N=5001, K=1536, n=5, r=24, x="f32", y="f32", order="mixed",
             ranks=True, idle=True),
        # a decode batch beside the output head
        dict(name="lora_64x131072x4096", op="lora", T=64, N=131072, K=4096, n=16, r=16, x="bf16", y="f32",
             order="mixed", ranks=False, idle=True),
        # a large decode batch of many tenants beside a wide projection
        dict(name="lora_257x8192x4096", op="lora", T=257, N=8192, K=4096, n=64, r=32, x="bf16", y="bf16",
             order="mixed", ranks=True, idle=False),
        # the prompts of eight requests, one behind the other
        dict(name="lora_16384x4096x4096", op="lora", T=16384, N=4096, K=4096, n=8, r=64, x="bf16", y="bf16",
             order="runs", ranks=False, idle=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["select", "select", "bias", "lora", "lora"])
    if op == "select":
        # decode batches of a few tokens up to training batches
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        E = max(1, _log(rng, max(8, 2 * groups), 1024) // groups) * groups
        T = min(_log(rng, 1, 65536), MAX_ROUTER // E)
        kept = rng.randint(1, groups)
        step = rng.random() < 0.5
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(16, E // groups * kept)), z=rng.choice(["bf16", "f32"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.6, groups=groups, kept=kept,
                    top=rng.choice([1, 2]), renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    masked=rng.random() < 0.4, step=step, add=step and rng.random() < 0.5)
    if op == "bias":
        return dict(op=op, L=_log(rng, 1, 96), E=_log(rng, 8, 1024))
    # decode batches and prompts over projections of hundreds of rows up to output heads
    K = _log(rng, 256, 8192) // 8 * 8
    N = _log(rng, 256, 131072)
    r = rng.choice([8, 16, 32, 64, 128])
    T = min(_log(rng, 1, 16384), MAX_LORA // (N + K))
    n = max(1, min(_log(rng, 1, 64), MAX_POOL // (r * (N + K))))
    return dict(op=op, T=T, N=N, K=K, n=n, r=r, x=rng.choice(["bf16", "bf16", "f32"]), y=rng.choice(["bf16", "f32"]),
                order="runs" if T > 1024 else rng.choice(["mixed", "runs"]), ranks=rng.random() < 0.4,
                idle=rng.random() < 0.4)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def _ranks(case):
    """Ranks of the pool's adapters: all r, or from r down."""
    n, r = case["n"], case["r"]
    return [r - 5 * a % r if case["ranks"] else r for a in range(n)]


def work(case):
    if case["op"] == "select":
        T, E, k, b = case["T"], case["E"], case["k"], _BYTES[case["z"]]
        n = T * E * b + T * k * 8 + (4 * E if case["bias"] else 0) + (T if case["masked"] else 0)
        if case["step"]:  # dz written, the picks and their gradients read, what is added read
            n += T * E * b * (2 if case["add"] else 1) + T * k * 4
        return {"bytes": n, "flops": T * E * (8 if case["step"] else 4)}
    if case["op"] == "bias":
        return {"bytes": 12 * case["L"] * case["E"], "flops": 4 * case["L"] * case["E"]}
    T, N, K, n, r = case["T"], case["N"], case["K"], case["n"], case["r"]
    ranks = _ranks(case)
    used = sorted(ranks[a] for a in range(n))[::-1][:min(n, T)]
    return {"bytes": T * K * _BYTES[case["x"]] + 2 * T * N * _BYTES[case["y"]] + 2 * sum(used) * (N + K) + T * 4,
            "flops": 2 * T * (N + K) * sum(ranks) // n}


# ----------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def prepare(case, seed):
    g, dev = _generator(seed), "cuda"
    s = dict(case=case)
    if case["op"] == "select":
        T, E, k = case["T"], case["E"], case["k"]
        z = torch.randn(T, E, device=dev, generator=g) * 1.5 + torch.randn(E, device=dev, generator=g) * 0.7
        s["z"] = z.to(_TYPES[case["z"]])
        s["bias"] = None
        if case["bias"]:  # some steps of a thousandth, as moe_bias_balance leaves them
            s["bias"] = torch.randint(-60, 61, (E,), device=dev, generator=g).float() * 0.001
        s["mask"] = None
        if case["masked"]:  # a padded batch: the first token is never padding
            s["mask"] = ((torch.rand(T, device=dev, generator=g) < 0.9) | (torch.arange(T, device=dev) == 0)).to(torch.uint8)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["w"] = torch.empty(T, k, device=dev)
        if case["step"]:
            s["dw"] = torch.randn(T, k, device=dev, generator=g)
            s["add"] = (1e-3 * torch.randn(T, E, device=dev, generator=g)).to(s["z"].dtype) if case["add"] else None
            s["dz"] = torch.empty_like(s["z"])
        return s
    if case["op"] == "bias":
        L, E = case["L"], case["E"]
        # picks of 4096 tokens, top-8, spread unevenly; small multiples of the rate as the bias so far
        s["counts"] = torch.poisson(torch.rand(L, E, device=dev, generator=g) * (65536.0 / E), generator=g).to(torch.int32)
        s["bias"] = torch.randint(-60, 61, (L, E), device=dev, generator=g).float() * 0.001
        s["out"] = torch.empty(L, E, device=dev)
        return s
    T, N, K, n, r = case["T"], case["N"], case["K"], case["n"], case["r"]
    s["x"] = torch.randn(T, K, device=dev, generator=g).to(_TYPES[case["x"]])
    s["a"] = (torch.randn(n, r, K, device=dev, generator=g) * K ** -0.5).bfloat16()
    s["b"] = (torch.randn(n, N, r, device=dev, generator=g) * 0.3 * r ** -0.5).bfloat16()
    s["ranks"] = torch.tensor(_ranks(case), dtype=torch.int32, device=dev) if case["ranks"] else None
    s["scale"] = 0.5 + 1.5 * torch.rand(n, device=dev, generator=g)
    at = torch.arange(T, device=dev)
    ids = at * n // T if case["order"] == "runs" else (at % n)[torch.randperm(T, device=dev, generator=g)]
    if case["idle"]:  # one request in five has no adapter
        ids = torch.where(torch.rand(T, device=dev, generator=g) < 0.2, -1, ids)
    s["ids"] = ids.to(torch.int32)
    s["base"] = torch.randn(T, N, device=dev, generator=g).to(_TYPES[case["y"]])
    s["y"] = torch.empty_like(s["base"])
    return s


# -------------------------------------------------------------- one pass


def run(state):
    op = state["case"]["op"]
    if op == "select":
        return _own_select(state) if own else _select(state)
    if op == "bias":
        return _own_bias(state) if own else _bias(state)
    return _own_lora(state) if own else _lora(state)


def _format(m, name):
    return m.MOE_X_BF16 if name == "bf16" else m.MOE_X_F32


def _own_select(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    if "rule" not in s:  # kept by the caller, as a layer keeps it
        s["rule"] = m.select_rule(score=c["score"], groups=c["groups"], groups_kept=c["kept"], group_top=c["top"],
                                  renorm=c["renorm"], scale=c["scale"])
    zt = _format(m, c["z"])
    m.moe_route_select(s["z"], zt, s["bias"], s["mask"], None, c["T"], c["E"], c["k"], s["rule"], s["ids"], s["w"])
    out = {"ids": s["ids"], "w": s["w"]}
    if c["step"]:
        m.moe_route_select_bwd(s["z"], zt, s["ids"], s["dw"], c["T"], c["E"], c["k"], s["rule"], s["add"], s["dz"])
        out["dz"] = s["dz"]
    return out


def _own_bias(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    m.moe_bias_balance(s["counts"], s["bias"], c["L"], c["E"], 0.001, s["out"])
    return s["out"]


def _own_lora(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    if "ws" not in s:  # kept by the caller, as every workspace is
        s["ws_bytes"] = m.moe_lora_workspace_bytes(c["T"], c["K"], c["r"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    m.moe_lora_add(s["x"], _format(m, c["x"]), c["K"], s["a"], s["b"], s["ranks"], s["scale"], s["ids"], c["n"], c["r"],
                   c["T"], c["N"], c["K"], s["base"], c["N"], s["y"], _format(m, c["y"]), c["N"], s["ws"], s["ws_bytes"])
    return s["y"]


def _scores(z, score):
    if score == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-z))
    e = torch.exp(z - z.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _select(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["z"].double()  # in 64 bits: choices next to one another decide which expert is taken
    p = _scores(z, c["score"])
    choice = p if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        best = choice.view(T, G, E // G).topk(min(c["top"], E // G), dim=2).values.sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["kept"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, order, True)
        choice = torch.where(kept.repeat_interleave(E // G, dim=1), choice, -math.inf)
    by_z = torch.sort(z, dim=1, descending=True, stable=True).indices  # ties: the higher logit, then the lower id
    order = torch.sort(choice.gather(1, by_z), dim=1, descending=True, stable=True).indices[:, :k]
    ids = by_z.gather(1, order)
    picked = p.gather(1, ids)
    total = picked.sum(dim=1, keepdim=True) if c["renorm"] else torch.ones_like(picked[:, :1])
    share = picked / total
    live = torch.ones(T, dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"] != 0
    out = {"ids": torch.where(live[:, None], ids, -1).to(torch.int32),
           "w": torch.where(live[:, None], c["scale"] * share, 0.0).float()}
    if c["step"]:
        h = c["scale"] * s["dw"].double()
        dp = (h - (h * share).sum(dim=1, keepdim=True) if c["renorm"] else h) / total
        if c["score"] == "sigmoid":
            dz = torch.zeros_like(z).scatter_(1, ids, dp * picked * (1.0 - picked))
        else:
            dz = torch.zeros_like(z).scatter_(1, ids, dp)
            dz = p * (dz - (dz * p).sum(dim=1, keepdim=True))
        dz = torch.where(live[:, None], dz, 0.0)
        out["dz"] = (dz if s["add"] is None else dz + s["add"].double()).to(s["z"].dtype)
    return out


def _bias(s):
    counts = s["counts"].long()
    return s["bias"] + 0.001 * torch.sign(counts.sum(dim=1, keepdim=True) - s["case"]["E"] * counts).float()


def _lora(s):
    c = s["case"]
    n, r = c["n"], c["r"]
    ranks = torch.full((n,), r, device="cuda") if s["ranks"] is None else s["ranks"]
    # every adapter's inner products, then those of the token's own adapter alone
    h = s["x"].float() @ s["a"].float().view(n * r, c["K"]).T
    at = torch.arange(n * r, device="cuda")
    mine = (at[None] // r == s["ids"][:, None]) & (at % r < ranks.repeat_interleave(r))
    h = torch.where(mine, h * s["scale"].repeat_interleave(r), 0.0)
    y = h @ s["b"].float().transpose(0, 1).reshape(c["N"], n * r).T
    return (y + s["base"].float()).to(_TYPES[c["y"]])


# ------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"select": _exact_select, "bias": _exact_bias, "lora": _exact_lora}[case["op"]](s)


def _exact_select(s):
    c = s["case"]
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    z = s["z"].double()
    if c["score"] == "softmax":
        log_p = z - torch.logsumexp(z, dim=1, keepdim=True)
    else:
        log_p = torch.clamp(z, max=0.0) - torch.log1p(torch.exp(-z.abs()))
    p = log_p.exp()
    left = p.clone() if s["bias"] is None else p + s["bias"].double()
    if G > 1:
        rest = left.view(T, G, -1).clone()
        value = torch.zeros(T, G, dtype=torch.float64, device="cuda")
        for _ in range(min(c["top"], E // G)):
            top = rest.max(dim=2, keepdim=True)
            value += top.values[:, :, 0]
            rest.scatter_(2, top.indices, -math.inf)
        g = torch.arange(G, device="cuda")
        ahead = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & (g[None, :] < g[:, None]))
        left.view(T, G, -1)[ahead.sum(dim=2) >= c["kept"]] = -math.inf
    picks = []
    for _ in range(k):
        first = left == left.max(dim=1, keepdim=True).values
        first &= z == torch.where(first, z, -math.inf).max(dim=1, keepdim=True).values
        picks.append(first.to(torch.uint8).argmax(dim=1))  # of what is left the lowest id
        left[torch.arange(T, device="cuda"), picks[-1]] = -math.inf
    ids = torch.stack(picks, dim=1)
    mine = log_p.gather(1, ids)
    share = torch.softmax(mine, dim=1) if c["renorm"] else mine.exp()
    live = torch.ones(T, 1, device="cuda", dtype=torch.float64) if s["mask"] is None else (s["mask"] != 0).double()[:, None]
    out = {"ids": torch.where(live > 0, ids, -1).int(), "w": c["scale"] * share * live}
    if c["step"]:
        # through d log p: of a sigmoid 1 - p, of a softmax one less p everywhere
        dlog = c["scale"] * s["dw"].double() * share * live
        if c["renorm"]:
            dlog = dlog - share * dlog.sum(dim=1, keepdim=True)
        if c["score"] == "sigmoid":
            dz = torch.zeros_like(z).scatter_add_(1, ids, dlog * torch.sigmoid(-z.gather(1, ids)))
        else:
            dz = torch.zeros_like(z).scatter_add_(1, ids, dlog) - p * dlog.sum(dim=1, keepdim=True)
        out["dz"] = dz if s["add"] is None else dz + s["add"].double()
    return out


def _exact_bias(s):
    counts = s["counts"].double()
    mean = counts.mean(dim=1, keepdim=True)
    step = torch.where(counts < mean, 1.0, torch.where(counts > mean, -1.0, 0.0)).double()
    return s["bias"].double() + 0.001 * step


def _exact_lora(s):
    c = s["case"]
    y = s["base"].double()
    ids = s["ids"].tolist()
    ranks = [c["r"]] * c["n"] if s["ranks"] is None else s["ranks"].tolist()
    for a in sorted(set(ids) - {-1}):
        rows = torch.tensor([t for t, i in enumerate(ids) if i == a], device="cuda")
        down = s["a"][a, :ranks[a]].double().t().contiguous()
        up = s["b"][a, :, :ranks[a]].double().t().contiguous()
        y[rows] += float(s["scale"][a]) * ((s["x"][rows].double() @ down) @ up)
    return y
