"""Cases, plain forms and exact values of the operators around the expert layer.

linear_q4   y = x W^T (+ bias) with 4-bit weights and a scale for each group of inputs: the dense projections and the
            output head next to 4-bit experts
sample      one token id for each row of logits, with temperature, min-p, top-k and top-p, from given random numbers
balance     the router's per-expert counts and shares, the balance and z losses, and their gradient

``run`` computes the plain form with elementary torch operations, or, where ``own`` is true, calls this repository's
entry points on the same state.
"""
import math

import torch

own = False

MAX_LINEAR = 131072 * 4096 * 64      # N * K * T of the largest product
MAX_WEIGHTS = 131072 * 4096          # N * K
MAX_LOGITS = 128 * 131072            # T * V
MAX_ROUTER = 65537 * 512             # T * E


def listed():
    return [
        # one token through a square projection of a 2048-wide layer: latency counts
        dict(name="q4_1x2048x2048", op="linear_q4", T=1, N=2048, K=2048, group=32, x="bf16", y="f32", bias=False),
        # one token through the output head: the weight stream of a decode step
        dict(name="q4_1x131072x2048", op="linear_q4", T=1, N=131072, K=2048, group=32, x="bf16", y="f32", bias=False),
        # a small decode batch, fp32 activations, odd row and token counts, with a bias
        dict(name="q4_7x5001x1536_f32", op="linear_q4", T=7, N=5001, K=1536, group=64, x="f32", y="f32", bias=True),
        # a decode batch through a wide projection kept in the activations' type
        dict(name="q4_16x8192x4096", op="linear_q4", T=16, N=8192, K=4096, group=128, x="bf16", y="bf16", bias=True),
        # a large decode batch through the output head: the largest product
        dict(name="q4_64x131072x4096", op="linear_q4", T=64, N=131072, K=4096, group=128, x="bf16", y="f32", bias=False),
        # one request's next token: all three cuts on
        dict(name="sample_1x131072", op="sample", T=1, V=131072, logits="f32", cuts="all"),
        # a ragged decode batch over a small vocabulary, bf16 logits with many ties, requests with settings of their own
        dict(name="sample_17x5003_bf16", op="sample", T=17, V=5003, logits="bf16", cuts="mixed"),
        # a decode batch whose requests have settings of their own
        dict(name="sample_64x131072", op="sample", T=64, V=131072, logits="f32", cuts="mixed"),
        # a wide batch, top-p alone: the boundary may lie anywhere
        dict(name="sample_128x100003_bf16", op="sample", T=128, V=100003, logits="bf16", cuts="p"),
        # a decode batch's routing profile (the brightness behind a bias table)
        dict(name="balance_64x128", op="balance", T=64, E=128, k=8, z="f32", masked=False, step=False),
        # a prefill batch with padding: losses, profile and gradient
        dict(name="balance_16384x288_step", op="balance", T=16384, E=288, k=8, z="f32", masked=True, step=True),
        # a large training batch of bf16 logits, one token over a round number
        dict(name="balance_65537x512_step", op="balance", T=65537, E=512, k=10, z="bf16", masked=False, step=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear_q4", "sample", "balance"])
    if op == "linear_q4":
        # decode batches of one to 64 tokens over projections of hundreds of rows up to output heads
        group = rng.choice([32, 64, 128])
        K = max(group, _log(rng, 256, 8192) // group * group)
        N = min(_log(rng, 256, 131072), MAX_WEIGHTS // K)
        T = min(_log(rng, 1, 64), MAX_LINEAR // (N * K))
        return dict(op=op, T=T, N=N, K=K, group=group, x=rng.choice(["bf16", "bf16", "f32"]),
                    y=rng.choice(["bf16", "f32"]), bias=rng.random() < 0.5)
    if op == "sample":
        V = _log(rng, 1000, 160000)
        T = min(_log(rng, 1, 128), MAX_LOGITS // V)
        return dict(op=op, T=T, V=V, logits=rng.choice(["bf16", "f32"]),
                    cuts=rng.choice(["none", "k", "p", "min", "all", "mixed"]))
    # decode batches of a few tokens up to training batches
    E = _log(rng, 8, 1024)
    T = min(_log(rng, 1, 65536), MAX_ROUTER // E)
    return dict(op=op, T=T, E=E, k=rng.randint(1, min(10, E)), z=rng.choice(["bf16", "f32"]),
                masked=rng.random() < 0.5, step=rng.random() < 0.6)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def work(case):
    if case["op"] == "linear_q4":
        T, N, K = case["T"], case["N"], case["K"]
        return {"bytes": N * K // 2 + N * (K // case["group"]) * 2 + T * K * _BYTES[case["x"]]
                + T * N * _BYTES[case["y"]] + (4 * N if case["bias"] else 0), "flops": 2 * T * N * K}
    if case["op"] == "sample":
        T, V = case["T"], case["V"]
        return {"bytes": T * V * _BYTES[case["logits"]] + T * 28, "flops": T * V}
    T, E, k = case["T"], case["E"], case["k"]
    passes = 2 if case["step"] else 1  # z read, and dz written
    return {"bytes": passes * T * E * _BYTES[case["z"]] + T * k * 4 + T * (5 if case["masked"] else 4) + E * 12,
            "flops": 8 * passes * T * E}


# ----------------------------------------------------------------- inputs


def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _settings(cuts, T, g):
    """Per-row temperature, top-k, top-p and min-p as a server's requests bring them (None: a cut that is off for all)."""
    dev = "cuda"
    row = torch.arange(T, device=dev)
    temperature = 0.6 + 0.8 * torch.rand(T, device=dev, generator=g)
    if cuts == "mixed":
        temperature = torch.where(row % 7 == 3, torch.zeros_like(temperature), temperature)  # greedy requests
        top_k = torch.where(row % 3 == 0, 40, torch.where(row % 3 == 1, 0, 5 + 11 * row)).to(torch.int32)
        top_p = torch.where(row % 2 == 0, 0.9, 1.0).to(torch.float32)
        min_p = torch.where(row % 4 < 2, 0.0, 0.02).to(torch.float32)
        return temperature, top_k, top_p, min_p
    top_k = torch.full((T,), 50, dtype=torch.int32, device=dev) if cuts in ("k", "all") else None
    top_p = torch.full((T,), 0.95, device=dev) if cuts in ("p", "all") else None
    min_p = torch.full((T,), 0.01, device=dev) if cuts in ("min", "all") else None
    return temperature, top_k, top_p, min_p


def prepare(case, seed):
    g, dev = _generator(seed), "cuda"
    if case["op"] == "linear_q4":
        T, N, K, group = case["T"], case["N"], case["K"], case["group"]
        s = dict(case=case)
        s["wq"] = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device=dev, generator=g)
        s["scales"] = (0.003 + 0.004 * torch.rand(N, K // group, device=dev, generator=g)).half()
        s["x"] = torch.randn(T, K, device=dev, generator=g).to(_TYPES[case["x"]])
        s["bias"] = 0.1 * torch.randn(N, device=dev, generator=g) if case["bias"] else None
        s["out"] = torch.empty(T, N, dtype=_TYPES[case["y"]], device=dev)
        return s
    if case["op"] == "sample":
        T, V = case["T"], case["V"]
        s = dict(case=case)
        # a broad bulk and a few tokens that stand out, as an output head gives them
        bulk = 2.0 * torch.randn(T, V, device=dev, generator=g)
        head = torch.rand(T, V, device=dev, generator=g).log_().neg_().sub_(7.0).clamp_(min=0.0)
        s["logits"] = bulk.add_(head, alpha=2.5).to(_TYPES[case["logits"]])
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _settings(case["cuts"], T, g)
        s["u"] = torch.rand(T, device=dev, generator=g)
        s["ids"] = torch.empty(T, dtype=torch.int32, device=dev)
        s["prob"] = torch.empty(T, device=dev)
        return s
    T, E, k = case["T"], case["E"], case["k"]
    s = dict(case=case)
    z = torch.randn(T, E, device=dev, generator=g) * 1.5 + torch.randn(E, device=dev, generator=g) * 0.7
    s["z"] = z.to(_TYPES[case["z"]])
    s["ids"] = s["z"].float().topk(k, dim=1).indices.to(torch.int32)
    s["mask"] = None
    if case["masked"]:  # a padded batch: the first token is never padding
        s["mask"] = ((torch.rand(T, device=dev, generator=g) < 0.9) | (torch.arange(T, device=dev) == 0)).to(torch.uint8)
    s["dloss"] = torch.tensor([0.01, 0.001], device=dev)
    s["counts"] = torch.empty(E, dtype=torch.int32, device=dev)
    s["totals"] = torch.empty(2, dtype=torch.int32, device=dev)
    s["share"] = torch.empty(E, dtype=torch.float64, device=dev)
    s["lse"] = torch.empty(T, device=dev)
    s["loss"] = torch.empty(2, device=dev)
    s["dz"] = torch.empty_like(s["z"]) if case["step"] else None
    return s


# -------------------------------------------------------------- one pass


def run(state):
    c = state["case"]
    if c["op"] == "linear_q4":
        return _own_linear(state) if own else _linear(state)
    if c["op"] == "sample":
        return _own_sample(state) if own else _sample(state)
    return _own_balance(state) if own else _balance(state)


def _format(m, name):
    return m.MOE_X_BF16 if name == "bf16" else m.MOE_X_F32


def _own_linear(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    m.moe_linear_q4(s["x"], _format(m, c["x"]), c["K"], s["wq"], s["scales"], c["group"], s["bias"], c["T"], c["N"],
                    c["K"], s["out"], _format(m, c["y"]), c["N"])
    return s["out"]


def _own_sample(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    if "ws" not in s:  # kept by the caller, as every workspace is
        s["ws_bytes"] = m.moe_sample_workspace_bytes(c["T"], c["V"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    m.moe_sample(s["logits"], _format(m, c["logits"]), c["V"], c["T"], c["V"], s["temperature"], s["min_p"], s["top_k"],
                 s["top_p"], s["u"], s["ids"], s["prob"], s["ws"], s["ws_bytes"])
    return {"ids": s["ids"], "prob": s["prob"]}


def _own_balance(s):
    import expert_vram_slot_amd as m
    c = s["case"]
    if "ws" not in s:
        s["ws_bytes"] = m.moe_balance_workspace_bytes(c["T"], c["E"])
        s["ws"] = torch.empty(s["ws_bytes"], dtype=torch.uint8, device="cuda")
    zt = _format(m, c["z"])
    m.moe_balance_loss(s["z"], zt, s["ids"], s["mask"], c["T"], c["E"], c["k"], s["counts"], s["totals"], s["share"],
                       s["lse"], s["loss"], s["ws"], s["ws_bytes"])
    out = {n: s[n] for n in ("counts", "totals", "share", "lse", "loss")}
    if c["step"]:
        m.moe_balance_loss_bwd(s["z"], zt, s["lse"], s["mask"], s["counts"], s["totals"], s["dloss"], c["T"], c["E"],
                               s["dz"])
        out["dz"] = s["dz"]
    return out


def _linear(s):
    c = s["case"]
    N, K, group = c["N"], c["K"], c["group"]
    b = s["wq"].view(N, K // 32, 16)
    q = torch.cat([b & 15, b >> 4], dim=2)  # byte j of a block: input j low, input j + 16 high
    w = (q.view(N, K // group, group).float() - 8.0) * s["scales"].float()[:, :, None]
    y = s["x"].float() @ w.view(N, K).T
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(_TYPES[c["y"]])


def _sample(s):
    logits, V = s["logits"].double(), s["case"]["V"]
    live = logits > -math.inf  # false for NaN too
    l = torch.where(live, logits, -math.inf)
    top = l.max(dim=1, keepdim=True).values
    temperature = s["temperature"].double()[:, None]
    greedy = ~(temperature > 0)
    w = torch.where(live, torch.exp((l - top) / torch.where(greedy, 1.0, temperature)), 0.0)
    w = torch.where(live & (l == top), 1.0, w)
    if s["min_p"] is not None:
        low = w < s["min_p"].double()[:, None].clamp(max=1.0)
        w, l = torch.where(low, 0.0, w), torch.where(low, -math.inf, l)
    order = torch.sort(l, dim=1, descending=True, stable=True).indices  # ties: the lower id first
    ranked = w.gather(1, order)
    rank = torch.arange(V, device=w.device)[None]
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        ranked = torch.where((k > 0) & (rank >= k), 0.0, ranked)
    ranked = torch.where(greedy & (rank >= 1), 0.0, ranked)
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = ranked.cumsum(dim=1) - ranked
        cut = (p < 1) & (before >= p * ranked.sum(dim=1, keepdim=True)) & (rank > 0)
        ranked = torch.where(cut, 0.0, ranked)
    kept = torch.zeros_like(w).scatter_(1, order, ranked)
    cum = kept.cumsum(dim=1)
    total = cum[:, -1:]
    ids = (cum > s["u"].double()[:, None] * total).to(torch.uint8).argmax(dim=1)
    prob = kept.gather(1, ids[:, None])[:, 0] / total[:, 0]
    empty = total[:, 0] == 0
    return {"ids": torch.where(empty, -1, ids).to(torch.int32), "prob": torch.where(empty, 0.0, prob).float()}


def _balance(s):
    c = s["case"]
    E = c["E"]
    z = s["z"].double()  # in 64 bits: the shares are sums over every token
    lse = torch.logsumexp(z, dim=1)
    p = torch.exp(z - lse[:, None])
    live = torch.ones_like(lse) if s["mask"] is None else s["mask"].double()
    n = live.sum()
    ids = s["ids"].long()
    hit = torch.where(live[:, None] > 0, ids, E).reshape(-1)
    counts = torch.zeros(E + 1, dtype=torch.int64, device=z.device).index_add_(0, hit, torch.ones_like(hit))[:E]
    picks = counts.sum()
    share = (p * live[:, None]).sum(dim=0) / n.clamp(min=1)
    f = counts.double() / picks.clamp(min=1)
    zero = torch.where(live > 0, lse, 0.0)
    loss = torch.stack([E * (f * share).sum(), (zero * zero).sum() / n.clamp(min=1)])
    out = {"counts": counts.to(torch.int32), "totals": torch.stack([n.long(), picks]).to(torch.int32), "share": share,
           "lse": zero.float(), "loss": loss.float()}
    if c["step"]:
        d = s["dloss"].double()
        inner = f[None] - (p * f).sum(dim=1, keepdim=True)
        dz = p * (d[0] * E * inner + d[1] * 2.0 * lse[:, None]) / n.clamp(min=1)
        out["dz"] = (dz * live[:, None]).to(s["z"].dtype)
    return out


# ------------------------------------------------- the definitions in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear_q4":
        return _exact_linear(s)
    if case["op"] == "sample":
        return _exact_sample(s)
    return _exact_balance(s)


def _exact_linear(s):
    c = s["case"]
    x = s["x"].double()
    value = torch.arange(16, dtype=torch.float64, device="cuda") - 8.0
    rows = []
    for r in range(0, c["N"], 16384):
        codes = s["wq"][r:r + 16384].long()
        n = codes.shape[0]
        w = torch.empty(n, c["K"] // 32, 32, dtype=torch.float64, device="cuda")
        w[:, :, :16] = value[(codes % 16).view(n, -1, 16)]
        w[:, :, 16:] = value[(codes // 16).view(n, -1, 16)]
        w = w.view(n, c["K"]) * s["scales"][r:r + 16384].double().repeat_interleave(c["group"], dim=1)
        rows.append(x @ w.t().contiguous())
    y = torch.cat(rows, dim=1)
    return y if s["bias"] is None else y + s["bias"].double()


def _exact_sample(s):
    import numpy as np
    logits = s["logits"].double().cpu().numpy()
    T, V = logits.shape
    host = {n: None if s[n] is None else s[n].double().cpu().numpy() for n in ("temperature", "min_p", "top_k", "top_p", "u")}
    ids, prob = np.full(T, -1, np.int32), np.zeros(T)
    for t in range(T):
        l = logits[t]
        index = np.nonzero(l > -np.inf)[0]
        if not len(index):
            continue
        index = index[np.argsort(-l[index], kind="stable")]
        top, temp = l[index[0]], host["temperature"][t]
        if not temp > 0:
            ids[t], prob[t] = index[0], 1.0
            continue
        w = np.where(l[index] == top, 1.0, np.exp((l[index] - top) / temp))
        keep = len(index)
        if host["min_p"] is not None:
            keep = int(np.sum(w >= min(host["min_p"][t], 1.0)))
        if host["top_k"] is not None and host["top_k"][t] > 0:
            keep = min(keep, int(host["top_k"][t]))
        if host["top_p"] is not None and host["top_p"][t] < 1:
            mass = np.cumsum(w[:keep])
            keep = min(keep, 1 + int(np.searchsorted(mass, host["top_p"][t] * mass[-1], side="left")))
        index, w = index[:keep], w[:keep]
        by_id = np.argsort(index)
        index, w = index[by_id], w[by_id]
        mass = np.cumsum(w)
        at = min(int(np.searchsorted(mass, host["u"][t] * mass[-1], side="right")), keep - 1)
        ids[t], prob[t] = index[at], w[at] / mass[-1]
    return {"ids": ids, "prob": prob}


def _exact_balance(s):
    c = s["case"]
    T, E = c["T"], c["E"]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if s["mask"] is None else s["mask"] != 0
    n = int(live.sum())
    counts = torch.bincount(s["ids"][live].reshape(-1).long(), minlength=E)
    picks = int(counts.sum())
    z = s["z"].double()
    top = z.amax(dim=1, keepdim=True)
    e = (z - top).exp()
    total = e.sum(dim=1, keepdim=True)
    lse = (total.log() + top)[:, 0]
    p = e / total
    share = p[live].sum(dim=0) / max(n, 1)
    f = counts.double() / max(picks, 1)
    lse = torch.where(live, lse, torch.zeros_like(lse))
    loss = torch.stack([E * torch.dot(f, share), lse.square().sum() / max(n, 1)])
    out = {"counts": counts.int(), "totals": torch.tensor([n, picks], dtype=torch.int32), "share": share, "lse": lse,
           "loss": loss}
    if c["step"]:
        d = s["dloss"].double()
        g = d[0] * E / max(n, 1) * f
        dp = g - (p @ g)[:, None]
        dz = p * dp + (2.0 * d[1] / max(n, 1)) * lse[:, None] * p
        out["dz"] = torch.where(live[:, None], dz, torch.zeros_like(dz))
    return out
