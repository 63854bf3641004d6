"""Plain 64-bit references of moe_route_select (and its gradient), moe_bias_balance and moe_lora_add (numpy only)."""
import numpy as np


def scores(z, score):
    """s of every expert of [T][E] logits; 0 where the logit is not above -inf."""
    z = np.where(z > -np.inf, z.astype(np.float64), -np.inf)
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(z))
            return np.where(z >= 0, 1 / (1 + e), e / (1 + e))
        m = z.max(axis=1, keepdims=True)
        e = np.where(z == -np.inf, 0.0, np.where(z == m, 1.0, np.exp(z - m)))
        total = e.sum(axis=1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total > 0)


def log_scores(z, score):
    """log s up to a constant of the row, for ratios of scores too small for a double."""
    z = z.astype(np.float64)
    return np.minimum(z, 0) - np.log1p(np.exp(-np.abs(z))) if score == "sigmoid" else z


def choose(z, s, k, bias=None, groups=1, kept=1, top=1):
    """Picks of one token: z, s [E] in double; -1 where there are no more."""
    E = len(z)
    b = np.zeros(E) if bias is None else bias.astype(np.float64)
    is_open = (z > -np.inf) & (b > -np.inf)
    with np.errstate(invalid="ignore"):
        c = np.where(is_open, s + b, -np.inf)
    gs = E // groups
    if groups > 1:
        value = np.full(groups, -np.inf)
        for g in range(groups):
            best = np.sort(c[g * gs:(g + 1) * gs][is_open[g * gs:(g + 1) * gs]])[::-1][:top]
            if len(best):
                value[g] = best.sum()
        some = [g for g in range(groups) if is_open[g * gs:(g + 1) * gs].any()]
        keep = sorted(some, key=lambda g: (-value[g], g))[:kept]
        is_open = is_open & np.isin(np.arange(E) // gs, keep)
    order = sorted(np.nonzero(is_open)[0], key=lambda e: (-c[e], -z[e], e))[:k]
    return np.array(list(order) + [-1] * (k - len(order)), np.int64)


def shares(z, s, ids, score, renorm):
    """Weights over scale of one token's picks."""
    ok = (ids >= 0) & (ids < len(z))
    ok[ok] = z[ids[ok]] > -np.inf
    q = np.zeros(len(ids))
    if ok.any():
        if renorm:
            l = log_scores(z[ids[ok]], score)
            with np.errstate(invalid="ignore"):
                r = np.where(l == l.max(), 1.0, np.exp(l - l.max()))
            q[ok] = r / r.sum()
        else:
            q[ok] = s[ids[ok]]
    return q, ok


def select(z, k, score="softmax", bias=None, mask=None, ids_in=None, groups=1, kept=1, top=1, renorm=True, scale=1.0):
    """(ids, w, s) of [T][E] logits."""
    T = len(z)
    z = np.where(z > -np.inf, z.astype(np.float64), -np.inf)
    s = scores(z, score)
    ids, w = np.full((T, k), -1, np.int64), np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        ids[t] = choose(z[t], s[t], k, bias, groups, kept, top) if ids_in is None else ids_in[t]
        w[t] = scale * shares(z[t], s[t], ids[t], score, renorm)[0]
    return ids, w, s


def select_grad(z, ids, dw, score="softmax", renorm=True, scale=1.0):
    """(dz, size): size, the sum of the magnitudes of what is added up in each place."""
    z = np.where(z > -np.inf, z.astype(np.float64), -np.inf)
    s = scores(z, score)
    dz, size = np.zeros(z.shape), np.zeros(z.shape)
    for t in range(len(z)):
        q, ok = shares(z[t], s[t], ids[t], score, renorm)
        h = np.where(ok, scale * np.where(ok, dw[t], 0), 0)
        at, q, h = ids[t][ok], q[ok], h[ok]
        with np.errstate(over="ignore"):
            rest = 1 / (1 + np.exp(z[t][at])) if score == "sigmoid" else np.ones(len(at))  # 1 - s
        dot, mag = (h * q).sum(), np.abs(h * q).sum()
        if score == "sigmoid" and not renorm:
            dot = mag = 0.0
        if score == "softmax" and not renorm:
            dz[t], size[t] = -s[t] * dot, s[t] * mag
            np.add.at(dz[t], at, h * q)
            np.add.at(size[t], at, np.abs(h * q))
        else:
            np.add.at(dz[t], at, q * rest * (h - dot))
            np.add.at(size[t], at, q * rest * (np.abs(h) + mag))
    return dz, size


def bias_balance(counts, bias, rate):
    """fp32, [L][E]."""
    out = bias.copy()
    for l in range(len(bias)):
        on = bias[l] > -np.inf
        n, total = int(on.sum()), int(counts[l][on].astype(np.int64).sum())
        step = np.sign(total - n * counts[l].astype(np.int64)).astype(np.float32)
        out[l] = np.where(on, bias[l] + np.float32(rate) * step, bias[l])
    return out


def lora(x, a, b, ids, ranks=None, scale=None, base=None):
    """(y, size): in double, and the sum of the magnitudes of the terms."""
    T, N = len(x), b.shape[1]
    y = np.zeros((T, N)) if base is None else base.astype(np.float64)
    size = np.abs(y)
    for t in range(T):
        i = int(ids[t])
        if not 0 <= i < len(a):
            continue
        r = a.shape[1] if ranks is None else min(max(int(ranks[i]), 0), a.shape[1])
        f = 1.0 if scale is None else float(scale[i])
        down, up = a[i, :r].astype(np.float64), b[i, :, :r].astype(np.float64)
        xt = x[t].astype(np.float64)
        y[t] = y[t] + f * (up @ (down @ xt))
        size[t] = size[t] + abs(f) * (np.abs(up) @ (np.abs(down) @ np.abs(xt)))
    return y, size
