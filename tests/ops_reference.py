"""Plain 64-bit references of moe_linear_q4, moe_sample and moe_balance_loss (numpy only)."""
import numpy as np


def codes(wq):
    """uint8 [N][K/2] -> codes [N][K]: byte j of a 16-byte block holds input j low, input j + 16 high."""
    n, half = wq.shape
    b = wq.reshape(n, half // 16, 16)
    return np.concatenate([b & 15, b >> 4], axis=2).reshape(n, 2 * half)


def linear_q4(x, wq, scales, group, bias=None):
    """(y, bound): y in double, and the sum of |x| * scale * (code + 8), the size every partial sum stays below."""
    q = codes(wq).astype(np.float64)
    d = np.repeat(scales.astype(np.float64), group, axis=1)
    y = x.astype(np.float64) @ ((q - 8) * d).T
    size = np.abs(x.astype(np.float64)) @ ((q + 8) * np.abs(d)).T
    if bias is not None:
        y, size = y + bias, size + np.abs(bias)
    return y, size


def sample_row(l, u, temperature=1.0, min_p=0.0, top_k=0, top_p=1.0):
    """(id, prob, ids kept) of one row; l in double."""
    cand = np.nonzero(l > -np.inf)[0]
    if not len(cand):
        return -1, 0.0, cand
    order = cand[np.argsort(-l[cand], kind="stable")]
    if not temperature > 0:
        return int(order[0]), 1.0, order[:1]
    top = l[order[0]]
    with np.errstate(invalid="ignore", over="ignore"):
        w = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / temperature))
    if min_p > 0:
        keep = int(np.sum(w >= min(min_p, 1.0)))
        order, w = order[:keep], w[:keep]
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        keep = max(1, int(np.sum(before < max(top_p, 0.0) * w.sum())))
        order, w = order[:keep], w[:keep]
    by_id = np.argsort(order)
    ids, w = order[by_id], w[by_id]
    u = 0.0 if not u > 0 else u
    cum = np.cumsum(w)
    at = int(np.searchsorted(cum, u * cum[-1], side="right"))
    at = min(at, int(np.nonzero(w > 0)[0][-1]))
    return int(ids[at]), float(w[at] / cum[-1]), ids


def balance(z, ids, mask=None):
    """Outputs of moe_balance_loss in double (z: finite, -inf or NaN)."""
    T, E = z.shape
    z = z.astype(np.float64)
    live = np.ones(T, bool) if mask is None else mask != 0
    live = live & ~np.all(z == -np.inf, axis=1)
    p, lse = np.zeros((T, E)), np.zeros(T)
    for t in np.nonzero(live)[0]:
        m = z[t].max()
        e = np.exp(z[t] - m)
        p[t], lse[t] = e / e.sum(), m + np.log(e.sum())
    picked = ids[live].reshape(-1)
    picked = picked[(picked >= 0) & (picked < E)]
    counts = np.bincount(picked, minlength=E)
    n, picks = int(live.sum()), int(counts.sum())
    share = p.sum(axis=0) / max(n, 1)
    loss = np.array([E * float((counts / max(picks, 1)) @ share), float((lse ** 2).sum()) / max(n, 1)])
    return dict(counts=counts, totals=np.array([n, picks]), share=share, lse=lse, loss=loss, p=p, live=live)


def balance_grad(z, ids, dloss, mask=None):
    o = balance(z, ids, mask)
    n, picks = int(o["totals"][0]), int(o["totals"][1])
    E = z.shape[1]
    f = o["counts"] / max(picks, 1)
    p = o["p"]
    d = p * (dloss[0] * E * (f[None] - (p @ f)[:, None]) + 2 * dloss[1] * o["lse"][:, None]) / max(n, 1)
    return np.where(o["live"][:, None], d, 0.0)
