"""Plain float64 reference of the sparse-MLP operators, on the CPU: routing
of tokens to experts and the experts' gated MLP, each with its gradient by
its formula, written as loops over rows and experts."""
import math

import numpy as np


def scores(z, scoring):
    """Scores of one row of float64 logits."""
    with np.errstate(over="ignore", invalid="ignore"):
        if scoring == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = z.max() if not np.isnan(z).any() else math.nan
        if m == -math.inf:
            return np.zeros_like(z)
        p = np.exp(z - m)
        return p / p.sum()


def _order(keys):
    """Indices by falling key, ties to the lowest index."""
    return sorted(range(len(keys)), key=lambda j: (-keys[j], j))


def select(z, top_k, scoring="softmax", bias=None, n_group=1, topk_group=1,
           group_top=1):
    """The chosen experts of one row."""
    E = len(z)
    dead = np.isnan(z) | (z == -math.inf)
    value = scores(z, scoring) + (0.0 if bias is None else bias)
    value = np.where(dead | np.isnan(value), -math.inf, value)
    key = value if bias is not None else np.where(dead, -math.inf, z)
    allowed = range(E)
    if n_group > 1 and topk_group < n_group:
        per = E // n_group
        src = value if group_top == 2 else key
        rank = []
        for g in range(n_group):
            r = sum(sorted(src[g * per:(g + 1) * per])[::-1][:group_top])
            rank.append(-math.inf if math.isnan(r) else r)
        kept = set(_order(rank)[:topk_group])
        allowed = [j for j in range(E) if j // per in kept]
    return [j for j in _order(key) if j in set(allowed)][:top_k]


def route(z, top_k, scoring="softmax", bias=None, n_group=1, topk_group=1,
          group_top=1, renormalize=True, scale=1.0):
    """(weights [L,K], experts [L,K]) of logits z [L,E]."""
    L = z.shape[0]
    w = np.zeros((L, top_k))
    e = np.zeros((L, top_k), dtype=np.int64)
    for i in range(L):
        e[i] = select(z[i], top_k, scoring, bias, n_group, topk_group,
                      group_top)
        w[i] = weights_of(z[i], e[i], scoring, renormalize, scale)
    return w, e


def weights_of(z, chosen, scoring, renormalize, scale):
    p = scores(z, scoring)[chosen]
    if renormalize:
        t = p.sum()
        p = np.zeros_like(p) if t == 0 else p / t
    return scale * p


def route_grad(z, experts, dw, scoring, renormalize, scale):
    """dlogits [L,E] by the formulas."""
    dz = np.zeros_like(z)
    for i in range(z.shape[0]):
        s = scores(z[i], scoring)
        p = s[experts[i]]
        u = scale * dw[i]
        t = p.sum()
        if renormalize:
            q = np.zeros_like(p) if t == 0 else p / t
            slope = 1.0 if scoring == "softmax" else 1.0 - p
            dz[i, experts[i]] = q * slope * (u - (u * q).sum())
        elif scoring == "softmax":
            ds = np.zeros_like(s)
            ds[experts[i]] = u
            dz[i] = s * (ds - (u * p).sum())
        else:
            dz[i, experts[i]] = p * (1.0 - p) * u
    return dz


def experts_mlp(x, Wg, Wu, Wd, w, experts, dy=None):
    """y, and with dy also (dx, dWg, dWu, dWd, dweights), all float64. Slots
    whose expert is outside [0, E) are dropped."""
    L, K = experts.shape
    y = np.zeros_like(x)
    grads = [np.zeros_like(t) for t in (x, Wg, Wu, Wd, w)]
    for i in range(Wg.shape[0]):
        t, k = np.nonzero(experts == i)
        if not len(t):
            continue
        r, wt = x[t], w[t, k][:, None]
        g, u = r @ Wg[i].T, r @ Wu[i].T
        with np.errstate(over="ignore"):
            sg = 1.0 / (1.0 + np.exp(-g))
        a = g * sg * u
        np.add.at(y, t, wt * (a @ Wd[i].T))
        if dy is None:
            continue
        da = dy[t] @ Wd[i]
        grads[4][t, k] = (da * a).sum(1)
        da = wt * da
        dg = da * u * sg * (1.0 + g * (1.0 - sg))
        du = da * g * sg
        np.add.at(grads[0], t, dg @ Wg[i] + du @ Wu[i])
        grads[1][i] = dg.T @ r
        grads[2][i] = du.T @ r
        grads[3][i] = dy[t].T @ (wt * a)
    return y if dy is None else (y, *grads)
