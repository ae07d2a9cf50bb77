"""Log-probabilities, policy and preference losses and routing in FP64 numpy, row
by row, straight from their definitions in include/gbdt.h."""
import math

import numpy as np


def row(x, a, T):
    """(counts, logp, 1 - p_a, gradient of logp, (m, o)) of one row."""
    C = len(x)
    nothing = (False, 0.0, 0.0, np.zeros(C), (0.0, 0.0))
    if a < 0 or a >= C or np.all(x == -np.inf):
        return nothing
    others = np.delete(x, a)
    with np.errstate(all="ignore"):
        m = np.max(others) if C > 1 else -np.inf  # (NaN where there is one)
        if np.isnan(x).any() or np.isposinf(x).any():
            return True, np.nan, np.nan, np.full(C, np.nan), (np.nan, np.nan)
        v = np.exp((x - m) / T) if m > -np.inf else np.zeros(C)
        v[a] = 0.0
        o = v.sum()
        if o == 0.0:
            return True, 0.0, 0.0, np.zeros(C), (m, 0.0)
        if x[a] == -np.inf:
            return True, -np.inf, 1.0, np.zeros(C), (m, o)
        L = (m - x[a]) / T + math.log(o)
        logp = -(max(L, 0.0) + math.log1p(math.exp(-abs(L))))
        against = 1.0 / (1.0 + math.exp(-L)) if L > 0 else math.exp(L) / (1.0 + math.exp(L))
        g = -against * v / o / T
        g[a] = against / T
        return True, logp, against, g, (m, o)


def policy(logp, old, ref, A, low, high, kl):
    """(loss, slope) of a row that counts."""
    with np.errstate(all="ignore"):
        r = np.exp(np.float64(logp) - np.float64(old))
        by = r * A if A != 0 else 0.0
        cut = min(max(r, 1 - low), 1 + high) * A if A != 0 else 0.0
        loss = -(by if by < cut or by != by else cut)
        slope = 0.0 if (A > 0 and r > 1 + high) or (A < 0 and r < 1 - low) else -by
        if ref is not None and kl > 0:
            y = np.float64(ref) - logp
            loss += kl * (np.inf if np.isinf(y) else np.expm1(y) - y if abs(y) > 1e-3 else
                          y * y * (0.5 + y / 6 + y * y / 24 + y ** 3 / 120))
            slope -= kl * np.expm1(y)
        return loss, slope


def softplus(z):
    return max(z, 0.0) + math.log1p(math.exp(-abs(z))) if z == z else np.nan


def pair(won, lost, smoothing):
    """(loss, slope in won - lost)"""
    with np.errstate(all="ignore"):
        z = np.float64(won) - np.float64(lost)
        if z != z:
            return np.nan, np.nan
        loss = (1 - smoothing) * softplus(-z) + (smoothing * softplus(z) if smoothing else 0.0)
        up = 1 / (1 + np.exp(-z))
        down = 1 / (1 + np.exp(z))
        return loss, smoothing * up - (1 - smoothing) * down


def values(x, sigmoid):
    x = np.where(np.isnan(x), -np.inf, x)
    with np.errstate(all="ignore"):
        if sigmoid:
            e = np.exp(-np.abs(x))
            return np.where(x < 0, e / (1 + e), 1 / (1 + e))
        x = np.minimum(x, np.finfo(np.float32).max)
        m = x.max()
        if m == -np.inf:
            return np.zeros(len(x))
        e = np.exp(x - m)
        return e / e.sum()


def route(x, r, bias):
    """(classes, weights) of one row; r: a Routing."""
    E, G = len(x), r.n_groups
    x = np.where(np.isnan(x), -np.inf, x)
    s = values(x, r.score)
    v = x + 0.0
    if bias is not None or (G > 1 and r.group_top == 2):
        with np.errstate(all="ignore"):
            v = s + (0.0 if bias is None else bias.astype(np.float64))
        v = np.where((x == -np.inf) | np.isnan(v), -np.inf, v)
    if G > 1:
        size = E // G
        ranks = []
        for g in range(G):
            part = np.sort(v[g * size:(g + 1) * size])[::-1]
            rank = part[0]
            if r.group_top == 2 and size > 1 and part[1] > -np.inf:
                rank = part[0] + part[1]
            ranks.append(rank)
        order = np.lexsort((np.arange(G), -np.array(ranks)))[: r.groups_kept]
        for g in range(G):
            if g not in order:
                v[g * size:(g + 1) * size] = -np.inf
    order = np.lexsort((np.arange(E), -v))[: r.k]
    chosen = np.array([c if v[c] > -np.inf else -1 for c in order], dtype=np.int32)
    w = np.array([s[c] if c >= 0 else 0.0 for c in chosen])
    if r.renormalise:
        if not r.score and (chosen >= 0).any():
            # the same quotient where the values themselves underflow
            z = np.minimum(x[chosen[chosen >= 0]], np.finfo(np.float32).max)
            w[chosen >= 0] = np.exp(z - z.max())
        total = w.sum()
        w = w / total if total > 0 else np.zeros(r.k)
    return chosen, r.scale * w


def route_grad(x, r, chosen, dw):
    """The Jacobian of the weights, and with it the gradient."""
    E = len(x)
    s = values(x, r.score)
    ok = (chosen >= 0) & (chosen < E)
    c = chosen[ok]
    d = dw[ok].astype(np.float64)
    with np.errstate(all="ignore"):
        if r.score:
            J = np.zeros((len(c), E))
            J[np.arange(len(c)), c] = s[c] * (1 - s[c])
        else:
            J = -np.outer(s[c], s)
            J[np.arange(len(c)), c] += s[c]
        if r.renormalise:
            total = s[c].sum()
            if total == 0:
                return np.zeros(E)
            J = J / total - np.outer(s[c], J.sum(0)) / total ** 2
        return r.scale * (d @ J)
