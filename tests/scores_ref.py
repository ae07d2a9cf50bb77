"""The operators on rows of class scores in FP64 numpy, row by row, straight
from their definitions in include/gbdt.h, and inputs for their tests."""
import math

import numpy as np
import torch

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -23, "bf16": 2.0 ** -7, "f16": 2.0 ** -10}  # torch.finfo(t).eps


def order(x):
    """Classes of a row, score descending, class ascending; NaN as -inf."""
    v = np.where(np.isnan(x), -np.inf, x) + 0.0
    return np.lexsort((np.arange(len(v)), -v)), v


def weights(v, T):
    """exp((v - max v) / T); a +inf score takes all the weight, -inf none."""
    m = v.max()
    if m == -np.inf:
        return np.zeros(len(v))
    if m == np.inf:
        return (v == np.inf).astype(np.float64)
    with np.errstate(over="ignore", under="ignore"):
        return np.exp((v - m) / T)


def top_scores(x, k, T):
    o, v = order(x)
    take = [c for c in o[:k] if v[c] > -np.inf]
    w = weights(v, T)
    inside = np.zeros(len(v), dtype=bool)
    inside[take] = True
    total = w.sum()
    rest = w[~inside].sum() / total if total > 0 else 0.0
    values = np.full(k, -np.inf)
    classes = np.full(k, -1, dtype=np.int32)
    values[: len(take)] = v[take]
    classes[: len(take)] = take
    return values, classes, rest


def distill(x, tv, tc, rest, T, weight):
    """(loss, gradient, (max, sum in S, sum outside S)) of one row."""
    C = len(x)
    named = (tc >= 0) & (tc < C)
    cls = tc[named]
    t = tv[named].astype(np.float64)
    r = 0.0 if rest is None else min(max(float(rest), 0.0), 1.0)
    inside = np.zeros(C, dtype=bool)
    inside[cls] = True
    has = bool(np.any(~(t == -np.inf)))
    masked = bool(np.all(x == -np.inf))
    m = np.nanmax(x) if not np.all(np.isnan(x)) else np.nan
    with np.errstate(all="ignore"):
        w = np.zeros(C) if masked else np.exp((x - m) / T)
        stats = (m, w[inside].sum(), w[~inside].sum())
        if not has or masked:
            return 0.0, np.zeros(C), stats
        e = np.exp((t - t.max()) / T)
        p = (1.0 - r) * e / e.sum()
        s = w.sum()
        q = w / s
        qr = w[~inside].sum() / s
        loss = 0.0
        for j in range(len(cls)):
            if p[j] != 0:
                # log q_j as it is, not through a q_j that has underflowed
                loss += p[j] * (math.log(p[j]) - ((x[cls[j]] - m) / T - math.log(s))) if p[j] == p[j] else np.nan
        if r > 0:
            loss += r * (math.log(r) - (math.log(qr) if qr > 0 else -np.inf)) if qr == qr else np.nan
        g = q * (1.0 - r / qr) if qr > 0 else (np.zeros(C) if qr == 0 else np.full(C, np.nan))
        g[inside] = q[inside]
        g[cls] -= p
        g = g * (weight * T) if weight != 0 else np.zeros(C)
    return T * T * loss, g, stats


def sample(x, u, T, top_k, top_p, min_p):
    o, v = order(x)
    if v[o[0]] == -np.inf:
        return -1, -np.inf
    if T == 0:
        return int(o[0]), 0.0
    w = weights(v, T)[o]
    n = len(v) if top_k <= 0 else min(top_k, len(v))
    run = np.cumsum(w[:n])
    if top_p < 1:
        n = min(n, int(np.searchsorted(run, top_p * run[-1], side="left")) + 1)
    keep = max(1, int(np.sum((w[:n] >= min_p) & (w[:n] > 0))))
    run = run[:keep]
    j = min(int(np.searchsorted(run, u * run[-1], side="right")), keep - 1)
    return int(o[j]), math.log(w[j] / run[-1])


def rows(n, C, dtype, seed, spread=2.0, pad=0):
    """Rows of a wide bulk with a few high scores, rounded to the type: the
    device tensor (rows `pad` elements further apart) and its values."""
    g = np.random.default_rng(seed)
    x = g.normal(0.0, spread, (n, C))
    hot = min(8, C // 4)
    for i in range(n):
        at = g.choice(C, hot, replace=False)
        x[i, at] += 4.0 + 3.0 * np.abs(g.normal(0.0, 1.0, hot))
    t = torch.from_numpy(x).to(TYPES[dtype])
    return place(t, pad), t.double().numpy()


def place(t, pad=0, device="cuda"):
    out = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype)[:, : t.shape[1]]
    out.copy_(t)
    if pad == 0:
        return out.contiguous().to(device)
    buf = torch.full((t.shape[0] * (t.shape[1] + pad),), 7.0, dtype=t.dtype, device=device)
    view = buf.as_strided((t.shape[0], t.shape[1]), (t.shape[1] + pad, 1))
    view.copy_(t.to(device))
    return view


def records(x, k, seed, T, rest=True, holes=True):
    """Teacher records of rows near x: values, classes (some padding entries,
    entries not in order), rest."""
    g = np.random.default_rng(seed + 1)
    n, C = x.shape
    t = np.where(np.isfinite(x), x, 0.0) + g.normal(0.0, 0.7, x.shape)
    tv = np.zeros((n, k), dtype=np.float32)
    tc = np.full((n, k), -1, dtype=np.int32)
    tr = np.zeros(n, dtype=np.float32)
    for i in range(n):
        kk = min(k, C)
        top = np.argsort(-t[i], kind="stable")[:kk]
        top = top[g.permutation(kk)]
        if holes and kk > 2:
            top = top[: kk - 1]
        tv[i, : len(top)] = t[i, top]
        tc[i, : len(top)] = top
        w = np.exp((t[i] - t[i].max()) / T)
        out = np.ones(C, dtype=bool)
        out[top] = False
        tr[i] = w[out].sum() / w.sum()
    return tv, tc, (tr if rest else None)
