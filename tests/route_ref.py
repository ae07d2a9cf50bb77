"""The routing weights' gradient in extended precision, row by row, in a form whose
terms do not cancel: with s the experts' values, J the chosen experts and w_j = s_j /
sum_J s,
  softmax:                  dx_j = scale s_j (sum_J s_i (d_j - d_i) + d_j R),
                            dx_c = -scale s_c sum_J s_i d_i outside J,
  softmax, renormalised:    dx_j = scale w_j sum_J w_i (d_j - d_i),
  sigmoid:                  dx_j = scale s(x_j) s(-x_j) d_j,
  sigmoid, renormalised:    dx_j = scale w_j s(-x_j) sum_J w_i (d_j - d_i),
R the softmax mass outside J."""
import numpy as np

LONG = np.longdouble
MOST = LONG(np.finfo(np.float32).max)


def sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x < 0, e / (1 + e), 1 / (1 + e))


def parts(x, r, chosen):
    """(experts, their s or w, R, softmax values of all experts) of one row."""
    x = np.where(np.isnan(x), -np.inf, x).astype(LONG)
    c = chosen[(chosen >= 0) & (chosen < len(x))]
    none = np.zeros(len(x), dtype=LONG)
    with np.errstate(all="ignore"):
        if r.score:
            s = sigmoid(x)[c]
            return (c, s / s.sum() if r.renormalise and s.sum() > 0 else s), LONG(0), none
        x = np.minimum(x, MOST)
        if r.renormalise:
            e = np.exp(x[c] - x[c].max()) if len(c) and x[c].max() > -np.inf else none[c]
            return (c, e / e.sum() if len(c) and e.sum() > 0 else e), LONG(0), none
        if x.max() == -np.inf:
            return (c, none[c]), LONG(0), none
        e = np.exp(x - x.max())
        out = np.ones(len(x), dtype=bool)
        out[c] = False
        return (c, e[c] / e.sum()), e[out].sum() / e.sum(), e / e.sum()


def grad(x, r, chosen, dw):
    """The gradient, and what its terms add up to at most (for tolerances)."""
    (c, s), R, every = parts(x, r, chosen)
    d = dw[(chosen >= 0) & (chosen < len(x))].astype(LONG)
    away = sigmoid(-np.where(np.isnan(x), -np.inf, x).astype(LONG))[c] if r.score else LONG(1)
    if r.score and not r.renormalise:
        mine = size = s * away * d
    else:
        mine = s * away * ((s[None] * (d[:, None] - d[None])).sum(1) + d * R)
        size = s * away * (np.abs(d) + (s * np.abs(d)).sum())
    g, b = -every * (s * d).sum(), every * (s * np.abs(d)).sum()
    g[c], b[c] = mine, np.abs(size)
    return np.float64(r.scale) * g, abs(np.float64(r.scale)) * b
