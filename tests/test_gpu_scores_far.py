"""Distillation of students that are certain: the largest score lies gaps of up
to thousands of temperatures above the classes outside the record, where
exponentials taken against the row's maximum underflow.  The reference is in
logarithms, so it has no such limit.

Tolerances.  The loss's and the gradient's exponentials of the classes outside
are FP32: a difference, a factor and a product, each off by half a step
(2^-24), move the exponent by 3 * 2^-24 times its size, and the exponential is
off by one step (2^-23).  With D the spread of the classes outside over T (at
most 40: e^-40 adds nothing a float would show) a sum of them is off by
(3 D + 2) 2^-24; six more half steps are for the results' own roundings.  A
gradient from stored statistics may take the exponent from the row's maximum,
as long as the sums fit FP32 (gaps up to 88): D + 88 instead of D there.
Products of two such values are off by twice that, results in a smaller type
by half its step.
"""
import numpy as np
import pytest
import torch

import scores_ref as ref

DEV = "cuda"
COLD = float(np.float32(0.2))  # a temperature that FP32 holds
GAPS = [0.0, 10.0, 50.0, 80.0, 86.0, 88.0, 90.0, 95.0, 100.0, 110.0, 120.0, 300.0, 700.0, 1000.0, 2000.0]


def log_sum(z):
    """log sum exp of the rows; -inf where nothing is left."""
    m = z.max(1, keepdims=True)
    with np.errstate(divide="ignore"):
        return (np.where(np.isneginf(m), 0.0, m) +
                np.log(np.exp(z - np.where(np.isneginf(m), 0.0, m)).sum(1, keepdims=True)))[:, 0]


def reference(x, tv, tc, tr, T, weight):
    """(loss, gradient, q, p, r q_c / q_r) of rows without NaN, in FP64."""
    n, C = x.shape
    inside = np.zeros((n, C), dtype=bool)
    t = np.full((n, C), -np.inf)
    for i in range(n):
        named = tc[i] >= 0
        inside[i, tc[i][named]] = True
        t[i, tc[i][named]] = tv[i][named]
    z = (x - x.max(1, keepdims=True)) / T
    log_q = z - log_sum(z)[:, None]
    log_qr = log_sum(np.where(inside, -np.inf, log_q))
    log_t = t / T - log_sum(t / T)[:, None]
    r, weight = tr.astype(np.float64), weight.astype(np.float64)
    p = (1.0 - r)[:, None] * np.exp(log_t)
    with np.errstate(divide="ignore", invalid="ignore"):
        loss = np.where(p > 0, p * (np.log(p) - log_q), 0.0).sum(1)
        loss = loss + np.where(r > 0, r * (np.log(r) - log_qr), 0.0)
        away = r[:, None] * np.exp(np.where(inside | np.isneginf(log_q), -np.inf, log_q - log_qr[:, None]))
    q = np.exp(log_q)
    grad = (q - p - away) * (weight[:, None] * T)
    return T * T * loss, grad, q, p, away


def far_rows(n, C, dtype, T, seed):
    """Rows whose first listed class is a gap above the classes outside: some
    with half of these masked, some with one of them 20 T above the others."""
    g = np.random.default_rng(seed)
    k = max(1, min(5, C - 2))
    x = g.normal(0.0, T, (n, C))
    tc = np.full((n, k + 1), -1, dtype=np.int32)  # (an entry of padding)
    tv = np.zeros((n, k + 1), dtype=np.float32)
    for i in range(n):
        cls = g.choice(C, k, replace=False)
        out = np.ones(C, dtype=bool)
        out[cls] = False
        if i % 4 == 1:
            x[i, (g.random(C) < 0.5) & out & (np.arange(C) != np.flatnonzero(out)[0])] = -np.inf
        if i % 4 == 2:
            x[i, out] = -20.0 * T
            x[i, np.flatnonzero(out)[-1]] = 0.0
        x[i, cls[0]] = x[i, out].max() + GAPS[i % len(GAPS)] * T
        tc[i, 1:] = cls
        tv[i, 1:] = g.normal(0.0, T, k)
        tv[i, 1] = 3.0 * T
    tr = np.array([0.01, 0.1, 1.0, 0.5, 0.0])[np.arange(n) // len(GAPS) % 5 if n > 3 * len(GAPS) else
                                               np.arange(n) % 5].astype(np.float32)
    t = torch.from_numpy(x).to(ref.TYPES[dtype])
    weight = np.array([1.0, 0.25, -2.0, 3.0], dtype=np.float32)[np.arange(n) % 4]
    return t, t.double().numpy(), tv, tc, tr, weight


def spread(x, tc, T):
    """The finite scores outside the record: their range over T, row by row."""
    out = np.isfinite(x)
    for i in range(len(x)):
        out[i, tc[i][tc[i] >= 0]] = False
    hi = np.where(out, x, -np.inf).max(1)
    return np.minimum(40.0, (hi - np.where(out, x, np.inf).min(1)) / T)


@pytest.mark.parametrize("T", [COLD, 1.0, 2.0])
def test_reference(T):
    """The reference in logarithms against the one of sums where these do not
    underflow, and its gradient against central differences at any gap: their
    error is h^2 times a third derivative below 1 / T, and the loss's own
    rounding over h."""
    _, x, tv, tc, tr, weight = far_rows(30, 12, "f32", T, 3)
    loss, grad, _, _, _ = reference(x, tv, tc, tr, T, weight)
    for i in range(len(x)):
        if GAPS[i % len(GAPS)] <= 300.0:
            wl, wg, _ = ref.distill(x[i], tv[i], tc[i], tr[i], T, float(weight[i]))
            assert abs(loss[i] - wl) <= 1e-11 * (1.0 + abs(wl))
            assert np.all(np.abs(grad[i] - wg) <= 1e-11 * (1.0 + np.abs(wg)))
        h = 1e-4 * T
        for c in np.flatnonzero(np.isfinite(x[i])):
            up, down = x[i:i + 1].copy(), x[i:i + 1].copy()
            up[0, c] += h
            down[0, c] -= h
            s = slice(i, i + 1)
            d = (reference(up, tv[s], tc[s], tr[s], T, weight[s])[0][0] -
                 reference(down, tv[s], tc[s], tr[s], T, weight[s])[0][0]) / (2 * h)
            bound = (h / T) ** 2 * T + 1e-15 * (1.0 + abs(loss[i])) / h
            assert abs(d * weight[i] - grad[i, c]) <= abs(weight[i]) * bound * 4, (i, c)


# rows by one thread; four rows a wave; a wave, 256 and 1,024 threads a row; rows split over workgroups
SHAPES = [(75, 7), (75, 15), (75, 30), (75, 60), (75, 100), (75, 1000), (75, 9001), (30, 70001), (150, 70001)]


def on_device(case):
    import histogram_split_finding_amd as g
    t, x, tv, tc, tr, weight = case
    dev = [torch.from_numpy(a).to(DEV) for a in (tv, tc, tr, weight)]
    xd = ref.place(t)
    return (g, xd, dev, g.new_workspace(g.gbdt_scores_workspace_bytes(*x.shape)),
            torch.full((x.shape[0],), 7.0, device=DEV), torch.full((x.shape[0], 3), 7.0, device=DEV),
            torch.full_like(xd, 7.0))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [COLD, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,C", SHAPES)
def test_loss(n, C, dtype, T):
    print("far loss: %d x %d %s T=%s" % (n, C, dtype, T), flush=True)
    case = far_rows(n, C, dtype, T, C)
    _, x, tv, tc, tr, weight = case
    want = reference(x, tv, tc, tr, T, weight)[0]
    g, xd, (tvd, tcd, trd, wd), ws, loss, stats, grad = on_device(case)
    tol = T * T * (3 * spread(x, tc, T) + 8) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want)
    g.gbdt_distill_loss(xd, tvd, tcd, trd, T, loss, stats, ws)
    got = loss.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), (got - want, tol)
    loss.fill_(7.0)
    g.gbdt_distill_step(xd, tvd, tcd, trd, T, wd, loss, grad, ws)
    got = loss.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol), (got - want, tol)
    assert g.gbdt_read_error(ws) == 0


def check_grad(got, case, T, dtype, beyond):
    _, x, tv, tc, tr, weight = case
    _, want, q, p, away = reference(x, tv, tc, tr, T, weight)
    e = ((3 * (spread(x, tc, T) + beyond) + 8) * 2.0 ** -24)[:, None]
    tiny = {"f32": 1e-36, "bf16": 1e-36, "f16": 2.0 ** -25}[dtype]
    tol = np.abs(weight)[:, None] * T * (q + p + away) * 2 * e + ref.EPS[dtype] / 2 * np.abs(want) + tiny
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), [(GAPS[i % len(GAPS)], tr[i], got[i, c], want[i, c]) for i, c in np.argwhere(bad)[:5]]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [COLD, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,C", SHAPES)
def test_step_gradient(n, C, dtype, T):
    print("far step: %d x %d %s T=%s" % (n, C, dtype, T), flush=True)
    case = far_rows(n, C, dtype, T, C)
    g, xd, (tvd, tcd, trd, wd), ws, loss, stats, grad = on_device(case)
    g.gbdt_distill_step(xd, tvd, tcd, trd, T, wd, loss, grad, ws)
    check_grad(grad, case, T, dtype, 0.0)
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("T", [COLD, 1.0])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,C", SHAPES)
def test_gradient_from_statistics(n, C, dtype, T):
    print("far gradient: %d x %d %s T=%s" % (n, C, dtype, T), flush=True)
    case = far_rows(n, C, dtype, T, C)
    g, xd, (tvd, tcd, trd, wd), ws, loss, stats, grad = on_device(case)
    g.gbdt_distill_loss(xd, tvd, tcd, trd, T, loss, stats, ws)
    g.gbdt_distill_grad(xd, tvd, tcd, trd, T, stats, wd, grad, ws)
    check_grad(grad, case, T, dtype, 88.0)
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [7, 60, 1000, 9001, 70001])
def test_rows_of_nan(C, dtype):
    """Loss and both gradients: NaN for rows with a NaN or +inf score, a row of
    NaN alone among them, 0 for masked rows and rows of weight 0."""
    print("NaN rows: C=%d %s" % (C, dtype), flush=True)
    n = 12
    case = far_rows(n, C, dtype, 1.0, C + 1)
    t, x, tv, tc, tr, weight = case
    listed = tc[:, 1]
    outside = [int(np.setdiff1d(np.arange(C), tc[i])[0]) for i in range(n)]
    tr[:] = 0.25
    t[0] = float("nan")
    t[1, int(listed[1])] = float("nan")
    t[2, outside[2]] = float("nan")
    t[3, int(listed[3])] = float("inf")
    t[4, outside[4]] = float("inf")
    t[5], weight[5] = float("nan"), 0.0
    t[6] = float("-inf")
    t[7, int(listed[7])], weight[7] = float("inf"), 0.0
    g, xd, (tvd, tcd, trd, wd), ws, loss, stats, grad = on_device(case)
    step_loss, step_grad = torch.full_like(loss, 7.0), torch.full_like(grad, 7.0)
    g.gbdt_distill_loss(xd, tvd, tcd, trd, 1.0, loss, stats, ws)
    g.gbdt_distill_grad(xd, tvd, tcd, trd, 1.0, stats, wd, grad, ws)
    g.gbdt_distill_step(xd, tvd, tcd, trd, 1.0, wd, step_loss, step_grad, ws)
    assert g.gbdt_read_error(ws) == 0
    for l, d in ((loss, grad), (step_loss, step_grad)):
        l, d = l.cpu(), d.cpu()
        for i in (0, 1, 2, 3, 4, 5, 7):
            assert bool(l[i].isnan()), i
        for i in (0, 1, 2, 3, 4):
            assert bool(d[i].isnan().any()), i
        assert l[6].item() == 0.0
        for i in (5, 6, 7):
            assert bool((d[i] == 0).all()), i
        assert bool(l[8:].isfinite().all()) and bool(d[8:].isfinite().all())
