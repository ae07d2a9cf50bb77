"""Log-probabilities, policy and preference losses and their gradients on the GPU
against the FP64 reference in learn_ref.py.

Tolerances.  A score's FP32 exponential exp2((x - m) c): the difference, c and
the product are each off by half a step (2^-24 relative), which moves the exponent
by 3 2^-24 D with D = |x - m| / T, and the exponential itself by a step (2^-23): a sum
of them, with D at most 40 where it matters, is off by e = (3 D + 6) 2^-24 with the
sums' own roundings.  The logarithm of the odds is then off by e, logp by
(1 - p_a) e, the gradient at the class by e relative (and one more half step each
for o as FP32 statistics, the product and the result); elsewhere its own FP32
exponential adds (3 D_c + 2) 2^-24.  A slope's error follows logp's: |r A| + kl e^y
times it; which side of the clip a ratio is on is decided in FP64.  Results below
FP32's normal numbers, 2^-126 times the slope, may be 0.
"""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import learn_ref as lref
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

SIZES = [1, 2, 7, 8, 9, 16, 17, 32, 33, 40, 64, 65, 100, 129, 257, 300, 513, 1000, 1024, 1025, 2048, 2049, 4099, 8193,
         20011, 40001, 70001]
STEP = 2.0 ** -24
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}


def to_dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def workspace(x, pref=False):
    size = g.gbdt_preference_workspace_bytes if pref else g.gbdt_scores_workspace_bytes
    return g.new_workspace(size(x.shape[0], x.shape[1]))


def spread(x, T):
    """e, and D_c of each class against the largest other."""
    fin = x[np.isfinite(x)]
    D = min(40.0, (fin.max() - fin.min()) / T) if len(fin) else 0.0
    e = (3 * D + 6) * STEP
    with np.errstate(all="ignore"):
        Dc = np.where(np.isfinite(x), np.abs(x - (fin.max() if len(fin) else 0.0)) / T, 0.0)
    return e, Dc


def same(a, b, tol):
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    with np.errstate(all="ignore"):
        ok = (a == b) | (np.isnan(a) & np.isnan(b)) | (np.abs(a - b) <= tol)
    return bool(np.all(ok))


def draw_classes(xh, seed, ignored=0.2):
    """A class of each row, likely ones and any, some padding."""
    r = np.random.default_rng(seed)
    n, C = xh.shape
    cls = r.integers(0, C, n)
    best = np.argmax(np.where(np.isnan(xh), -np.inf, xh), 1)
    cls = np.where(r.random(n) < 0.5, best, cls)
    cls[r.random(n) < ignored] = -1
    return cls.astype(np.int32)


def grad_tol(want, x, a, T, dtype, e, slope, dslope):
    """Of a row's gradient slope * dlogp/dx."""
    _, Dc = spread(x, T)
    rel = (3 * Dc + 8) * STEP + 2 * e + ref.EPS[dtype] / 2
    if 0 <= a < len(x):
        rel[a] = 6 * STEP + 2 * e + ref.EPS[dtype] / 2
    # the slope's own error moves all of it
    tol = np.abs(want) * rel + TINY[dtype] * max(1.0, abs(slope) / T)
    return tol + np.abs(want) * (dslope / abs(slope) if slope else 0.0)


def buffer(n, C, pad, dtype):
    b = torch.full((n * (C + pad),), 7.0, dtype=dtype, device=DEV)
    return b, b.as_strided((n, C), (C + pad, 1))


def check_logp(x, xh, cls, T, dtype, pad=0):
    """logp, stats, and the gradient for random dlogp."""
    n, C = xh.shape
    r = np.random.default_rng(C + n)
    d = r.normal(0.0, 1.0, n).astype(np.float32)
    d[r.random(n) < 0.1] = 0.0
    ws = workspace(x)
    logp, stats = torch.full((n,), 7.0, device=DEV), torch.full((n, 2), 7.0, device=DEV)
    buf, grad = buffer(n, C, pad, x.dtype)
    cd = to_dev(cls)
    g.gbdt_class_logp(x, cd, T, logp, stats, ws)
    g.gbdt_class_logp_grad(x, cd, T, stats, to_dev(d), grad, ws)
    assert g.gbdt_read_error(ws) == 0
    if pad:
        assert bool((buf.view(n, C + pad)[:, C:] == 7.0).all())
    again = torch.full((n,), 7.0, device=DEV)
    g.gbdt_class_logp(x, cd, T, again, None, ws)
    assert torch.equal(again.nan_to_num(9.0), logp.nan_to_num(9.0))
    lp, st, gr = logp.cpu().numpy(), stats.cpu().numpy(), grad.double().cpu().numpy()
    for i in range(n):
        counts, wl, against, wg, wst = lref.row(xh[i], int(cls[i]), T)
        e, _ = spread(xh[i], T)
        tol = STEP * abs(wl) + against * e + 2.0 ** -126 if np.isfinite(wl) else 0.0
        assert same(lp[i], wl, tol), (i, lp[i], wl, tol)
        if not np.isnan(wl):
            assert st[i, 0] == np.float32(wst[0]) and same(st[i, 1], wst[1], (e + STEP) * wst[1]), (i, st[i], wst)
        want = wg * d[i] if d[i] != 0 and counts else np.zeros(C)
        tol = grad_tol(want, xh[i], int(cls[i]), T, dtype, e, float(d[i]), 0.0)
        off = np.abs(gr[i] - want)
        assert same(gr[i], want, tol), (i, np.nanmax(off / tol), int(np.nanargmax(off / tol)), cls[i])


def policy_rows(logp, seed):
    """Per-row inputs whose ratio keeps away from the clip's borders."""
    r = np.random.default_rng(seed)
    n = len(logp)
    base = np.where(np.isfinite(logp), logp, -3.0)
    old = (base + r.choice([-0.6, -0.1, 0.0, 0.05, 0.5], n) + r.uniform(-0.02, 0.02, n)).astype(np.float32)
    rf = (base + r.normal(0.0, 0.5, n)).astype(np.float32)
    A = r.normal(0.0, 1.0, n).astype(np.float32)
    A[r.random(n) < 0.1] = 0.0
    w = r.uniform(0.5, 2.0, n).astype(np.float32)
    w[r.random(n) < 0.1] = 0.0
    return old, rf, A, w


def check_policy(x, xh, cls, T, dtype, pad=0, with_ref=True, with_weight=True, low=0.2, high=0.28, kl=0.04, rows=None):
    """gbdt_policy_loss, its gradient through gbdt_class_logp_grad, and the step."""
    n, C = xh.shape
    lrows = [lref.row(xh[i], int(cls[i]), T) for i in range(n)]
    old, rf, A, w = rows if rows is not None else policy_rows(np.array([q[1] for q in lrows]), n + C)
    rf, w = (rf if with_ref else None), (w if with_weight else None)
    ws = workspace(x)
    full = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    loss, logp, dlogp, stats, loss2, logp2 = full(n), full(n), full(n), full(n, 2), full(n), full(n)
    bufs = [buffer(n, C, pad, x.dtype) for _ in range(2)]
    args = (to_dev(cls), T, to_dev(old), to_dev(rf), to_dev(A), to_dev(w), low, high, kl)
    g.gbdt_policy_loss(x, *args, loss, logp, dlogp, stats, ws)
    g.gbdt_class_logp_grad(x, args[0], T, stats, dlogp, bufs[0][1], ws)
    g.gbdt_policy_step(x, *args, loss2, logp2, bufs[1][1], ws)
    assert g.gbdt_read_error(ws) == 0
    for b, _ in bufs:
        if pad:
            assert bool((b.view(n, C + pad)[:, C:] == 7.0).all())
    got = [t.double().cpu().numpy() for t in (loss, loss2, logp, logp2, dlogp)]
    gr = [b[1].double().cpu().numpy() for b in bufs]
    for i in range(n):
        counts, wl, against, wg, _ = lrows[i]
        e, _ = spread(xh[i], T)
        weight = 1.0 if w is None else float(w[i])
        dl = (against * e if np.isfinite(wl) else 0.0) + 2.0 ** -40  # of logp, before its rounding
        loss_w, slope = lref.policy(wl, old[i], None if rf is None else rf[i], float(A[i]), low, high, kl)
        if not counts:
            loss_w = slope = 0.0
        if counts and 0 <= cls[i] < C and xh[i][cls[i]] == -np.inf:
            slope = 0.0
        slope = slope * weight if weight != 0 else 0.0
        with np.errstate(all="ignore"):
            ratio = np.exp(wl - np.float64(old[i]))
            steep = abs(ratio * A[i]) + (kl * np.exp(np.float64(rf[i]) - wl) if rf is not None else 0.0)
        steep = steep if np.isfinite(steep) else 0.0
        for l in got[:2]:
            tol = STEP * abs(loss_w) + (steep + kl) * dl + 2.0 ** -126 if np.isfinite(loss_w) else 0.0
            assert same(l[i], loss_w, tol), (i, l[i], loss_w, tol)
        for l in got[2:4]:
            assert same(l[i], wl, STEP * abs(wl) + dl + 2.0 ** -126 if np.isfinite(wl) else 0.0), (i, l[i], wl)
        dslope = abs(weight) * (steep * dl + STEP * 2.0 ** -20)
        assert same(got[4][i], slope, STEP * abs(slope) + dslope + 2.0 ** -126), (i, got[4][i], slope)
        want = wg * slope if slope != 0 else np.zeros(C)
        tol = grad_tol(want, xh[i], int(cls[i]), T, dtype, e, slope, dslope)
        for q in gr:
            off = np.abs(q[i] - want)
            assert same(q[i], want, tol), (i, np.nanmax(off / tol), cls[i], slope)


def check_pairs(x, xh, cls, T, dtype, offsets, beta, smoothing, average, pad=0, with_ref=True, with_weight=True):
    n, C = xh.shape
    P = len(offsets) // 2
    r = np.random.default_rng(n + C + P)
    lrows = [lref.row(xh[i], int(cls[i]), T) for i in range(n)]
    base = np.array([q[1] if np.isfinite(q[1]) else -3.0 for q in lrows])
    rf = (base + r.normal(0.0, 0.5, n)).astype(np.float32) if with_ref else None
    w = r.uniform(0.5, 2.0, P).astype(np.float32) if with_weight else None
    if with_weight and P > 2:
        w[1] = 0.0
    full = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    loss, rewards, loss2, rewards2 = full(P), full(P, 2), full(P), full(P, 2)
    logp, dlogp, stats = full(n), full(n), full(n, 2)
    buf, grad = buffer(n, C, pad, x.dtype)
    ws = workspace(x, True)
    args = (to_dev(cls), T, to_dev(np.array(offsets, dtype=np.int64)), to_dev(rf), to_dev(w), beta, smoothing, average)
    g.gbdt_preference_loss(x, *args, loss, rewards, logp, dlogp, stats, ws)
    g.gbdt_preference_step(x, *args, loss2, rewards2, grad, ws)
    assert g.gbdt_read_error(ws) == 0
    inside = np.zeros(n, dtype=bool)
    inside[offsets[0]:offsets[-1]] = True
    for t in (logp, dlogp, stats, grad):
        assert bool((t[to_dev(~inside)] == 7.0).all())
    if pad:
        assert bool((buf.view(n, C + pad)[:, C:] == 7.0).all())
    slope, dslope = np.zeros(n), np.zeros(n)
    lp = logp.double().cpu().numpy()
    for p in range(P):
        S, dS, per = [], [], []
        for s in (2 * p, 2 * p + 1):
            rows = [i for i in range(offsets[s], offsets[s + 1]) if lrows[i][0]]
            with np.errstate(all="ignore"):
                S.append(beta * sum(lrows[i][1] - (float(rf[i]) if rf is not None else 0.0) for i in rows))
            per.append(1.0 / len(rows) if average and rows else 1.0)
            # logp as FP32 results: its rounding, and e
            off = sum(STEP * abs(lrows[i][1]) + lrows[i][2] * spread(xh[i], T)[0] for i in rows
                      if np.isfinite(lrows[i][1]))
            dS.append(abs(beta) * off * per[-1] + 2.0 ** -40 * (1 + abs(beta)))
            S[-1] *= per[-1]
        wl, dz = lref.pair(S[0], S[1], smoothing)
        weight = 1.0 if w is None else float(w[p])
        tz = sum(dS)
        for l, rw in ((loss, rewards), (loss2, rewards2)):
            assert same(l[p].item(), wl, STEP * abs(wl) + tz + 2.0 ** -126 if np.isfinite(wl) else 0.0), (p, l[p], wl)
            for k in range(2):
                fin = np.isfinite(S[k])
                assert same(rw[p, k].item(), S[k], STEP * abs(S[k]) + dS[k] if fin else 0.0), (p, k, rw[p], S)
        for k, s in enumerate((2 * p, 2 * p + 1)):
            for i in range(offsets[s], offsets[s + 1]):
                if lrows[i][0] and np.isfinite(lrows[i][1]) and weight != 0:
                    slope[i] = weight * beta * dz * per[k] * (1 if k == 0 else -1)
                    # |d^2 loss / dz^2| is at most 1/4
                    dslope[i] = abs(weight * beta * per[k]) * (0.25 * tz + 2.0 ** -40)
    dl = dlogp.double().cpu().numpy()
    gr = grad.double().cpu().numpy()
    for i in np.flatnonzero(inside):
        assert same(dl[i], slope[i], STEP * abs(slope[i]) + dslope[i]), (i, dl[i], slope[i])
        assert same(lp[i], lrows[i][1], STEP * abs(lrows[i][1]) + spread(xh[i], T)[0] + 2.0 ** -126
                    if np.isfinite(lrows[i][1]) else 0.0), i
        want = lrows[i][3] * slope[i] if slope[i] != 0 else np.zeros(C)
        e, _ = spread(xh[i], T)
        tol = grad_tol(want, xh[i], int(cls[i]), T, dtype, e, slope[i], dslope[i])
        assert same(gr[i], want, tol), (i, np.nanmax(np.abs(gr[i] - want) / tol))


# ------------------------------------------------------------------ shapes --

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", SIZES)
def test_sizes(C, dtype):
    for n, T in ((1, 1.0), (9, 1.7)):
        say("learn: %d x %d %s" % (n, C, dtype))
        x, xh = ref.rows(n, C, dtype, 500 + C, pad=C % 4)
        cls = draw_classes(xh, C, 0.2 if n > 1 else 0.0)
        check_logp(x, xh, cls, T, dtype, pad=C % 5)
        check_policy(x, xh, cls, T, dtype, pad=C % 3, with_ref=C % 2 == 0, with_weight=n > 1)
        cuts = [0, 1, 1] if n == 1 else [1, 4, 4, 6, 8]
        check_pairs(x, xh, cls, T, dtype, cuts, 0.3, 0.1 if C % 2 else 0.0, C % 3 == 0, pad=C % 2,
                    with_ref=C % 2 == 1, with_weight=C % 4 < 2)


@pytest.mark.parametrize("C,n", [(7, 1000), (20, 517), (40, 777), (150, 300), (1000, 130), (33333, 130)])
def test_many_rows(C, n):
    say("learn, many rows: %d x %d" % (n, C))
    x, xh = ref.rows(n, C, "f32", 7)
    cls = draw_classes(xh, n)
    check_logp(x, xh, cls, 1.0, "f32")
    check_policy(x, xh, cls, 1.0, "f32")
    r = np.random.default_rng(n)
    cuts = np.sort(r.integers(0, n + 1, 2 * 20 + 1)).tolist()
    check_pairs(x, xh, cls, 1.0, "f32", cuts, 0.1, 0.05, False)
    check_pairs(x, xh, cls, 1.0, "f32", cuts, 0.1, 0.0, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [7, 60, 1000, 2049])
def test_few_rows_as_many(C, dtype):
    """The rows of a few pairs alone, and as the first of many rows: the same losses,
    rewards, statistics and gradients, and those of loss and step."""
    say("learn, few rows as many: C=%d %s" % (C, dtype))
    n, more = 300, 700
    x, xh = ref.rows(n + more, C, dtype, C)
    cls = draw_classes(xh, 4)
    cuts = np.array([0, 90, 100, 100, 290], dtype=np.int64)
    got = []
    for rows in (n, n + more):
        f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
        part = x[:rows]
        ws = workspace(part, True)
        loss, rewards, logp, dlogp, stats, grad = f(2), f(2, 2), f(rows), f(rows), f(rows, 2), torch.zeros_like(part)
        args = (to_dev(cls[:rows]), 1.0, to_dev(cuts), None, None, 0.1, 0.1, False)
        g.gbdt_preference_loss(part, *args, loss, rewards, logp, dlogp, stats, ws)
        loss2 = f(2)
        g.gbdt_preference_step(part, *args, loss2, None, grad, ws)
        assert torch.equal(loss, loss2) and g.gbdt_read_error(ws) == 0
        got.append([t.double().cpu().numpy()[:290] for t in (loss, rewards, stats[:, 0], stats[:, 1], logp, dlogp, grad)])
    # sums in another order: FP32 terms in FP64 sums, then what follows from one rounding of o
    for a, b in zip(*got):
        assert np.allclose(a, b, rtol=8 * STEP, atol=8 * STEP * np.abs(b).max())


@pytest.mark.parametrize("C,n", [(4100, (1 << 20) + 5)])
def test_more_rows_than_a_grid(C, n):
    """A second launch takes up where the first grid ends."""
    say("learn, rows of two grids: %d x %d" % (n, C))
    few, xh = ref.rows(64, C, "bf16", 9)
    x = few.repeat((n + 63) // 64, 1)[:n]
    cls = to_dev(draw_classes(xh, 1, 0.0)).repeat((n + 63) // 64)[:n].contiguous()
    ws = workspace(x)
    logp, stats = torch.zeros(n, device=DEV), torch.zeros(n, 2, device=DEV)
    g.gbdt_class_logp(x, cls, 1.0, logp, stats, ws)
    want = logp[:64].repeat((n + 63) // 64)[:n]
    assert torch.equal(logp, want) and bool((want < 0).all())
    grad = torch.empty_like(x)
    g.gbdt_class_logp_grad(x, cls, 1.0, stats, torch.ones(n, device=DEV), grad, ws)
    assert torch.equal(grad[-69:], grad[:n][(n - 69) % 64:][:69])
    assert g.gbdt_read_error(ws) == 0


def test_long_sequences():
    """More rows of a sequence than a workgroup has threads, and pairs of one row."""
    say("learn: long sequences")
    n, C = 3000, 11
    x, xh = ref.rows(n, C, "bf16", 3)
    cls = draw_classes(xh, 5)
    check_pairs(x, xh, cls, 1.0, "bf16", [0, 1300, 2700, 2701, 2702], 0.02, 0.0, False)
    check_pairs(x, xh, cls, 1.0, "bf16", [0, 1300, 2700, 2701, 2702], 0.5, 0.2, True)


# ------------------------------------------------- masks, ties, odd values --

def odd_rows(C, dtype):
    info = torch.finfo(ref.TYPES[dtype])
    r = np.random.default_rng(C)
    b = r.normal(0.0, 1.0, (14, C))
    b[0] = -np.inf                                  # nothing left
    b[1] = 0.5                                      # all equal
    b[2] = -np.inf
    b[2, C // 2] = -3.0                             # the class alone is left
    b[3] = info.min                                 # the type's lowest everywhere
    b[4, : C // 2] = -np.inf                        # half masked, the class among them
    b[5] = b[5] * 0.5
    b[5, C - 1] = 90.0                              # certain of its class
    b[6, 0] = 60.0                                  # certain of another
    b[7] = -np.inf
    b[7, [0, C - 1]] = [-2.0, 2.0]                  # two left
    b[8, 0], b[8, C - 1] = info.max, info.min       # the whole range
    b[9] *= 1e-3                                    # a narrow row
    b[10] = info.tiny * r.integers(0, 3, C)         # next to zero
    b[11] = -1000.0
    b[11, 1] = 0.0                                  # far from a certain class
    b[12] = np.sort(b[12])
    b[13, : C - 1] = -np.inf                        # the other alone is left
    cls = np.array([1, 0, C // 2, 1, 0, C - 1, 1, C - 1, 0, 0, 0, 1, C - 1, 0], dtype=np.int32)
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    return t, cls


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", [2, 7, 32, 33, 300, 2000, 5000, 9001, 33333])
def test_odd_rows(C, dtype):
    say("learn, odd rows: C=%d %s" % (C, dtype))
    t, cls = odd_rows(C, dtype)
    x, xh = ref.place(t), t.double().numpy()
    check_logp(x, xh, cls, 1.0, dtype)
    check_policy(x, xh, cls, 1.0, dtype)
    check_policy(x, xh, cls, 1.0, dtype, with_ref=False)
    cuts = [0, 3, 4, 6, 9, 12, 12]  # (a sequence with a logp of -inf is the preferred one of its pair)
    check_pairs(x, xh, cls, 1.0, dtype, cuts, 0.1, 0.0, False)
    check_pairs(x, xh, cls, 1.0, dtype, cuts, 0.1, 0.2, True)


@pytest.mark.parametrize("C", [3, 40, 700, 9001, 33333])
def test_certain_rows_keep_their_digits(C):
    """Scores from 10 to 700 temperatures above all others: 1 - p_a and logp are
    e^-10 to e^-86 (as FP32 has it) and keep their relative error."""
    gaps = [10.0, 30.0, 60.0, 80.0, 200.0, 700.0]
    say("learn, certain rows: C=%d" % C)
    r = np.random.default_rng(C)
    b = r.normal(0.0, 1.0, (len(gaps), C)).astype(np.float32)
    cls = r.integers(0, C, len(gaps)).astype(np.int32)
    for i, gap in enumerate(gaps):
        b[i, cls[i]] = np.delete(b[i], cls[i]).max() + gap
    t = torch.from_numpy(b)
    x, xh = ref.place(t), t.double().numpy()
    check_logp(x, xh, cls, 1.0, "f32")
    check_policy(x, xh, cls, 1.0, "f32")
    # the same, told from the other side: classes that are all but impossible
    cls = ((cls + 1) % C).astype(np.int32)
    check_logp(x, xh, cls, 1.0, "f32")


@pytest.mark.parametrize("C", [5, 50, 700, 9001, 33333])
def test_nan_and_inf(C):
    say("learn, NaN and inf: C=%d" % C)
    r = np.random.default_rng(C)
    b = r.normal(0.0, 1.0, (8, C))
    cls = np.full(8, 2, dtype=np.int32)
    b[0, 1] = np.nan
    b[1, 2] = np.nan
    b[2, 3] = np.inf
    b[3, 2] = np.inf
    b[4] = np.nan
    b[5, 1] = np.nan
    cls[5] = -1                      # does not count
    b[6, [0, 2]] = [np.nan, -np.inf]  # a class of probability 0: the row's gradient is 0
    t = torch.from_numpy(b).float()
    x = ref.place(t)
    n = 8
    ws = workspace(x)
    f = lambda v: torch.full((n,), v, device=DEV)  # noqa: E731
    loss, logp, grad = f(7.0), f(7.0), torch.full((n, C), 7.0, device=DEV)
    g.gbdt_policy_step(x, to_dev(cls), 1.0, f(-1.0), f(-1.0), f(1.0), None, 0.2, 0.2, 0.1, loss, logp, grad, ws)
    assert bool(loss[:5].isnan().all()) and bool(logp[:5].isnan().all()) and bool(grad[:5].isnan().all())
    assert loss[5].item() == 0.0 and logp[5].item() == 0.0 and bool((grad[5:7] == 0).all())
    assert bool(grad[7].isfinite().all()) and bool(grad[7].abs().sum() > 0)
    # a weight or a dlogp of 0 leaves the scores alone, whatever they are
    zero = f(0.0)
    g.gbdt_policy_step(x, to_dev(cls), 1.0, f(-1.0), f(-1.0), f(1.0), zero, 0.2, 0.2, 0.1, loss, logp, grad, ws)
    assert bool((grad == 0).all())
    stats = torch.zeros(n, 2, device=DEV)
    g.gbdt_class_logp(x, to_dev(cls), 1.0, logp, stats, ws)
    grad.fill_(7.0)
    g.gbdt_class_logp_grad(x, to_dev(cls), 1.0, stats, zero, grad, ws)
    assert bool((grad == 0).all())
    g.gbdt_class_logp_grad(x, to_dev(cls), 1.0, stats, f(1.0), grad, ws)
    assert bool(grad[:5].isnan().all()) and bool((grad[5:7] == 0).all()) and bool(grad[7].isfinite().all())
    # NaN and infinities among the rows' own inputs
    y = torch.zeros(n, C, device=DEV)
    cls = to_dev(np.full(n, 1, dtype=np.int32))
    inf, nan = float("inf"), float("nan")
    own = -float(np.log(C))
    A = torch.tensor([nan, 0.0, 1.0, -1.0, 1.0, 0.0, 1.0, 1.0], device=DEV)
    old = torch.tensor([own, -inf, -inf, -inf, nan, nan, inf, own], device=DEV)
    rf = torch.tensor([own, own, own, own, own, own, own, -inf], device=DEV)
    g.gbdt_policy_step(y, cls, 1.0, old, rf, A, None, 0.2, 0.2, 0.5, loss, logp, grad, ws)
    l = loss.cpu().numpy()
    assert np.isnan(l[0]) and abs(l[1]) < 1e-6 and abs(l[2] + 1.2) < 1e-6 and l[3] == np.inf
    assert np.isnan(l[4]) and abs(l[5]) < 1e-6 and abs(l[6]) < 1e-6 and l[7] == np.inf
    fin = grad.isfinite().all(1).cpu().tolist()
    assert fin == [False, True, True, False, False, True, True, True]
    assert g.gbdt_read_error(ws) == 0


def test_clip_borders():
    """One class: logp is 0, and the ratio exactly 1 and 2 from old_logp 0 and, as
    far as FP32 goes, on both sides of it."""
    say("learn: borders")
    n = 8
    x = torch.zeros(n, 1, device=DEV)
    cls = torch.zeros(n, dtype=torch.int32, device=DEV)
    old = torch.tensor([0.0, 0.0, 1e-6, -1e-6, 1e-6, -1e-6, 0.0, 0.0], device=DEV)
    A = torch.tensor([1.0, -1.0, 1.0, 1.0, -1.0, -1.0, 2.0, -0.0], device=DEV)
    ws = workspace(x)
    loss, dlogp, stats = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV), torch.zeros(n, 2, device=DEV)
    g.gbdt_policy_loss(x, cls, 1.0, old, None, A, None, 0.0, 0.0, 0.0, loss, None, dlogp, stats, ws)
    # at the border r A counts; past it, on the side that A would push further, it does not
    want = [-1.0, 1.0, -np.exp(-1e-6), 0.0, 0.0, np.exp(1e-6), -2.0, 0.0]
    assert np.allclose(dlogp.cpu().numpy(), want, rtol=2.0 ** -23, atol=0.0)
    assert np.allclose(loss.cpu().numpy(), [-1.0, 1.0, -np.exp(-1e-6), -1.0, 1.0, np.exp(1e-6), -2.0, 0.0],
                       rtol=2.0 ** -23, atol=0.0)
    assert bool((stats[:, 0] == float("-inf")).all()) and bool((stats[:, 1] == 0).all())


@pytest.mark.parametrize("C,n", [(2, 64), (7, 300), (20, 64), (40, 200), (60, 64), (100, 64), (200, 40), (700, 64),
                                 (1500, 20), (3000, 20), (6000, 20), (9001, 130), (20011, 20), (70001, 20), (70001, 140)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_ratios_next_to_the_borders(C, n, dtype):
    """Ratios within a few parts in ten million of 0.8 and 1.28, on both sides, as old
    log-probabilities in FP32 come to lie: FP32 exponentials could not tell the side."""
    say("learn, next to the borders: %d x %d %s" % (n, C, dtype))
    T = 1.3
    x, xh = ref.rows(n, C, dtype, C + n, pad=C % 3)
    cls = draw_classes(xh, C, 0.0)
    r = np.random.default_rng(C)
    lp = np.array([lref.row(xh[i], int(cls[i]), T)[1] for i in range(n)])
    border = np.where(r.random(n) < 0.5, 0.8, 1.28)
    old = (lp - np.log(border)).astype(np.float32)
    for _ in range(2):
        old = np.where(r.random(n) < 0.3, np.nextafter(old, np.float32(r.choice([-99, 99]))), old)
    A = np.where(border < 1, -1.0, 1.0).astype(np.float32) * r.uniform(0.5, 2.0, n).astype(np.float32)
    ratio = np.exp(lp - old.astype(np.float64))
    # (the FP64 functions of either side are off by a few 2^-52; old is a rounding and at most
    # two steps, of 2^-23 |old| each, away)
    off = np.abs(ratio / border - 1)
    assert np.all(off > 1e-13) and np.all(off <= 3 * 2.0 ** -23 * np.abs(old) + 1e-9)
    kept = np.where(border < 1, ratio >= border, ratio <= border)
    assert 0 < kept.sum() < n
    check_policy(x, xh, cls, T, dtype, with_ref=False, rows=(old, None, A, np.ones(n, dtype=np.float32)))


@pytest.mark.parametrize("C", [5, 300, 3001])
def test_gradient_against_differences(C):
    """Central differences of the FP64 losses; h^2 times a third derivative of order
    1, and the loss's own rounding over h, bound the error."""
    say("learn, differences: C=%d" % C)
    h, n, T = 1e-4, 4, 1.3
    x, xh = ref.rows(n, C, "f32", 11, spread=1.0)
    cls = np.array([0, C - 1, C // 2, 1], dtype=np.int32)
    lp = np.array([lref.row(xh[i], int(cls[i]), T)[1] for i in range(n)])
    old, rf = (lp + 0.05).astype(np.float32), (lp - 0.3).astype(np.float32)
    A = np.array([1.0, -0.5, 2.0, 0.7], dtype=np.float32)
    ws = workspace(x, True)
    loss, grad = torch.zeros(n, device=DEV), torch.zeros(n, C, device=DEV)
    g.gbdt_policy_step(x, to_dev(cls), T, to_dev(old), to_dev(rf), to_dev(A), None, 0.2, 0.2, 0.1, loss, None, grad, ws)
    pl, pg = torch.zeros(1, device=DEV), torch.zeros(n, C, device=DEV)
    off = torch.tensor([0, 2, 4], device=DEV)
    g.gbdt_preference_step(x, to_dev(cls), T, off, to_dev(rf), None, 0.4, 0.1, True, pl, None, pg, ws)

    def policy_loss(row, i):
        return lref.policy(lref.row(row, int(cls[i]), T)[1], old[i], rf[i], float(A[i]), 0.2, 0.2, 0.1)[0]

    def pair_loss(row, i):
        S = lp - rf.astype(np.float64)
        S[i] = lref.row(row, int(cls[i]), T)[1] - float(rf[i])
        return lref.pair(0.4 * S[:2].mean(), 0.4 * S[2:].mean(), 0.1)[0]

    for f, got in ((policy_loss, grad), (pair_loss, pg)):
        got = got.double().cpu().numpy()
        for i in range(n):
            for c in {0, 1, C // 2, C - 1}:
                a, b = xh[i].copy(), xh[i].copy()
                a[c] += h
                b[c] -= h
                diff = (f(a, i) - f(b, i)) / (2 * h)
                assert abs(diff - got[i, c]) <= 10 * h * h + 1e-13 / h + 1e-5 * abs(diff), (i, c, diff, got[i, c])


# ------------------------------------- far rows, streams, graphs, records --

def test_offsets_beyond_32_bits():
    """Rows 2^31 + 5 elements apart."""
    C, n, stride = 9001, 3, (1 << 31) + 5
    say("learn: rows %d elements apart" % stride)
    x0, xh = ref.rows(n, C, "bf16", 21)
    buf = torch.empty((n - 1) * stride + C, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((n, C), (stride, 1))
    x.copy_(x0)
    cls = np.array([5, 9000, 77], dtype=np.int32)
    check_logp(x, xh, cls, 1.0, "bf16")
    check_policy(x, xh, cls, 1.0, "bf16")
    check_pairs(x, xh, cls, 1.0, "bf16", [0, 1, 3], 0.1, 0.0, False)


def test_no_rows():
    x = torch.zeros(0, 12, device=DEV)
    ws = workspace(x, True)
    f, i, s = torch.zeros(0, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV), torch.zeros(0, 2, device=DEV)
    g.gbdt_class_logp(x, i, 1.0, f, s, ws)
    g.gbdt_class_logp_grad(x, i, 1.0, s, f, x, ws)
    g.gbdt_policy_step(x, i, 1.0, f, f, f, f, 0.2, 0.2, 0.1, f, f, x, ws)
    # pairs of nothing: both rewards 0
    off = torch.zeros(5, dtype=torch.int64, device=DEV)
    loss, rewards = torch.zeros(2, device=DEV), torch.full((2, 2), 7.0, device=DEV)
    g.gbdt_preference_step(x, i, 1.0, off, f, None, 0.1, 0.0, False, loss, rewards, x, ws)
    assert np.allclose(loss.cpu().numpy(), np.log(2.0), rtol=2.0 ** -23) and bool((rewards == 0).all())
    g.gbdt_preference_step(x, i, 1.0, off[:1], f, None, 0.1, 0.0, False, loss[:0], rewards[:0], x, ws)
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("C,n", [(7, 300), (60, 100), (9001, 40), (70000, 3)])
def test_streams_graphs_and_repeats(C, n):
    """On another stream; captured and replayed with other inputs and eager work in
    between: the same bits."""
    say("learn, graph: %d x %d" % (n, C))
    x, xh = ref.rows(n, C, "f32", 41)
    ws, ws2 = workspace(x, True), workspace(x, True)
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    cls = to_dev(draw_classes(xh, 1))
    old, rf, A, w = (to_dev(a) for a in policy_rows(np.full(n, -2.0), 3))
    off = to_dev(np.array([0, n // 3, n // 2, n // 2, n], dtype=np.int64))
    logp, stats, loss, dlogp = f(n), f(n, 2), f(n), f(n)
    g1, g2, g3 = f(n, C), f(n, C), f(n, C)
    ploss, rewards, plogp, pd, pstats = f(2), f(2, 2), f(n), f(n), f(n, 2)
    outs = [logp, stats, loss, dlogp, g1, g2, g3, ploss, rewards, plogp, pd, pstats]

    def work(ws):
        g.gbdt_class_logp(x, cls, 1.0, logp, None, ws)
        g.gbdt_policy_loss(x, cls, 1.0, old, rf, A, w, 0.2, 0.2, 0.1, loss, logp, dlogp, stats, ws)
        g.gbdt_class_logp_grad(x, cls, 1.0, stats, dlogp, g1, ws)
        g.gbdt_policy_step(x, cls, 1.0, old, rf, A, w, 0.2, 0.2, 0.1, loss, logp, g2, ws)
        g.gbdt_preference_loss(x, cls, 1.0, off, rf, None, 0.1, 0.0, False, ploss, rewards, plogp, pd, pstats, ws)
        g.gbdt_preference_step(x, cls, 1.0, off, rf, None, 0.1, 0.0, False, ploss, rewards, g3, ws)

    def taken():
        torch.cuda.synchronize()
        got = [t.cpu() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        return got

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work(ws)
    taken()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(ws)
    for k in range(4):
        fresh, _ = ref.rows(n, C, "f32", 50 + k)
        x.copy_(fresh)
        work(ws2)
        want = taken()
        graph.replay()
        for a, b in zip(want, taken()):
            assert torch.equal(a, b), k
        with torch.cuda.stream(s):
            work(ws)
        for a, b in zip(want, taken()):
            assert torch.equal(a, b), k
    assert g.gbdt_read_error(ws) == 0 and g.gbdt_read_error(ws2) == 0


@pytest.mark.parametrize("C", [7, 60, 500, 9001, 70000])
def test_device_side_checks(C):
    """Classes and offsets that only the device sees: recorded, in bounds, other rows right."""
    say("learn, device checks: C=%d" % C)
    n = 4
    x, xh = ref.rows(n, C, "f32", 61)
    ws = workspace(x, True)
    logp, stats, grad = torch.zeros(n, device=DEV), torch.zeros(n, 2, device=DEV), torch.zeros(n, C, device=DEV)

    def code():
        with pytest.raises(g.GbdtError) as e:
            g._check(g.gbdt_read_error(ws), "learn")
        assert g.gbdt_read_error(ws) == 0
        return e.value.code

    for bad in (C, C + 1000, 2 ** 31 - 1):
        cls = np.array([0, bad, -5, 1], dtype=np.int32)
        g.gbdt_class_logp(x, to_dev(cls), 1.0, logp, stats, ws)
        assert code() == -3
        assert logp[1].item() == 0.0 and bool((stats[1:3] == 0).all())
        for i in (0, 2, 3):
            assert same(logp[i].item(), lref.row(xh[i], int(cls[i]), 1.0)[1], 1e-4)
        grad.fill_(7.0)
        g.gbdt_class_logp_grad(x, to_dev(cls), 1.0, stats, torch.ones(n, device=DEV), grad, ws)
        assert code() == -3 and bool((grad[1:3] == 0).all()) and bool(grad[0].abs().sum() > 0)
    cls = to_dev(np.array([0, 1, 0, 1], dtype=np.int32))
    loss = torch.zeros(1, device=DEV)
    for cuts in ([0, 3, 2], [-1, 2, 4], [0, 2, 5], [2, 1, 0], [3 << 40, 1, -(1 << 62)]):
        off = to_dev(np.array(cuts, dtype=np.int64))
        g.gbdt_preference_step(x, cls, 1.0, off, None, None, 0.1, 0.0, False, loss, None, grad, ws)
        assert code() == -3
    g.gbdt_preference_step(x, cls, 1.0, to_dev(np.array([0, 2, 4])), None, None, 0.1, 0.0, False, loss, None, grad, ws)
    assert g.gbdt_read_error(ws) == 0
    wl = [lref.row(xh[i], [0, 1, 0, 1][i], 1.0)[1] for i in range(4)]
    assert same(loss.item(), lref.pair(0.1 * (wl[0] + wl[1]), 0.1 * (wl[2] + wl[3]), 0.0)[0], 1e-5)


def test_workspace_shared_with_other_operators():
    """A workspace that other operators used before: their partial results do no harm."""
    say("learn: shared workspace")
    C, n = 70000, 2
    x, xh = ref.rows(n, C, "bf16", 5)
    ws = workspace(x)
    v, c = torch.zeros(n, 20, device=DEV), torch.zeros(n, 20, dtype=torch.int32, device=DEV)
    rest = torch.zeros(n, device=DEV)
    out = torch.zeros(n, dtype=torch.int32, device=DEV)
    logp, want = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    cls = torch.zeros(n, dtype=torch.int32, device=DEV)
    g.gbdt_class_logp(x, cls, 1.0, want, None, workspace(x))
    for _ in range(3):
        g.gbdt_top_scores(x, 20, 1.0, v, c, rest, ws)
        loss, grad = torch.zeros(n, device=DEV), torch.zeros_like(x)
        g.gbdt_distill_step(x, v, c, rest, 1.0, None, loss, grad, ws)
        g.gbdt_sample_classes(x, rest.clamp(0, 0.9), None, None, None, None, out, None, ws)
        places = torch.zeros(20000, dtype=torch.int32, device=DEV)
        offsets, order = torch.zeros(1025, dtype=torch.int32, device=DEV), torch.zeros_like(places)
        g.gbdt_route_lists(places, 1024, offsets, order, None, ws)
        logp.zero_()
        g.gbdt_class_logp(x, cls, 1.0, logp, None, ws)
        assert torch.equal(logp, want)
    assert g.gbdt_read_error(ws) == 0
