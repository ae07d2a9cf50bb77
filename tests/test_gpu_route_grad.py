"""The routing weights' gradient where scores are odd, against the reference in
route_ref.py.  STEP is half a step of FP32, relative."""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import learn_ref as lref
import route_ref as rref
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24
TINY = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}
FORMS = [dict(), dict(sigmoid=True), dict(renormalise=False), dict(sigmoid=True, renormalise=False, scale=2.5)]


def to_dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def workspace(n, E):
    return g.new_workspace(g.gbdt_scores_workspace_bytes(n, E))


def route(x, r, bias=None):
    n, E = x.shape
    classes = torch.full((n, r.k), 7, dtype=torch.int32, device=DEV)
    weights = torch.full((n, r.k), 7.0, device=DEV)
    ws = workspace(n, E)
    g.gbdt_route_classes(x, r, to_dev(bias), classes, weights, ws)
    assert g.gbdt_read_error(ws) == 0
    return classes, weights


def gradient(x, r, classes, dw):
    ws = workspace(*x.shape)
    grad = torch.full(x.shape, 7.0, dtype=x.dtype, device=DEV)
    g.gbdt_route_grad(x, r, classes, to_dev(dw), grad, ws)
    assert g.gbdt_read_error(ws) == 0
    return grad.double().cpu().numpy()


def nan_rows(E, dtype, seed):
    """Rows with none, one, some, half and all but one of their vectors of 16 bytes NaN,
    and with NaN here and there."""
    r = np.random.default_rng(seed)
    b = r.normal(0.0, 1.5, (9, E))
    VE = 4 if dtype == "f32" else 8
    V = (E + VE - 1) // VE
    for i, share in ((1, 1), (2, min(3, V)), (3, (V + 1) // 2), (4, V - 1)):
        for v in r.permutation(V)[:share]:
            b[i, v * VE:(v + 1) * VE] = np.nan
    b[5, r.random(E) < 0.5] = np.nan
    b[6, r.random(E) < 0.95] = np.nan
    b[7, : max(1, E // 2)] = np.nan  # (with -inf behind them)
    b[7, E // 2:: 3] = -np.inf
    b[8] = np.nan
    return torch.from_numpy(b).to(ref.TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [1, 3, 4, 8, 12, 16, 60, 64, 100, 256, 257, 1000, 1024])
def test_vectors_of_nan(E, dtype):
    """NaN experts are out of service, whole vectors of them too: the others' gradient
    is what it is without them.  The softmax's sum is of FP32 exponentials, off by
    (3 D + 5) STEP, which both a value and the sum it is taken from can be (6 D + 10)."""
    say("route gradient, NaN: %d %s" % (E, dtype))
    t = nan_rows(E, dtype, E)
    x, xh = ref.place(t, E % 3), t.double().numpy()
    k = min(E, 6)
    dw = np.random.default_rng(E).normal(0.0, 1.0, (len(xh), k)).astype(np.float32)
    for form in FORMS:
        r = g.make_routing(k, **form)
        classes, weights = route(x, r)
        got, c = gradient(x, r, classes, dw), classes.cpu().numpy()
        assert bool(weights.isfinite().all())
        for i in range(len(xh)):
            want, size = rref.grad(xh[i], r, c[i], dw[i])
            fin = xh[i][np.isfinite(xh[i])]
            D = np.ptp(fin) if len(fin) else 0.0
            tol = (ref.EPS[dtype] / 2 + 2 * STEP) * np.abs(want) + size * (6 * D + 10) * STEP + TINY[dtype]
            assert np.all(np.abs(got[i] - want) <= tol), (form, i, got[i], want)
            assert np.all(got[i][~np.isfinite(xh[i])] == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_saturated_sigmoids(renormalise, dtype):
    """Scores from -80 to 80: the derivative s(x) s(-x) keeps its digits on both sides.
    FP64, rounded once; 2^-45 for the functions and for what cancels in the mean."""
    say("route gradient, saturated: %s %s" % (renormalise, dtype))
    E, k = 40, 16
    rng = np.random.default_rng(3)
    b = np.stack([np.linspace(-80.0, 80.0, E), rng.uniform(-80.0, 80.0, E), rng.uniform(10.0, 60.0, E),
                  rng.uniform(-60.0, -10.0, E), np.where(np.arange(E) % 2, 30.0, -30.0)])
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    x, xh = ref.place(t), t.double().numpy()
    r = g.make_routing(k, sigmoid=True, renormalise=renormalise, scale=1.5)
    c = np.stack([rng.permutation(E)[:k] for _ in b]).astype(np.int32)
    dw = rng.normal(0.0, 1.0, (len(b), k)).astype(np.float32)
    got = gradient(x, r, to_dev(c), dw)
    for i in range(len(b)):
        want, size = rref.grad(xh[i], r, c[i], dw[i])
        tol = (ref.EPS[dtype] / 2 + STEP) * np.abs(want) + 2.0 ** -45 * size + TINY[dtype]
        assert np.all(np.abs(got[i] - want) <= tol), (i, got[i], want)


def sharp_tolerance(x, r, chosen, dw, want, dtype):
    """Softmax values as they are.  A sum of FP32 exponentials is off by q = (3 D + 5)
    STEP: the exponent (difference, constant, product, STEP D each), the exponential (2
    STEP), three additions; D as far as terms of the mass R outside the choice go, those
    40 below its largest adding nothing.  So are R and each value s.  What the kernel
    adds up for a chosen expert: d_j - u, s_i (d_i - u) and u R, u the dweight of the
    largest chosen score where R is below 1/2, else 0.  Others: their own exponential,
    two products, and sum s d."""
    (c, s), R, every = rref.parts(x, r, chosen)
    d = dw[(chosen >= 0) & (chosen < len(x))].astype(np.float64)
    s, R, every = s.astype(np.float64), float(R), every.astype(np.float64)
    top, scale = (int(np.argmax(x[c])) if len(c) else 0), abs(r.scale)
    fin = np.isfinite(x)
    D = np.where(fin, x[fin].max() - x, 0.0) if fin.any() else np.zeros(len(x))
    outside = fin.copy()
    outside[c] = False
    far = min(90.0, D[outside].min() + 40.0, D[outside].max()) if outside.any() else 0.0
    q = 0.0 if r.renormalise else (3 * far + 5) * STEP
    us = [d[top] if len(c) else 0.0]
    us = us if r.renormalise or R < 0.499 else [0.0] if R > 0.501 else us + [0.0]
    tol = (ref.EPS[dtype] / 2 + STEP + q) * np.abs(want)
    terms = max(np.abs(s * (d - u)).sum() + abs(u) * R for u in us) if len(c) else 0.0
    mine = max(np.abs(d - u) for u in us) if len(c) == 1 else sum(np.abs(d - u) for u in us) if len(c) else 0.0
    rest = scale * every * np.abs(s * d).sum() * (q + 2.0 ** -45) + (3 * np.minimum(D, 90.0) + 4) * STEP * np.abs(want)
    rest[c] = scale * s * (q * terms + 2.0 ** -45 * (mine + terms))
    return tol + rest + TINY[dtype] * (1 + scale * np.abs(d).sum())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("E", [2, 9, 60, 129, 256, 1000])
@pytest.mark.parametrize("renormalise", [False, True])
def test_a_router_that_is_sure(E, renormalise, dtype):
    """One expert far above the others, two experts, and all chosen but a few: 1 - s, and
    the mass outside the choice, keep their digits."""
    say("route gradient, sure: %d %s %s" % (E, renormalise, dtype))
    rng = np.random.default_rng(E)
    b = rng.normal(0.0, 1.0, (9, E))
    for i, gap in enumerate((0.0, 3.0, 8.0, 15.0, 25.0, 40.0, 70.0)):
        b[i, rng.integers(E)] += gap
    b[7, : 2] += 20.0   # two of them
    b[8, 0] -= 30.0
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    x, xh = ref.place(t), t.double().numpy()
    for k in sorted({1, 2, min(E, 8), min(E, 32)}):
        for same in (False, True):  # (equal dweights: renormalised weights have no gradient, others R alone)
            r = g.make_routing(k, renormalise=renormalise, scale=2.5)
            classes, _ = route(x, r)
            c = classes.cpu().numpy()
            dw = rng.normal(0.0, 1.0, (len(b), k)).astype(np.float32)
            dw = np.full_like(dw, 0.75) if same else dw
            got = gradient(x, r, classes, dw)
            for i in range(len(b)):
                want, _ = rref.grad(xh[i], r, c[i], dw[i])
                tol = sharp_tolerance(xh[i], r, c[i], dw[i], want, dtype)
                assert np.all(np.abs(got[i] - want) <= tol), (k, i, np.max(np.abs(got[i] - want) / tol), got[i], want)


@pytest.mark.parametrize("E", [9, 60, 256])
def test_experts_of_little_mass(E):
    """The choice, by a bias, is of experts that the softmax has little of, with dweights
    of very different sizes: each keeps the digits of its own."""
    say("route gradient, little mass: %d" % E)
    rng = np.random.default_rng(E)
    b = rng.normal(0.0, 1.0, (6, E)).astype(np.float32)
    b[:, 5:] += np.float32(6.0)
    b[3:, 0] += np.linspace(4.0, 9.0, 3).astype(np.float32)
    x, xh = ref.place(torch.from_numpy(b)), b.astype(np.float64)
    k = 4
    r = g.make_routing(k, renormalise=False)
    c = np.tile(np.arange(k, dtype=np.int32), (len(b), 1))
    dw = (rng.normal(0.0, 1.0, (len(b), k)) * 10.0 ** rng.integers(-8, 1, (len(b), k))).astype(np.float32)
    got = gradient(x, r, to_dev(c), dw)
    for i in range(len(b)):
        want, _ = rref.grad(xh[i], r, c[i], dw[i])
        tol = sharp_tolerance(xh[i], r, c[i], dw[i], want, "f32")
        assert np.all(np.abs(got[i] - want) <= tol), (i, np.max(np.abs(got[i] - want) / tol), got[i], want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [16, 60, 256, 1000])
@pytest.mark.parametrize("renormalise", [False, True])
def test_odd_rows(E, renormalise, dtype):
    """Nothing left, all equal, half out of service, infinities, far apart, the lowest."""
    say("route gradient, odd rows: %d %s %s" % (E, renormalise, dtype))
    rng = np.random.default_rng(E)
    b = np.round(rng.normal(0.0, 1.5, (14, E)))
    b[0] = -np.inf
    b[1] = 0.0
    b[2] = -np.inf
    b[2, E // 2] = 1.0
    b[3, : E // 2] = -np.inf
    b[4, 1:] = -np.inf
    b[5, rng.random(E) < 0.5] = np.nan
    b[6] = np.where(rng.random(E) < 0.5, 0.0, -0.0)
    b[7, [1, 3]] = np.inf
    b[8] = 200.0 + np.round(rng.normal(0.0, 1.0, E))
    b[9] = -200.0 + np.round(rng.normal(0.0, 1.0, E))
    b[10] = -np.inf
    b[10, [0, E - 1]] = [-300.0, 300.0]
    b[11] = np.where(np.arange(E) % 5 == 0, 3.0, -np.inf)
    b[12] = -6.0e4
    b[13, : E - 3] = np.nan
    b[13, E - 1] = np.inf
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    x = ref.place(t, E % 5)
    # (+inf counts as the largest FP32 number)
    xh = np.minimum(t.double().numpy(), float(np.finfo(np.float32).max))
    for k in (1, 8):
        r = g.make_routing(k, renormalise=renormalise, scale=1.5)
        classes, _ = route(x, r)
        c = classes.cpu().numpy()
        dw = rng.normal(0.0, 1.0, (len(b), k)).astype(np.float32)
        got = gradient(x, r, classes, dw)
        for i in range(len(b)):
            want, _ = rref.grad(xh[i], r, c[i], dw[i])
            tol = sharp_tolerance(xh[i], r, c[i], dw[i], want, dtype)
            assert np.all(np.abs(got[i] - want) <= tol), (k, i, got[i], want)


@pytest.mark.parametrize("scale", [2.5, 1000.0])
def test_values_next_to_nothing(scale):
    """Sigmoid values of some e^-700: their quotients are ordinary numbers, and so are the
    weights and their gradient.  FP64, rounded once; 2^-40 for the functions."""
    say("route, values next to nothing: %g" % scale)
    E, k = 12, 4
    rng = np.random.default_rng(4)
    b = rng.uniform(-706.9, -706.0, (3, E)).astype(np.float32)
    x, xh = ref.place(torch.from_numpy(b)), b.astype(np.float64)
    r = g.make_routing(k, sigmoid=True, scale=scale)
    classes, weights = route(x, r)
    dw = rng.normal(0.0, 1.0, (len(b), k)).astype(np.float32)
    got, c = gradient(x, r, classes, dw), classes.cpu().numpy()
    for i in range(len(b)):
        wc, ww = lref.route(xh[i], r, None)
        assert np.array_equal(c[i], wc)
        assert np.all(np.abs(weights[i].double().cpu().numpy() - ww) <= (STEP + 2.0 ** -40) * np.abs(ww)), (i, weights[i])
        want, size = rref.grad(xh[i], r, c[i], dw[i])
        assert np.all(np.abs(got[i] - want) <= STEP * np.abs(want) + 2.0 ** -40 * size), (i, got[i], want)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_dweights_that_are_no_numbers(form, bad):
    """They reach experts in service; one out of service has gradient 0."""
    say("route gradient, dweight %g: %s" % (bad, form))
    E, k = 30, 4
    b = np.random.default_rng(5).normal(0.0, 1.0, (4, E)).astype(np.float32)
    b[:, 20:] = -np.inf
    b[:, [3, 7]] = np.nan
    x = ref.place(torch.from_numpy(b))
    r = g.make_routing(k, **form)
    classes, _ = route(x, r)
    dw = np.ones((4, k), dtype=np.float32)
    dw[:2, 1] = bad
    got, c = gradient(x, r, classes, dw), classes.cpu().numpy()
    out = ~np.isfinite(b)
    assert np.all(got[out] == 0)
    assert np.all(np.isfinite(got[2:]))
    for i in range(2):
        assert not np.isfinite(got[i, c[i, 1]])
        if not r.score and not r.renormalise:
            assert not np.isfinite(got[i][~out[i]]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("renormalise", [False, True])
def test_odd_sigmoids(renormalise, dtype):
    """Infinities, NaN, the largest numbers and equal scores under a sigmoid: FP64, rounded
    once, and 2^-45 as above."""
    say("route gradient, odd sigmoids: %s %s" % (renormalise, dtype))
    E, k = 60, 8
    rng = np.random.default_rng(6)
    b = np.round(rng.normal(0.0, 1.5, (8, E)))
    b[0] = -np.inf
    b[1] = 0.0
    b[2, rng.random(E) < 0.5] = np.nan
    b[3, ::2] = np.inf
    b[4] = np.where(np.arange(E) % 3 == 0, 6.0e4, -6.0e4)
    b[5, 1:] = -np.inf
    b[6] = np.nan
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    x, xh = ref.place(t, 3), t.double().numpy()
    r = g.make_routing(k, sigmoid=True, renormalise=renormalise, scale=0.7)
    for c in (route(x, r)[0].cpu().numpy(), np.stack([rng.permutation(E)[:k] for _ in b]).astype(np.int32)):
        dw = rng.normal(0.0, 1.0, (len(b), k)).astype(np.float32)
        got = gradient(x, r, to_dev(c), dw)
        for i in range(len(b)):
            want, size = rref.grad(xh[i], r, c[i], dw[i])
            tol = (ref.EPS[dtype] / 2 + STEP) * np.abs(want) + 2.0 ** -45 * size + TINY[dtype]
            assert np.all(np.abs(got[i] - want) <= tol), (i, got[i], want)
