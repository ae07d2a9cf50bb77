"""The routing weights' gradient where scores are odd, against the reference in
route_ref.py.  STEP is half a step of FP32, relative."""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
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
