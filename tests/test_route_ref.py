"""The reference of the routing weights' gradient: against the Jacobian where nothing
cancels, and against 60 digits where much does."""
from decimal import Decimal, getcontext

import numpy as np
import pytest

import histogram_split_finding_amd as g
import learn_ref as lref
import route_ref as rref

FORMS = [dict(), dict(sigmoid=True), dict(renormalise=False), dict(sigmoid=True, renormalise=False, scale=2.5)]


@pytest.mark.parametrize("form", FORMS)
def test_against_the_jacobian(form):
    rng = np.random.default_rng(1)
    for E, k in ((1, 1), (7, 3), (60, 8)):
        x = rng.normal(0.0, 1.5, E)
        x[0] = x[0] if E == 1 else -np.inf
        r = g.make_routing(k, **form)
        chosen = lref.route(x, r, None)[0]
        chosen[-1] = chosen[-1] if E == 1 else -1
        dw = rng.normal(0.0, 1.0, k).astype(np.float32)
        want, size = rref.grad(x, r, chosen, dw)
        # (a few roundings of each of its terms on the Jacobian's side)
        assert np.all(np.abs(lref.route_grad(x, r, chosen, dw) - want) <= 2.0 ** -46 * (size + size.max()))


@pytest.mark.parametrize("form", FORMS)
def test_saturated_against_60_digits(form):
    getcontext().prec = 60
    rng = np.random.default_rng(2)
    E, k = 9, 3
    for top in (20.0, 45.0, 90.0, 300.0):
        x = rng.normal(0.0, 1.0, E)
        x[4] += top
        r = g.make_routing(k, **form)
        chosen = lref.route(x, r, None)[0]
        dw = rng.normal(0.0, 1.0, k).astype(np.float32)
        want, _ = rref.grad(x, r, chosen, dw)
        X, d = [Decimal(v) for v in x], [Decimal(float(v)) for v in dw]
        if r.score:
            s = [1 / (1 + (-v).exp()) for v in X]
            slope = [v * (1 - v) for v in s]
        else:
            e = [v.exp() for v in X]
            s = [v / sum(e) for v in e]
        N = sum(s[c] for c in chosen) if r.renormalise else Decimal(1)
        mean = sum(s[c] * d[j] for j, c in enumerate(chosen)) / N if r.renormalise else Decimal(0)
        ds = {int(c): (d[j] - mean) / N for j, c in enumerate(chosen)}
        pull = sum(ds[int(c)] * s[c] for c in chosen)
        for c in range(E):
            exact = slope[c] * ds.get(c, Decimal(0)) if r.score else s[c] * (ds.get(c, Decimal(0)) - pull)
            exact *= Decimal(r.scale)
            # (60 digits leave 1e-50 of what cancels; exp(x) in 64 bits of mantissa is off by |x| 2^-64)
            assert abs(Decimal(float(want[c])) - exact) <= abs(exact) * Decimal(2.0 ** -52) + Decimal(1e-50), (top, c)
