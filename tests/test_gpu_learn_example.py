"""The operators as they are used together: draws, policy steps, preference steps;
routed ensembles.  What is checked is that they run, and that the gradients that the
example follows are those of its losses."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import learn_ref as lref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "learn_from_draws.py")
    spec = importlib.util.spec_from_file_location("learn_from_draws", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_policy_runs():
    say("example: policy")
    rewards, losses = example().policy(rows=2000, steps=6)
    assert len(rewards) == len(losses) == 6 and np.all(np.isfinite(rewards)) and np.all(np.isfinite(losses))
    # the first step's margins are 0: its log-probabilities are the reference's
    assert abs(losses[0] - np.log(2.0)) < 1e-5


def test_router_runs():
    say("example: router")
    errors, shares = example().router(rows=1500, steps=3)
    assert len(errors) == 3 and np.all(np.isfinite(errors)) and abs(sum(shares) - 1.0) < 1e-5


def test_weight_gradients_of_draws():
    """The gradient of a linear policy's weights, drawn classes and all, against
    differences of the FP64 loss.  h^2 times third derivatives of order 30 (the
    features' size cubed), FP32 sums of 40 terms."""
    say("example: gradients")
    gen = np.random.default_rng(3)
    n, F, C = 40, 3, 7
    x = gen.normal(0.0, 1.0, (n, F)).astype(np.float32)
    w = gen.normal(0.0, 0.5, (F, C)).astype(np.float32)
    xd, wd = torch.from_numpy(x).to(DEV), torch.from_numpy(w).to(DEV)
    ws = g.new_workspace(g.gbdt_preference_workspace_bytes(n, C))
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    classes, old, loss, grad = torch.zeros(n, dtype=torch.int32, device=DEV), f(n), f(n), f(n, C)
    scores = (xd.double() @ wd.double()).float()
    g.gbdt_sample_classes(scores, torch.rand(n, device=DEV), None, None, None, None, classes, old, ws)
    # (steps later: ratios away from 1 and from the borders)
    old += torch.from_numpy(gen.choice([-0.1, 0.1, 0.5, -0.5], n).astype(np.float32)).to(DEV)
    A = torch.from_numpy(gen.normal(0.0, 1.0, n).astype(np.float32)).to(DEV)
    g.gbdt_policy_step(scores, classes, 1.0, old, old, A, None, 0.2, 0.2, 0.1, loss, None, grad, ws)
    got = (xd.double().t() @ grad.double()).cpu().numpy()
    off = torch.tensor([0, 10, 20, 30, 40], device=DEV)
    pl, pg = f(2), f(n, C)
    g.gbdt_preference_step(scores, classes, 1.0, off, old, None, 0.3, 0.1, False, pl, None, pg, ws)
    got2 = (xd.double().t() @ pg.double()).cpu().numpy()
    assert g.gbdt_read_error(ws) == 0
    cls, o, a = classes.cpu().numpy(), old.cpu().numpy(), A.cpu().numpy()

    def losses(weights):
        z = x.astype(np.float64) @ weights
        lp = [lref.row(z[i], int(cls[i]), 1.0)[1] for i in range(n)]
        S = np.array([lp[i] - float(o[i]) for i in range(n)]).reshape(4, 10).sum(1) * 0.3
        return (sum(lref.policy(lp[i], o[i], o[i], float(a[i]), 0.2, 0.2, 0.1)[0] for i in range(n)),
                sum(lref.pair(S[2 * p], S[2 * p + 1], 0.1)[0] for p in range(2)))

    h = 1e-4
    for q in range(F):
        for c in range(C):
            up, down = w.astype(np.float64), w.astype(np.float64)
            up[q, c] += h
            down[q, c] -= h
            u, d = losses(up), losses(down)
            assert abs((u[0] - d[0]) / (2 * h) - got[q, c]) <= n * 30 * h * h + n * 1e-6 * (1 + np.abs(a).max())
            assert abs((u[1] - d[1]) / (2 * h) - got2[q, c]) <= n * 30 * h * h + n * 1e-6
