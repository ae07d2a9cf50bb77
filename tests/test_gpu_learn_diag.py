"""Diagnostics of the calls on drawn classes and of the routing: a record for each launch."""
import pytest
import torch

import histogram_split_finding_amd as g
import scores_ref as ref
from gpu_util import DEV, say
from test_gpu_scores_diag import kinds_of

pytestmark = pytest.mark.gpu

LOGP, PAIRS, ROUTE, LISTS = 19, 20, 21, 22


@pytest.mark.parametrize("C,forward,step", [
    (7, 1, 1),       # a thread a row
    (400, 1, 1),     # a wave a row
    (9001, 1, 1),    # a workgroup a row
    (70001, 1, 2),   # few long rows: parts, joined by the last of them, or by a second launch
])
def test_launches(C, forward, step):
    say("diagnostics: C=%d" % C)
    n = 5
    x, _ = ref.rows(n, C, "f32", C)
    cls = torch.zeros(n, dtype=torch.int32, device=DEV)
    f = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    off = torch.tensor([0, 2, 5], device=DEV)
    ws = g.new_workspace(g.gbdt_preference_workspace_bytes(n, C))
    logp, stats, dlogp, loss, grad = f(n), f(n, 2), f(n), f(n), f(n, C)
    pol = (logp, None, f(n), None, 0.2, 0.2, 0.0)
    pair = (off, None, None, 0.1, 0.0, False)
    assert kinds_of(lambda: g.gbdt_class_logp(x, cls, 1.0, f(n), stats, ws)) == [LOGP] * forward
    assert kinds_of(lambda: g.gbdt_class_logp_grad(x, cls, 1.0, stats, dlogp, grad, ws)) == [LOGP]
    assert kinds_of(lambda: g.gbdt_policy_loss(x, cls, 1.0, *pol, loss, None, dlogp, stats, ws)) == [LOGP] * forward
    assert kinds_of(lambda: g.gbdt_policy_step(x, cls, 1.0, *pol, loss, None, grad, ws)) == [LOGP] * step
    assert kinds_of(lambda: g.gbdt_preference_loss(x, cls, 1.0, *pair, loss[:1], None, logp, dlogp, stats, ws)) == \
        [LOGP] * forward + [PAIRS]
    assert kinds_of(lambda: g.gbdt_preference_step(x, cls, 1.0, *pair, loss[:1], None, grad, ws)) == \
        [LOGP] * forward + [PAIRS, LOGP]
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("n,lists", [(3, 1), (3000, 2)])
def test_routing_launches(n, lists):
    say("diagnostics: routing of %d rows" % n)
    E, k = 60, 4
    x, _ = ref.rows(n, E, "f32", 1)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(n, E))
    c, w = torch.zeros(n, k, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
    off, order = torch.zeros(E + 1, dtype=torch.int32, device=DEV), torch.zeros(n * k, dtype=torch.int32, device=DEV)
    r = g.make_routing(k)
    assert kinds_of(lambda: g.gbdt_route_classes(x, r, None, c, w, ws)) == [ROUTE]
    assert kinds_of(lambda: g.gbdt_route_grad(x, r, c, w, torch.zeros_like(x), ws)) == [ROUTE]
    assert kinds_of(lambda: g.gbdt_route_lists(c, E, off, order, None, ws)) == [LISTS] * lists
    assert g.gbdt_read_error(ws) == 0
