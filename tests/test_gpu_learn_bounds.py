"""Offsets of pairs that descend, leave the rows or lie apart: recorded, and no row is
read or written but those between the first offset and the last."""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import learn_ref as lref
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [7, 60, 500, 9001, 70000])
def test_offsets_that_descend(C, dtype):
    """Classes that name no score, with statistics of another call's rows beside them."""
    say("learn, offsets that descend: C=%d %s" % (C, dtype))
    n = 12
    x, xh = ref.rows(n, C, dtype, 61)
    ws = g.new_workspace(g.gbdt_preference_workspace_bytes(n, C))
    f = lambda *s: torch.full(s, 3.0, device=DEV)  # noqa: E731
    good = np.arange(n, dtype=np.int32) % C
    odd = good.copy()
    odd[6:] = [-100, -1, C, 2 ** 31 - 1, -2 ** 31, C + 5]
    for cuts in ([0, 6, 2], [0, 12, 3], [2, 1, 0], [0, -5, 4], [0, 6, 1 << 40], [5, 9, 2, 12, 4], [0, 3, 6, 12, 5],
                 [3, 4, -(1 << 62), 1 << 62, 5], [12, 0, 12]):
        pairs = len(cuts) // 2
        off = torch.tensor(cuts, dtype=torch.int64, device=DEV)
        lo = min(max(cuts[0], 0), n)
        hi = min(max(cuts[-1], lo), n)
        outside = torch.ones(n, dtype=torch.bool, device=DEV)
        outside[lo:hi] = False
        # the step's workspace has another call's statistics of all rows
        loss, grad = f(pairs), torch.full_like(x, 3.0)
        full = torch.tensor([0, 6, 12], device=DEV)
        g.gbdt_preference_step(x, torch.from_numpy(good).to(DEV), 1.0, full, None, None, 0.1, 0.0, False, f(1), None,
                               grad, ws)
        assert g.gbdt_read_error(ws) == 0
        cls = torch.from_numpy(odd).to(DEV)
        grad.fill_(3.0)
        logp, dlogp, stats = f(n), f(n), f(n, 2)
        g.gbdt_preference_step(x, cls, 1.0, off, None, None, 0.1, 0.0, False, loss, None, grad, ws)
        assert g.gbdt_read_error(ws) == -3
        g.gbdt_preference_loss(x, cls, 1.0, off, None, None, 0.1, 0.0, False, loss, None, logp, dlogp, stats, ws)
        assert g.gbdt_read_error(ws) == -3
        for t in (grad, logp, dlogp, stats):
            assert bool((t[outside] == 3.0).all()), cuts
    # and a call with good ones after it
    cls = torch.from_numpy(good).to(DEV)
    loss = f(1)
    g.gbdt_preference_step(x, cls, 1.0, torch.tensor([1, 5, 11], device=DEV), None, None, 0.1, 0.0, False, loss, None,
                           torch.empty_like(x), ws)
    assert g.gbdt_read_error(ws) == 0
    lp = [lref.row(xh[i], int(good[i]), 1.0)[1] for i in range(n)]
    # (ten log-probabilities, each off by some 1e-5 at most, times 0.1)
    assert abs(loss.item() - lref.pair(0.1 * sum(lp[1:5]), 0.1 * sum(lp[5:11]), 0.0)[0]) <= 1e-5
