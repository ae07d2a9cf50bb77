"""The calls on drawn classes and a workspace that others of the library have used."""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def results(x, cls, ws):
    """All of the calls that split a long row between workgroups."""
    n, C = x.shape
    f = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    old, A = torch.full((n,), -3.0, device=DEV), torch.ones(n, device=DEV)
    off = torch.tensor([0, n // 2, n], device=DEV)
    logp, stats, loss, dlogp, grad = f(n), f(n, 2), f(n), f(n), torch.full_like(x, 7.0)
    ploss, rewards, plogp, pd, pstats, pgrad = f(1), f(1, 2), f(n), f(n), f(n, 2), torch.full_like(x, 7.0)
    g.gbdt_class_logp(x, cls, 1.0, logp, stats, ws)
    g.gbdt_policy_loss(x, cls, 1.0, old, None, A, None, 0.2, 0.2, 0.0, loss, None, dlogp, stats, ws)
    g.gbdt_policy_step(x, cls, 1.0, old, None, A, None, 0.2, 0.2, 0.0, loss, None, grad, ws)
    g.gbdt_preference_loss(x, cls, 1.0, off, None, None, 0.1, 0.0, False, ploss, rewards, plogp, pd, pstats, ws)
    g.gbdt_preference_step(x, cls, 1.0, off, None, None, 0.1, 0.0, False, ploss, rewards, pgrad, ws)
    assert g.gbdt_read_error(ws) == 0
    return [logp, stats, loss, dlogp, grad, ploss, rewards, plogp, pd, pstats, pgrad]


@pytest.mark.parametrize("n,C", [(1, 70001), (5, 70001), (128, 40001)])
def test_after_a_training_call(n, C):
    """The setup of a training matrix leaves its census of bins in the workspace, and any
    call of the library what it likes behind the control block."""
    say("learn: workspace of a training call, %d x %d" % (n, C))
    x, _ = ref.rows(n, C, "bf16", 5)
    cls = torch.arange(n, dtype=torch.int32, device=DEV)
    rows, features = 5000, 40
    ft = g.FeatureTable([200] * features, DEV)
    size = max(g.gbdt_workspace_bytes(rows, 1, ft.total_bins), g.gbdt_preference_workspace_bytes(n, C))
    want = results(x, cls, g.new_workspace(size))
    ws = g.new_workspace(size)
    bins = torch.from_numpy(np.random.default_rng(1).integers(0, 200, (rows, features)).astype(np.uint8)).to(DEV)
    for _ in range(2):
        g.gbdt_pack_matrix(bins, g.RowBuffer(ft, rows, DEV), ft, ws)
        for a, b in zip(want, results(x, cls, ws)):
            assert torch.equal(a, b)
        ws[256:] = 0xA5
        for a, b in zip(want, results(x, cls, ws)):
            assert torch.equal(a, b)


def test_rows_that_share_a_counter():
    """Neighbouring rows, each split between workgroups, call after call and replayed."""
    say("learn: counters of neighbouring rows")
    n, C = 127, 33000
    x, _ = ref.rows(n, C, "f32", 9)
    cls = torch.arange(n, dtype=torch.int32, device=DEV)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(n, C))
    logp = torch.zeros(n, device=DEV)
    g.gbdt_class_logp(x, cls, 1.0, logp, None, ws)
    want = torch.log_softmax(x.double(), 1).gather(1, cls.long()[:, None])[:, 0]
    # (FP32 exponentials of differences up to some 10, and one rounding)
    assert bool(((logp.double() - want).abs() <= 2.0 ** -24 * want.abs() + 60 * 2.0 ** -24).all())
    first = logp.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.gbdt_class_logp(x, cls, 1.0, logp, None, ws)
        g.gbdt_class_logp(x[:3], cls[:3], 1.0, logp[:3], None, ws)
    for q in range(4):
        logp.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(logp, first), q
        g.gbdt_class_logp(x[1:], cls[1:], 1.0, logp[1:], None, ws)
        assert torch.equal(logp, first), q
    assert g.gbdt_read_error(ws) == 0
