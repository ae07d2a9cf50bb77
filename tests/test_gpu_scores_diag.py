"""Diagnostics of the calls on rows of class scores: a record for each launch."""
import ctypes

import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

TOP, DISTILL, SAMPLE = 16, 17, 18


def kinds_of(work, room=64):
    lib = g.load()
    assert lib.gbdt_diag_enable(room) == 0
    work()
    kinds, ms, n = np.zeros(room, np.int32), np.zeros(room, np.float32), ctypes.c_int32(0)
    rc = lib.gbdt_diag_read(room, kinds.ctypes.data_as(ctypes.c_void_p), ms.ctypes.data_as(ctypes.c_void_p),
                            ctypes.addressof(n))
    lib.gbdt_diag_disable()
    assert rc == 0 and bool((ms[: n.value] >= 0.0).all())
    return kinds[: n.value].tolist()


@pytest.mark.parametrize("C,tops,losses,grads,steps,samples", [
    (7, 1, 1, 1, 1, 1),       # a thread a row
    (400, 1, 1, 1, 1, 2),     # a wave a row; draws look for rows left over
    (9001, 2, 1, 1, 1, 2),
    (70001, 2, 2, 1, 2, 2),   # few long rows: sums of parts first
])
def test_launches(C, tops, losses, grads, steps, samples):
    say("diagnostics: C=%d" % C)
    n = 5
    x, _ = ref.rows(n, C, "f32", C)
    v, c = torch.zeros(n, 3, device=DEV), torch.zeros(n, 3, dtype=torch.int32, device=DEV)
    rest, loss, u = (torch.zeros(n, device=DEV) for _ in range(3))
    stats, grad = torch.zeros(n, 3, device=DEV), torch.zeros(n, C, device=DEV)
    out = torch.zeros(n, dtype=torch.int32, device=DEV)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(n, C))
    assert kinds_of(lambda: g.gbdt_top_scores(x, 3, 1.0, v, c, rest, ws)) == [TOP] * tops
    assert kinds_of(lambda: g.gbdt_distill_loss(x, v, c, rest, 1.0, loss, stats, ws)) == [DISTILL] * losses
    assert kinds_of(lambda: g.gbdt_distill_grad(x, v, c, rest, 1.0, stats, None, grad, ws)) == [DISTILL] * grads
    assert kinds_of(lambda: g.gbdt_distill_step(x, v, c, rest, 1.0, None, loss, grad, ws)) == [DISTILL] * steps
    assert kinds_of(lambda: g.gbdt_sample_classes(x, u, None, None, None, None, out, None, ws)) == [SAMPLE] * samples
    assert g.gbdt_read_error(ws) == 0
