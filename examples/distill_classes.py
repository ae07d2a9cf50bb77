"""A student of seven classes trained on a teacher's records, and labels drawn
from it.

The teacher scores rows once; what is kept of a row is its record (the first
two classes, their scores, the mass of the rest).  The student is a linear
model: its class scores are a product, the loss and the gradient of the scores
come from one call, and the gradient of its weights is a product again.

Run: python examples/distill_classes.py [rows] [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import histogram_split_finding_amd as g  # noqa: E402

CLASSES, FEATURES, LISTED, T = 7, 54, 2, 2.0


def run(rows=20000, steps=60, seed=0, device="cuda"):
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    x = torch.randn(rows, FEATURES, device=device, generator=gen)
    teacher = torch.randn(FEATURES, CLASSES, device=device, generator=gen) * 0.5
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(rows, CLASSES), device)

    values = torch.empty(rows, LISTED, device=device)
    classes = torch.empty(rows, LISTED, dtype=torch.int32, device=device)
    rest = torch.empty(rows, device=device)
    g.gbdt_top_scores(x @ teacher, LISTED, T, values, classes, rest, ws)

    weights = torch.zeros(FEATURES, CLASSES, device=device)
    loss = torch.empty(rows, device=device)
    grad = torch.empty(rows, CLASSES, device=device)
    history = []
    for _ in range(steps):
        g.gbdt_distill_step(x @ weights, values, classes, rest, T, None, loss, grad, ws)
        weights -= (x.t() @ grad) * (0.5 / rows)
        history.append(loss.mean())

    labels = torch.empty(rows, dtype=torch.int32, device=device)
    u = torch.rand(rows, device=device, generator=gen)
    top_p = torch.full((rows,), 0.9, device=device)
    g.gbdt_sample_classes(x @ weights, u, None, None, top_p, None, labels, None, ws)
    g._check(g.gbdt_read_error(ws), "distill_classes")
    agree = (labels.long() == (x @ teacher).argmax(1)).float().mean().item()
    return [h.item() for h in history], agree


if __name__ == "__main__":
    args = [int(a) for a in sys.argv[1:3]]
    losses, agree = run(*args)
    print("loss %.4f -> %.4f, labels drawn from the student equal the teacher's first class in %.1f%% of rows"
          % (losses[0], losses[-1], 100.0 * agree))
