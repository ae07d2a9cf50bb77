"""A seven-class policy that learns from its own draws, then from preferences, and
a router that sends rows to boosted ensembles.

The policy is a linear model over rows: classes are drawn with
gbdt_sample_classes, rewarded, and the weights follow the gradient of the scores
that gbdt_policy_step gives, with a KL term towards the first policy.  The
preference part does the same from pairs of row sequences.  The router chooses two
of four ensembles a row, each ensemble answers for its own rows (gbdt_route_lists
says which), the answers are mixed with the weights, and the router learns by the
gradient of the weights.

Run: python examples/learn_from_draws.py [rows] [steps]
"""
import os
import sys

import numpy as np
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import histogram_split_finding_amd as g  # noqa: E402

CLASSES, FEATURES, EXPERTS, CHOSEN = 7, 54, 4, 2


def policy(rows=20000, steps=40, seed=0, device="cuda"):
    """(mean reward of each step's draws, preference loss of each step)"""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    x = torch.randn(rows, FEATURES, device=device, generator=gen)
    best = (x @ torch.randn(FEATURES, CLASSES, device=device, generator=gen)).argmax(1)
    ws = g.new_workspace(g.gbdt_preference_workspace_bytes(rows, CLASSES), device)
    f = lambda *s: torch.empty(*s, device=device)  # noqa: E731
    weights = torch.zeros(FEATURES, CLASSES, device=device)
    classes, old, ref = torch.empty(rows, dtype=torch.int32, device=device), f(rows), f(rows)
    loss, grad, first = f(rows), f(rows, CLASSES), x @ weights
    rewards = []
    for _ in range(steps):
        scores = x @ weights
        u = torch.rand(rows, device=device, generator=gen)
        # (all classes kept, temperature 1: old is then what the policy's ratio is to)
        g.gbdt_sample_classes(scores, u, None, None, None, None, classes, old, ws)
        reward = (classes == best).float()
        g.gbdt_class_logp(first, classes, 1.0, ref, None, ws)
        for _ in range(2):  # two steps on the same draws: the second one's ratios are not 1
            g.gbdt_policy_step(x @ weights, classes, 1.0, old, ref, reward - reward.mean(), None, 0.2, 0.2, 0.01, loss,
                               None, grad, ws)
            weights -= (x.t() @ grad) * (1.0 / rows)
        rewards.append(reward.mean())
    # pairs of sequences of eight rows: the best classes against drawn ones, on the same rows
    pairs = rows // 16
    both = x[: 8 * pairs].view(pairs, 1, 8, FEATURES).expand(pairs, 2, 8, FEATURES).reshape(-1, FEATURES)
    named = torch.stack([best.int().view(-1)[: 8 * pairs].view(pairs, 8), classes[: 8 * pairs].view(pairs, 8)], 1)
    named, offsets = named.reshape(-1).contiguous(), torch.arange(0, 16 * pairs + 1, 8, device=device)
    n = both.shape[0]
    ref2, ploss, pgrad, margin = f(n), f(pairs), f(n, CLASSES), f(pairs, 2)
    g.gbdt_class_logp(both @ weights, named, 1.0, ref2, None, ws)
    losses = []
    for _ in range(steps):
        g.gbdt_preference_step(both @ weights, named, 1.0, offsets, ref2, None, 0.5, 0.0, False, ploss, margin, pgrad,
                               ws)
        weights -= (both.t() @ pgrad) * (4.0 / pairs)
        losses.append(ploss.mean())
    g._check(g.gbdt_read_error(ws), "learn_from_draws")
    return [r.item() for r in rewards], [p.item() for p in losses]


def router(rows=8000, steps=20, seed=0, device="cuda"):
    """(mean squared error of the mixture at each step, the experts' shares of the rows)"""
    rng = np.random.default_rng(seed)
    bins = rng.integers(0, 32, (rows, 8)).astype(np.uint8)
    region = bins[:, 0].astype(int) // 8
    label = bins[np.arange(rows), 1 + region].astype(np.float32) / 16.0
    params = g.make_params(max_depth=4)
    experts = []
    for e in range(EXPERTS):  # an ensemble for each region of the first feature
        mine = region == e
        ds = g.Dataset(bins[mine], label[mine], [32] * 8, device)
        experts.append(g.Booster(ds, params, device=device).train(5))
    x = torch.nn.functional.one_hot(torch.from_numpy(region), EXPERTS).float().to(device)
    x = x + 0.3 * torch.randn(rows, EXPERTS, device=device)
    gate, y = torch.zeros(EXPERTS, EXPERTS, device=device), torch.from_numpy(label).to(device)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(rows, EXPERTS), device)
    classes = torch.empty(rows, CHOSEN, dtype=torch.int32, device=device)
    weights, grad = torch.empty(rows, CHOSEN, device=device), torch.empty(rows, EXPERTS, device=device)
    offsets = torch.empty(EXPERTS + 1, dtype=torch.int32, device=device)
    order, place = torch.empty(rows * CHOSEN, dtype=torch.int32, device=device), torch.empty_like(classes)
    bias = torch.zeros(EXPERTS, device=device)
    routing = g.make_routing(CHOSEN, renormalise=True)
    errors = []
    for _ in range(steps):
        scores = x @ gate
        g.gbdt_route_classes(scores, routing, bias, classes, weights, ws)
        g.gbdt_route_lists(classes, EXPERTS, offsets, order, place, ws)
        cut = offsets.tolist()
        answers = torch.empty(rows * CHOSEN, device=device)
        for e, booster in enumerate(experts):  # each answers for its own rows
            own = order[cut[e]:cut[e + 1]].long() // CHOSEN
            if own.numel():
                held = g.Dataset(bins[own.cpu().numpy()], label[own.cpu().numpy()], [32] * 8, device)
                answers[cut[e]:cut[e + 1]] = booster.predict(held.X).float()
        answers = answers[place.long()]
        off = (weights * answers).sum(1) - y
        errors.append((off * off).mean())
        g.gbdt_route_grad(scores, routing, classes, 2.0 * off[:, None] * answers, grad, ws)
        gate -= (x.t() @ grad) * (20.0 / rows)
        counts = (offsets[1:] - offsets[:-1]).float()
        bias += 0.02 * torch.sign(counts.mean() - counts)  # experts with fewer rows get more
    g._check(g.gbdt_read_error(ws), "learn_from_draws")
    return [e.item() for e in errors], (counts / counts.sum()).tolist()


if __name__ == "__main__":
    args = [int(a) for a in sys.argv[1:3]]
    rewards, losses = policy(*args)
    print("reward %.3f -> %.3f, preference loss %.4f -> %.4f" % (rewards[0], rewards[-1], losses[0], losses[-1]))
    errors, shares = router()
    print("error of the routed ensembles %.4f -> %.4f, shares %s" % (errors[0], errors[-1], shares))
