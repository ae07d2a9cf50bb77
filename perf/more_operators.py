"""The operators that learn from drawn classes and that route rows, as they are measured.

Rows of class scores again.  A class of each row has a log-probability under
softmax(x / T), with its gradient; a clipped policy loss with a KL term and a
preference loss on pairs of row sequences are taken from these, with the
gradient of the scores; and a router's rows are sent to experts: softmax or
sigmoid values, a bias that only the choice sees, groups, top-k, renormalised
weights, the experts' lists of rows, and the gradient of the weights.  `run`
computes them with elementary torch operations where `own` is false and with
the framework's calls where it is true.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
CLIP_LOW, CLIP_HIGH, KL = 0.2, 0.28, 0.04
BETA, SMOOTHING = 0.1, 0.05


# ------------------------------------------------------------------- cases --

def listed():
    rows = dict(pad=0, masked=False, ignored=0.1)
    return [
        # the log-probability of one request's class in a row of a large class set: latency
        dict(name="logp_one_row", op="logp", n=1, C=131072, dtype="bf16", T=1.0, **{**rows, "ignored": 0.0}),
        # the backward pass of log-probabilities, rows apart by a padded stride
        dict(name="logp_grad_strided", op="logp_grad", n=2048, C=50001, dtype="f32", T=1.0, **{**rows, "pad": 15}),
        # an online policy's small batch: latency counts
        dict(name="policy_step_small", op="policy_step", n=32, C=4099, dtype="f32", T=1.0, **rows),
        # one round over a seven-class policy at the 581,012-row workload's row count
        dict(name="policy_step_7_classes", op="policy_step", n=581012, C=7, dtype="f32", T=1.0, **rows),
        # a training batch over a large class set, padded classes masked, loss and gradient in one call
        dict(name="policy_step_many_rows", op="policy_step", n=4096, C=131072, dtype="bf16", T=1.0,
             **{**rows, "masked": True}),
        # the forward pass alone, odd row length
        dict(name="policy_loss_odd_rows", op="policy_loss", n=1000, C=32003, dtype="f16", T=0.8, **rows),
        # a handful of short pairs: latency counts
        dict(name="preference_step_small", op="pref_step", n=100, C=1000, dtype="f16", T=1.0, pairs=4, average=False,
             **rows),
        # a training batch of ragged pairs over a large class set
        dict(name="preference_step_many", op="pref_step", n=4096, C=65537, dtype="bf16", T=1.0, pairs=32, average=False,
             **rows),
        # one row sent to its experts while it is answered: latency
        dict(name="route_one_row", op="route", n=1, E=256, dtype="f32", k=8, score="sigmoid", renorm=True, bias=True,
             groups=8, kept=4, top=2, masked=False),
        # a batch of rows sent to experts in groups, balanced by a bias
        dict(name="route_groups", op="route", n=16384, E=256, dtype="f32", k=8, score="sigmoid", renorm=True, bias=True,
             groups=8, kept=4, top=2, masked=False),
        # a long batch over fewer experts, weights as the softmax has them, an expert out of service
        dict(name="route_softmax", op="route", n=65536, E=60, dtype="bf16", k=4, score="softmax", renorm=False,
             bias=False, groups=1, kept=1, top=1, masked=True),
        # the backward pass of the routing weights
        dict(name="route_grad", op="route_grad", n=65536, E=128, dtype="f32", k=6, score="softmax", renorm=False,
             bias=False, groups=1, kept=1, top=1, masked=False),
    ]


def spread(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["logp", "logp_grad", "policy_loss", "policy_step", "pref_loss", "pref_step", "route", "route_grad"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("route", "route_grad"):
        size, groups = spread(rng, 1, 48), rng.choice([1, 1, 2, 4, 7, 8])
        E = max(2, size * groups)
        groups = groups if E % groups == 0 else 1
        kept = rng.randint(1, groups)
        k = min(spread(rng, 1, 16), kept * (E // groups))
        return dict(op=op, n=spread(rng, 1, min(65536, (1 << 23) // E)), E=E, dtype=dtype, k=k,
                    score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.6, bias=rng.random() < 0.5,
                    groups=groups, kept=kept, top=rng.choice([1, 2]), masked=rng.random() < 0.3)
    C = spread(rng, 2, 131072)
    n = spread(rng, 1, min(600000, max(1, (1 << 26) // C)))
    case = dict(op=op, n=n, C=C, dtype=dtype, T=rng.choice([0.7, 1.0, 1.0, 1.5]), pad=rng.choice([0, 0, 0, 1, 8, 13]),
                masked=rng.random() < 0.3, ignored=rng.choice([0.0, 0.1, 0.5]))
    if op in ("pref_loss", "pref_step"):
        case["pairs"] = spread(rng, 1, min(4096, max(1, n // 4)))
        case["average"] = rng.random() < 0.3
    return case


def work(case):
    n, es, op = case["n"], BYTES[case["dtype"]], case["op"]
    if op == "route":
        E, k = case["E"], case["k"]
        return {"bytes": n * E * es + 16 * n * k + 4 * (E + 1) + 4 * E * case["bias"], "flops": 12 * n * E}
    if op == "route_grad":
        E, k = case["E"], case["k"]
        # renormalised weights and sigmoid values depend on the chosen experts' scores alone
        read = n * E * es if case["score"] == "softmax" and not case["renorm"] else n * k * es
        return {"bytes": read + n * E * es + 8 * n * k, "flops": 4 * n * E}
    rows = n * case["C"] * es
    read = rows * (1.0 - case["ignored"])  # a row that names no class is not read
    elements = n * case["C"] * (1.0 - case["ignored"])
    if op == "logp":
        return {"bytes": read + 16 * n, "flops": 4 * elements}
    if op == "logp_grad":
        return {"bytes": read + rows + 16 * n, "flops": 4 * elements}
    per_row = 16 * n if op in ("policy_loss", "policy_step") else 4 * n
    if op in ("policy_loss", "pref_loss"):
        return {"bytes": read + 20 * n + per_row, "flops": 4 * elements}
    return {"bytes": read + rows + 12 * n + per_row, "flops": 8 * elements}


# ------------------------------------------------------------------ inputs --

def score_rows(case, gen, n, C):
    """Scores as a model over many classes gives them: a wide bulk, a few
    classes far above it, spread that differs from row to row; the last eighth
    of the classes -inf where the class set is padded."""
    x = torch.randn(n, C, device="cuda", generator=gen)
    x *= 1.0 + 1.5 * torch.rand(n, 1, device="cuda", generator=gen)
    hot = min(24, C // 4)
    if hot > 0:
        # (no class twice: the same seed gives the same bits)
        at = torch.randint(0, C, (n, 1), device="cuda", generator=gen)
        at = (at + C // hot * torch.arange(hot, device="cuda")) % C
        x.scatter_add_(1, at, 4.0 + 4.0 * torch.randn(n, hot, device="cuda", generator=gen).abs())
    if case["masked"] and C >= 16:
        x[:, C - C // 8:] = float("-inf")
    return x


def strided(case, x):
    """x in the case's type, in rows that lie `pad` elements further apart."""
    dtype = DTYPES[case["dtype"]]
    if case["pad"] == 0:
        return x.to(dtype)
    out = torch.zeros(x.shape[0], x.shape[1] + case["pad"], dtype=dtype, device="cuda")[:, :x.shape[1]]
    out.copy_(x)
    return out


def nearby(x, gen, by, T, classes):
    """Log-probabilities of the classes under scores that differ from x a little."""
    z = torch.randn(x.shape, device="cuda", generator=gen).mul_(by).add_(x).div_(T)
    top = z.amax(1)
    at = z.gather(1, classes[:, None])[:, 0]
    return at - top - z.sub_(top[:, None]).exp_().sum(1).log()


def prepare_route(case, gen):
    n, E = case["n"], case["E"]
    # experts that the data favours, some of them often
    x = torch.randn(n, E, device="cuda", generator=gen) + 0.7 * torch.randn(1, E, device="cuda", generator=gen)
    if case["masked"]:
        x[:, E // 2] = float("-inf")
    k = case["k"]
    state = dict(case=case, op=case["op"], scores=x.to(DTYPES[case["dtype"]]))
    state["bias"] = 0.1 * torch.randn(E, device="cuda", generator=gen) if case["bias"] else None
    state["classes"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
    state["weights"] = torch.empty(n, k, device="cuda")
    state["offsets"] = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    state["order"] = torch.full((n * k,), -1, dtype=torch.int32, device="cuda")
    state["place"] = torch.empty(n, k, dtype=torch.int32, device="cuda")
    if case["op"] == "route_grad":  # the forward pass's choice is in hand
        state["classes"] = plain_route(state)[0].contiguous()
        state["dweights"] = torch.randn(n, k, device="cuda", generator=gen)
        state["grad"] = torch.empty_like(state["scores"])
    if own:
        import histogram_split_finding_amd as g
        state["routing"] = g.make_routing(k, sigmoid=case["score"] == "sigmoid", renormalise=case["renorm"],
                                          scale=2.5, n_groups=case["groups"], groups_kept=case["kept"],
                                          group_top=case["top"])
        state["ws"] = g.new_workspace(g.gbdt_scores_workspace_bytes(n, E))
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    if case["op"] in ("route", "route_grad"):
        return prepare_route(case, gen)
    n, C, T, op = case["n"], case["C"], case["T"], case["op"]
    x = score_rows(case, gen, n, C)
    state = dict(case=case, op=op, scores=strided(case, x), n=n, C=C, T=T)
    # the classes as the policy of some steps ago drew them
    u = torch.rand(n, C, device="cuda", generator=gen).clamp_(1e-30, 1.0)
    classes = u.log_().neg_().log_().neg_().add_(x / T).argmax(1)
    del u
    old = nearby(x, gen, 0.1, T, classes)
    ref = nearby(x, gen, 0.3, T, classes)
    skip = torch.rand(n, device="cuda", generator=gen) < case["ignored"]
    state["classes"] = torch.where(skip, -torch.ones_like(classes), classes).to(torch.int32)
    state["ref"] = ref
    if op in ("policy_loss", "policy_step"):
        state["old"] = old
        state["advantage"] = torch.randn(n, device="cuda", generator=gen)
        state["weight"] = 0.5 + torch.rand(n, device="cuda", generator=gen)
    if op in ("pref_loss", "pref_step"):
        # 2 x pairs ragged sequences of rows, and a few rows behind the last
        lengths = 0.3 + torch.rand(2 * case["pairs"], device="cuda", generator=gen, dtype=torch.float64)
        ends = (torch.cumsum(lengths, 0) / lengths.sum() * (n - n // 50)).round().long()
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), ends])
        state["weight"] = 0.5 + torch.rand(case["pairs"], device="cuda", generator=gen)
        state["rewards"] = torch.empty(case["pairs"], 2, device="cuda")
        state["loss"] = torch.empty(case["pairs"], device="cuda")
    else:
        state["loss"] = torch.empty(n, device="cuda")
    # (rows behind the last sequence stay as they are)
    state["logp"] = torch.zeros(n, device="cuda")
    state["dlogp"] = torch.zeros(n, device="cuda")
    state["stats"] = torch.zeros(n, 2, device="cuda")
    if op.endswith("step") or op == "logp_grad":
        shape, apart = state["scores"].shape, state["scores"].stride()
        state["grad"] = torch.empty_strided(shape, apart, dtype=state["scores"].dtype, device="cuda").zero_()
    if op == "logp_grad":  # the forward pass's statistics are in hand
        state["stats"] = plain_rows(state)["stats"].float()
        state["dlogp"] = torch.randn(n, device="cuda", generator=gen)
    if own:
        import histogram_split_finding_amd as g
        size = g.gbdt_preference_workspace_bytes if op == "pref_step" else g.gbdt_scores_workspace_bytes
        state["ws"] = g.new_workspace(size(n, C))
    return state


# ------------------------------------------------------------- plain forms --

def plain_rows(state):
    """Of each row: whether it counts, its class, the other classes' largest
    score and sum, and the logarithm of the odds against the class.  The values
    of a row are few and their differences small: these in 64 bits; where a
    ratio next to the clip's border decides about a whole row, the exponentials
    too."""
    x, T = state["scores"].float(), state["T"]
    if state["op"] in ("policy_loss", "policy_step"):
        x = x.double()
    named = (state["classes"] >= 0) & (x.amax(1) > float("-inf"))
    at = state["classes"].clamp(min=0).long()[:, None]
    mine = x.gather(1, at)[:, 0].double()
    x = x.scatter(1, at, float("-inf"))  # (a copy)
    top = x.amax(1, keepdim=True)
    base = torch.where(top > float("-inf"), top, torch.zeros_like(top))
    others = torch.exp((x - base) / T)
    total = others.sum(1, dtype=torch.float64)
    stats = torch.stack([top[:, 0].double(), total], 1)
    odds = (top[:, 0].double() - mine) / T + torch.log(total)
    logp = -(torch.clamp(odds, min=0.0) + torch.log1p(torch.exp(-odds.abs())))
    zero = torch.zeros_like(odds)
    return dict(named=named, at=at, others=others, total=total, odds=odds,
                logp=torch.where(named, logp, zero), stats=torch.where(named[:, None], stats, zero[:, None]))


def plain_logp_grad(state, rows, dlogp):
    """dlogp / T times (1 at the class, else 0) - p, p from the odds against the class."""
    against = 1.0 / (1.0 + torch.exp(-rows["odds"]))
    factor = dlogp.double() / state["T"] * against
    factor = torch.where(rows["named"] & (dlogp != 0) & (against == against), factor, torch.zeros_like(factor))
    share = torch.where(rows["total"] > 0, factor / rows["total"], torch.zeros_like(factor))
    grad = rows["others"] * (-share).to(rows["others"].dtype)[:, None]
    grad.scatter_(1, rows["at"], factor.to(grad.dtype)[:, None])
    return grad.to(state["scores"].dtype)


def plain_policy(state, rows):
    logp, adv = rows["logp"], state["advantage"].double()
    ratio = torch.exp(logp - state["old"].double())
    clipped = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    away = state["ref"].double() - logp
    loss = -torch.minimum(ratio * adv, clipped * adv) + KL * (torch.exp(away) - away - 1.0)
    follows = ~(((adv > 0) & (ratio > 1.0 + CLIP_HIGH)) | ((adv < 0) & (ratio < 1.0 - CLIP_LOW)))
    slope = torch.where(follows, -adv * ratio, torch.zeros_like(ratio)) + KL * (1.0 - torch.exp(away))
    zero = torch.zeros_like(loss)
    loss = torch.where(rows["named"], loss, zero)
    dlogp = torch.where(rows["named"], slope * state["weight"].double(), zero)
    return loss.float(), logp.float(), dlogp.float()


def plain_preference(state, rows):
    cut, n = state["offsets"], state["n"]
    lead = rows["logp"] - state["ref"].double()
    lead = torch.where(rows["named"], lead, torch.zeros_like(lead))
    run = torch.cat([torch.zeros_like(lead[:1]), torch.cumsum(lead, 0)])
    total = run[cut[1:]] - run[cut[:-1]]
    count = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), torch.cumsum(rows["named"].long(), 0)])
    count = (count[cut[1:]] - count[cut[:-1]]).clamp(min=1)
    per = 1.0 / count.double() if state["case"]["average"] else torch.ones_like(total)
    rewards = (BETA * total * per).view(-1, 2)
    z = rewards[:, 0] - rewards[:, 1]
    tail = torch.log1p(torch.exp(-z.abs()))
    loss = (1.0 - SMOOTHING) * ((-z).clamp(min=0.0) + tail) + SMOOTHING * (z.clamp(min=0.0) + tail)
    slope = (SMOOTHING - 1.0) / (1.0 + torch.exp(z)) + SMOOTHING / (1.0 + torch.exp(-z))
    slope = slope * state["weight"].double() * BETA
    slope = torch.stack([slope, -slope], 1).view(-1) * per
    row = torch.arange(n, device="cuda")
    inside = (row >= cut[0]) & (row < cut[-1])
    seq = (torch.searchsorted(cut, row, right=True) - 1).clamp(0, slope.numel() - 1)
    dlogp = torch.where(inside & rows["named"], slope[seq], torch.zeros_like(lead))
    return loss.float(), rewards.float(), dlogp.float(), inside


def plain_route(state):
    case = state["case"]
    E, k, groups = case["E"], case["k"], case["groups"]
    # which value is larger decides: in 64 bits
    x = state["scores"].double()
    live = x > float("-inf")
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    by_value = state["bias"] is not None or (groups > 1 and case["top"] == 2)
    v = x
    if by_value:
        v = s if state["bias"] is None else s + state["bias"].double()[None]
        v = torch.where(live, v, torch.full_like(v, float("-inf")))
    if groups > 1:
        part = v.view(-1, groups, E // groups)
        best = torch.sort(part, dim=2, descending=True).values
        rank = best[:, :, 0]
        if case["top"] == 2 and E // groups > 1:
            rank = rank + torch.where(best[:, :, 1] > float("-inf"), best[:, :, 1], torch.zeros_like(rank))
        first = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :case["kept"]]
        keep = torch.zeros_like(rank).scatter_(1, first, 1.0) > 0
        v = torch.where(keep[:, :, None], part, torch.full_like(part, float("-inf"))).view(-1, E)
    v, classes = torch.sort(v, dim=1, descending=True, stable=True)
    v, classes = v[:, :k], classes[:, :k]
    w = torch.where(v > float("-inf"), s.gather(1, classes), torch.zeros_like(v))
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    classes = torch.where(v > float("-inf"), classes, torch.full_like(classes, -1)).to(torch.int32)
    return classes, (2.5 * w).float()


def plain_lists(state, classes):
    """The experts' lists of places in `classes`, one after another, each in ascending order."""
    E = state["case"]["E"]
    flat = classes.reshape(-1).long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    order = torch.sort(key, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), torch.cumsum(counts[:E], 0)])
    position = torch.arange(flat.numel(), device="cuda")
    place = torch.empty_like(position).scatter_(0, order, position)
    place = torch.where(flat >= 0, place, torch.full_like(place, -1)).view(classes.shape)
    order = torch.where(position < offsets[E], order, torch.full_like(order, -1))
    return offsets.to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def plain_route_grad(state):
    case, dw = state["case"], state["dweights"]
    x = state["scores"].float()
    named = state["classes"] >= 0
    at = state["classes"].clamp(min=0).long()
    zero = torch.zeros_like(dw)
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        s = torch.exp(x - torch.where(top > float("-inf"), top, torch.zeros_like(top)))
        s = s / s.sum(1, keepdim=True).clamp(min=1e-30)
    mine = torch.where(named, s.gather(1, at), zero)
    dw = torch.where(named, dw, zero)
    if case["renorm"]:
        total = mine.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.full_like(total, float("inf")))
        ds = 2.5 * (dw - (dw * mine).sum(1, keepdim=True) / total) / total
    else:
        ds = 2.5 * dw
    chosen = ds * mine * (1.0 - mine) if case["score"] == "sigmoid" else ds * mine
    grad = torch.zeros_like(x).scatter_add_(1, at, torch.where(named, chosen, zero))
    if case["score"] == "softmax" and not case["renorm"]:
        grad = grad - s * (ds * mine).sum(1, keepdim=True)
    return grad.to(state["scores"].dtype)


# --------------------------------------------------------------------- run --

def run_own(state):
    import histogram_split_finding_amd as g
    s, op = state, state["op"]
    x, ws = s["scores"], s["ws"]
    if op == "route":
        g.gbdt_route_classes(x, s["routing"], s["bias"], s["classes"], s["weights"], ws)
        g.gbdt_route_lists(s["classes"], s["case"]["E"], s["offsets"], s["order"], s["place"], ws)
        return s["classes"], s["weights"], s["offsets"], s["order"], s["place"]
    if op == "route_grad":
        g.gbdt_route_grad(x, s["routing"], s["classes"], s["dweights"], s["grad"], ws)
        return s["grad"]
    T, classes = s["T"], s["classes"]
    if op == "logp":
        g.gbdt_class_logp(x, classes, T, s["logp"], s["stats"], ws)
        return s["logp"], s["stats"]
    if op == "logp_grad":
        g.gbdt_class_logp_grad(x, classes, T, s["stats"], s["dlogp"], s["grad"], ws)
        return s["grad"]
    if op in ("policy_loss", "policy_step"):
        policy = (s["old"], s["ref"], s["advantage"], s["weight"], CLIP_LOW, CLIP_HIGH, KL)
        if op == "policy_loss":
            g.gbdt_policy_loss(x, classes, T, *policy, s["loss"], s["logp"], s["dlogp"], s["stats"], ws)
            return s["loss"], s["logp"], s["dlogp"], s["stats"]
        g.gbdt_policy_step(x, classes, T, *policy, s["loss"], s["logp"], s["grad"], ws)
        return s["loss"], s["logp"], s["grad"]
    pairs = (s["offsets"], s["ref"], s["weight"], BETA, SMOOTHING, s["case"]["average"])
    if op == "pref_loss":
        g.gbdt_preference_loss(x, classes, T, *pairs, s["loss"], s["rewards"], s["logp"], s["dlogp"], s["stats"], ws)
        return s["loss"], s["rewards"], s["logp"], s["dlogp"], s["stats"]
    g.gbdt_preference_step(x, classes, T, *pairs, s["loss"], s["rewards"], s["grad"], ws)
    return s["loss"], s["rewards"], s["grad"]


def run(state):
    if own:
        return run_own(state)
    op = state["op"]
    if op == "route":
        classes, weights = plain_route(state)
        return (classes, weights) + plain_lists(state, classes)
    if op == "route_grad":
        return plain_route_grad(state)
    rows = plain_rows(state)
    if op == "logp":
        return rows["logp"].float(), rows["stats"].float()
    if op == "logp_grad":
        return plain_logp_grad(state, rows, state["dlogp"])
    if op in ("policy_loss", "policy_step"):
        loss, logp, dlogp = plain_policy(state, rows)
        if op == "policy_loss":
            return loss, logp, dlogp, rows["stats"].float()
        return loss, logp, plain_logp_grad(state, rows, dlogp)
    loss, rewards, dlogp, inside = plain_preference(state, rows)
    if op == "pref_loss":
        zero = torch.zeros_like(dlogp)
        logp = torch.where(inside, rows["logp"].float(), zero)
        stats = torch.where(inside[:, None], rows["stats"].float(), zero[:, None])
        return loss, rewards, logp, dlogp, stats
    return loss, rewards, plain_logp_grad(state, rows, dlogp)


# --------------------------------------------------------------- in 64 bits --

def exact_logp(state, lo, hi):
    """Log-probabilities of all classes of rows [lo, hi), and what goes with the named one."""
    z = state["scores"][lo:hi].double()
    cls = state["classes"][lo:hi].long()
    counts = (cls >= 0) & (z > -math.inf).any(1)
    spot = torch.where(counts, cls, torch.zeros_like(cls))[:, None]
    rest = z.clone()
    rest.scatter_(1, spot, -math.inf)
    m = rest.max(1).values
    finite = torch.where(m > -math.inf, m, torch.zeros_like(m))
    others = torch.exp((rest - finite[:, None]) / state["T"]).sum(1)
    z /= state["T"]
    lp = z - torch.where(counts, torch.logsumexp(z, 1), torch.zeros_like(m))[:, None]
    mine = torch.where(counts, lp.gather(1, spot)[:, 0], torch.zeros_like(m))
    stats = torch.stack([m, others], 1) * 1.0
    stats[~counts] = 0.0
    return lp, spot, counts, mine, stats


def exact_rows(state, slope_of):
    """(logp, stats, slope, gradient) with the slope of a row's loss in its logp from slope_of, by parts of the rows."""
    n, C = state["n"], state["C"]
    step = max(1, (1 << 27) // C)
    out = []
    for lo in range(0, n, step):
        lp, spot, counts, mine, stats = exact_logp(state, lo, min(n, lo + step))
        grad = None
        if slope_of is not None:
            slope = torch.where(counts, slope_of[lo:lo + step], torch.zeros_like(mine))
            hit = torch.zeros_like(lp)
            hit.scatter_(1, spot, 1.0)
            grad = (hit - torch.exp(lp)) * (slope / state["T"])[:, None]
            grad[slope == 0] = 0.0
        out.append((mine, stats, counts, grad))
    logp, stats, counts = (torch.cat([o[j] for o in out]) for j in range(3))
    return logp, stats, counts, (None if slope_of is None else torch.cat([o[3] for o in out]))


def exact_policy(state, logp, counts):
    A, old, ref, w = (state[k].double() for k in ("advantage", "old", "ref", "weight"))
    r = torch.exp(logp - old)
    lo, hi = 1.0 - CLIP_LOW, 1.0 + CLIP_HIGH
    plain, limited = r * A, torch.clamp(r, lo, hi) * A
    kl = torch.expm1(ref - logp) - (ref - logp)
    loss = KL * kl - torch.where(plain <= limited, plain, limited)
    slope = torch.where(plain <= limited, -plain, torch.zeros_like(A)) - KL * torch.expm1(ref - logp)
    return loss * counts, slope * w * counts


def exact_pairs(state, logp, counts):
    cut = state["offsets"].tolist()
    gain = torch.where(counts, logp - state["ref"].double(), torch.zeros_like(logp)).cpu()
    counted = counts.cpu()
    mean = state["case"]["average"]
    slope = torch.zeros_like(gain)
    loss, rewards = [], []
    w = state["weight"].double().tolist()
    for p in range(state["case"]["pairs"]):
        a, b, c = cut[2 * p:2 * p + 3]
        share = [1.0 / max(1, int(counted[u:v].sum())) if mean else 1.0 for u, v in ((a, b), (b, c))]
        won, lost = BETA * float(gain[a:b].sum()) * share[0], BETA * float(gain[b:c].sum()) * share[1]
        z = won - lost
        up, down = math.log1p(math.exp(-abs(z))) + max(-z, 0.0), math.log1p(math.exp(-abs(z))) + max(z, 0.0)
        loss.append((1.0 - SMOOTHING) * up + SMOOTHING * down)
        rewards.append((won, lost))
        dz = SMOOTHING * math.exp(-up) - (1.0 - SMOOTHING) * math.exp(-down)
        slope[a:b] = w[p] * BETA * dz * share[0]
        slope[b:c] = -w[p] * BETA * dz * share[1]
    slope = torch.where(counted, slope, torch.zeros_like(slope)).cuda()
    return (torch.tensor(loss, dtype=torch.float64, device="cuda"),
            torch.tensor(rewards, dtype=torch.float64, device="cuda"), slope, (cut[0], cut[-1]))


def exact_values(state):
    """Experts' softmax or sigmoid values, -inf scores 0."""
    x = state["scores"].double()
    if state["case"]["score"] == "sigmoid":
        return x, torch.sigmoid(x)
    lse = torch.logsumexp(x, 1, keepdim=True)
    return x, torch.exp(x - torch.where(lse > -math.inf, lse, torch.zeros_like(lse)))


def exact_choice(state):
    """One class after the other: the best that is left."""
    case = state["case"]
    E, G, k = case["E"], case["groups"], case["k"]
    x, s = exact_values(state)
    n = x.shape[0]
    v = x.clone()
    if state["bias"] is not None or (G > 1 and case["top"] == 2):
        v = s + (0.0 if state["bias"] is None else state["bias"].double())
        v[x == -math.inf] = -math.inf

    def best(t):  # (value, the lowest index that has it)
        top = t.max(1, keepdim=True).values
        return top[:, 0], (t == top).to(torch.int8).argmax(1)

    rows = torch.arange(n, device="cuda")
    if G > 1:
        size = E // G
        ranks = []
        for q in range(G):
            part = v[:, q * size:(q + 1) * size].clone()
            first, at = best(part)
            if case["top"] == 2 and size > 1:
                part[rows, at] = -math.inf
                second = part.max(1).values
                first = torch.where(second > -math.inf, first + second, first)
            ranks.append(first)
        rank = torch.stack(ranks, 1)
        keep = torch.zeros(n, G, dtype=torch.bool, device="cuda")
        for _ in range(case["kept"]):
            left = torch.where(keep, torch.full_like(rank, -math.inf), rank)
            # (of groups with nothing in them any may be kept)
            _, at = best(left)
            keep[rows, at] = True
        v[~keep.repeat_interleave(size, 1)] = -math.inf
    chosen, weights = [], []
    for _ in range(k):
        top, at = best(v)
        there = top > -math.inf
        chosen.append(torch.where(there, at, torch.full_like(at, -1)))
        weights.append(torch.where(there, s[rows, at], torch.zeros_like(top)))
        v[rows, at] = -math.inf
    w = torch.stack(weights, 1)
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return torch.stack(chosen, 1).to(torch.int32), 2.5 * w


def exact_lists(state, chosen):
    E = state["case"]["E"]
    flat = chosen.reshape(-1).cpu()
    lists = [torch.nonzero(flat == e)[:, 0] for e in range(E)]
    offsets = torch.tensor([0] + [len(q) for q in lists]).cumsum(0)
    listed_ones = torch.cat(lists)
    order, place = torch.full_like(flat, -1), torch.full_like(flat, -1)
    order[:len(listed_ones)] = listed_ones.to(torch.int32)
    place[listed_ones] = torch.arange(len(listed_ones), dtype=torch.int32)
    return offsets.to(torch.int32).cuda(), order.cuda(), place.view(chosen.shape).cuda()


def exact_route_grad(state):
    """The weights' derivative as a matrix product: J = dw / ds, then ds / dx."""
    case = state["case"]
    x, s = exact_values(state)
    hit = torch.zeros(x.shape[0], x.shape[1] + 1, dtype=torch.float64, device="cuda")
    cls = state["classes"].long()
    cls = torch.where(cls >= 0, cls, torch.full_like(cls, x.shape[1]))
    up = hit.clone().scatter_(1, cls, state["dweights"].double())[:, :-1]
    hit = hit.scatter_(1, cls, 1.0)[:, :-1]
    ds = 2.5 * up * hit
    if case["renorm"]:
        total = (s * hit).sum(1, keepdim=True)
        safe = torch.where(total > 0, total, torch.ones_like(total))
        ds = hit * (ds / safe - (ds * s).sum(1, keepdim=True) / safe ** 2)
    if case["score"] == "sigmoid":
        return ds * s * (1.0 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True))


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "route":
        chosen, weights = exact_choice(state)
        return (chosen, weights) + exact_lists(state, chosen)
    if op == "route_grad":
        return exact_route_grad(state)
    if op == "logp_grad":
        return exact_rows(state, state["dlogp"].double())[3]
    logp, stats, counts, _ = exact_rows(state, None)
    if op == "logp":
        return logp, stats
    if op in ("policy_loss", "policy_step"):
        loss, slope = exact_policy(state, logp, counts)
        if op == "policy_loss":
            return loss, logp, slope, stats
        return loss, logp, exact_rows(state, slope)[3]
    loss, rewards, slope, (first, last) = exact_pairs(state, logp, counts)
    if op == "pref_loss":
        row = torch.arange(case["n"], device="cuda")
        outside = (row < first) | (row >= last)
        logp, stats = logp.clone(), stats.clone()
        logp[outside], stats[outside] = 0.0, 0.0
        return loss, rewards, logp, slope, stats
    return loss, rewards, exact_rows(state, slope)[3]
