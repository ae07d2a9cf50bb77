"""The operators on rows of class scores, as they are measured.

Three operators: a teacher's row reduced to its record (the top scores, their
classes, the probability mass of the rest), the distillation loss of a
student's rows against such records with its gradient, and the drawing of a
class from a row with temperature, top-k, top-p and min-p.  `run` computes
them with elementary torch operations where `own` is false and with the
framework's calls where it is true.

Scores of a row are ordered by value, descending, ties to the lowest class;
-0 equals +0 and NaN counts as -inf there.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one row of a large class set, reduced while its teacher answers one request: latency
        dict(name="top_one_row", op="top", n=1, C=131072, dtype="bf16", k=64, T=1.0, pad=0, masked=False),
        # a shard of teacher rows reduced to records before training, padded classes masked
        dict(name="top_many_rows", op="top", n=2048, C=131072, dtype="bf16", k=64, T=2.0, pad=0, masked=True),
        # per-row records of a seven-class ensemble's scores at the 581,012-row workload's row count
        dict(name="top_7_classes", op="top", n=581012, C=7, dtype="f32", k=3, T=1.0, pad=0, masked=False),
        # a small batch of an online student: latency counts
        dict(name="step_small", op="step", n=32, C=4099, dtype="f32", k=16, T=2.0, rest=True, pad=0, masked=False),
        # one boosting round's loss and gradients of a seven-class student
        dict(name="step_7_classes", op="step", n=581012, C=7, dtype="f32", k=3, T=2.0, rest=True, pad=0,
             masked=False),
        # a training batch over a large class set, loss and gradient in one call
        dict(name="step_many_rows", op="step", n=4096, C=131072, dtype="bf16", k=64, T=2.0, rest=True, pad=0,
             masked=True),
        # an evaluation pass (forward only), odd row length, teacher renormalised over its list
        dict(name="loss_odd_rows", op="loss", n=1000, C=32003, dtype="f16", k=32, T=1.5, rest=False, pad=0,
             masked=False),
        # the backward pass from the forward's statistics, rows apart by a padded stride
        dict(name="grad_strided_rows", op="grad", n=2048, C=50001, dtype="f32", k=32, T=2.0, rest=True, pad=15,
             masked=False),
        # the draw of one request: latency
        dict(name="sample_one_row", op="sample", n=1, C=131072, dtype="bf16", mode="k_p", pad=0, masked=False),
        # a batch of requests with their own temperatures and filters, no top-k: whole-row masses
        dict(name="sample_many_rows", op="sample", n=1024, C=100003, dtype="bf16", mode="p_min", pad=0,
             masked=False),
        # a serving batch drawn by temperature alone from 32-bit scores
        dict(name="sample_batch", op="sample", n=64, C=65536, dtype="f32", mode="plain", pad=0, masked=True),
        # a label drawn for every row of the seven-class workload
        dict(name="sample_7_classes", op="sample", n=581012, C=7, dtype="f32", mode="mixed", pad=0, masked=False),
    ]


def draw(rng):
    op = rng.choice(["top", "step", "loss", "grad", "sample"])
    C = int(round(math.exp(rng.uniform(math.log(2), math.log(131072)))))
    cap = min(600000, max(1, (1 << 26) // C))
    n = int(round(math.exp(rng.uniform(0.0, math.log(cap)))))
    case = dict(op=op, n=n, C=C, dtype=rng.choice(["f32", "bf16", "f16"]), pad=rng.choice([0, 0, 0, 1, 8, 13]),
                masked=rng.random() < 0.3)
    if op == "sample":
        case["mode"] = rng.choice(["plain", "k", "p", "k_p", "p_min", "mixed"])
    else:
        case["k"] = int(round(math.exp(rng.uniform(0.0, math.log(min(C, 256))))))
        case["T"] = rng.choice([1.0, 1.5, 2.0, 4.0])
        if op != "top":
            case["rest"] = rng.random() < 0.7
    return case


def work(case):
    n, C, es = case["n"], case["C"], BYTES[case["dtype"]]
    rows = n * C * es
    if case["op"] == "sample":
        return {"bytes": rows + n * (4 * 5 + 8), "flops": 3 * n * C}
    record = n * (8 * case["k"] + 4)
    if case["op"] == "top":
        return {"bytes": rows + record, "flops": 5 * n * C}
    if case["op"] == "loss":
        return {"bytes": rows + record + 16 * n, "flops": 5 * n * C}
    if case["op"] == "grad":
        return {"bytes": 2 * rows + record + 16 * n, "flops": 4 * n * C}
    return {"bytes": 2 * rows + record + 8 * n, "flops": 8 * n * C}


# ------------------------------------------------------------------ inputs --

def score_rows(case, gen, n, C):
    """Scores as a classifier over many classes gives them: a wide bulk, a few
    classes far above it, spread that differs from row to row; the last eighth
    of the classes -inf where the class set is padded."""
    x = torch.randn(n, C, device="cuda", generator=gen)
    x *= 1.0 + 1.5 * torch.rand(n, 1, device="cuda", generator=gen)
    hot = min(24, C // 4)
    if hot > 0:
        at = torch.randint(0, C, (n, hot), device="cuda", generator=gen)
        up = 4.0 + 4.0 * torch.randn(n, hot, device="cuda", generator=gen).abs()
        x.scatter_add_(1, at, up)
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


def sampling_rows(case, gen):
    """Per-row temperature, top-k (0: off), top-p (1: off) and min-p (0: off)."""
    n, mode = case["n"], case["mode"]
    r = torch.rand(4, n, device="cuda", generator=gen)
    temperature = 0.6 + 0.6 * r[0]
    top_k = torch.zeros(n, dtype=torch.int32, device="cuda")
    top_p = torch.ones(n, device="cuda")
    min_p = torch.zeros(n, device="cuda")
    if mode in ("k", "k_p", "mixed"):
        top_k = (1 + 99 * r[1]).to(torch.int32)
    if mode in ("p", "k_p", "p_min", "mixed"):
        top_p = 0.8 + 0.19 * r[2]
    if mode in ("p_min", "mixed"):
        min_p = 0.05 * r[3]
    if mode == "mixed":  # requests of every kind in one batch, greedy ones among them
        kind = torch.randint(0, 5, (n,), device="cuda", generator=gen)
        temperature[kind == 0] = 0.0
        top_k[kind == 1] = 0
        top_p[kind == 2] = 1.0
        min_p[kind == 3] = 0.0
    return dict(temperature=temperature, top_k=top_k, top_p=top_p, min_p=min_p)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    n, C, op = case["n"], case["C"], case["op"]
    x = score_rows(case, gen, n, C)
    state = dict(op=op, scores=strided(case, x), n=n, C=C)
    if op == "sample":
        state.update(sampling_rows(case, gen))
        state["u"] = torch.rand(n, device="cuda", generator=gen)
        state["out"] = torch.empty(n, dtype=torch.int32, device="cuda")
        state["logp"] = torch.empty(n, device="cuda")
    elif op == "top":
        state.update(k=case["k"], T=case["T"])
        state["values"] = torch.empty(n, case["k"], device="cuda")
        state["classes"] = torch.empty(n, case["k"], dtype=torch.int32, device="cuda")
        state["rest"] = torch.empty(n, device="cuda")
    else:
        # the teacher's record: its own opinion of the same rows
        x = x + 0.7 * torch.randn(n, C, device="cuda", generator=gen)
        values, classes = torch.topk(x, case["k"], dim=1)
        rest = None
        if case["rest"]:
            # (of a row listed whole there is no rest)
            soft = torch.softmax(x / case["T"], 1)
            rest = torch.zeros(n, device="cuda") if case["k"] == C else \
                soft.scatter_(1, classes, 0.0).sum(1).clamp_(0.0, 1.0)
        classes = torch.where(values > float("-inf"), classes, torch.full_like(classes, -1)).to(torch.int32)
        weight = 0.5 + torch.rand(n, device="cuda", generator=gen)
        weight[torch.rand(n, device="cuda", generator=gen) < 0.1] = 0.0  # rows that do not count
        state.update(T=case["T"], t_values=values, t_classes=classes, t_rest=rest, weight=weight)
        state["loss"] = torch.empty(n, device="cuda")
        state["stats"] = torch.empty(n, 3, device="cuda")
        state["grad"] = torch.empty_strided((n, C), state["scores"].stride(), dtype=state["scores"].dtype,
                                            device="cuda") if op != "loss" else None
        if op == "grad":  # the forward pass's statistics are in hand
            state["stats"] = plain_stats(state).float()
    if own:
        import histogram_split_finding_amd as g
        state["ws"] = g.new_workspace(g.gbdt_scores_workspace_bytes(n, C))
    return state


# ------------------------------------------------------------- plain forms --

def plain_order(scores):
    x = scores.float()
    x = torch.where(torch.isnan(x), torch.full_like(x, float("-inf")), x) + 0.0
    return torch.sort(x, dim=1, descending=True, stable=True)


def plain_top(state):
    v, idx = plain_order(state["scores"])
    k = state["k"]
    m = v[:, :1]
    w = torch.exp(torch.where(v == m, torch.zeros_like(v), v - m) / state["T"])
    w = torch.where(v > float("-inf"), w, torch.zeros_like(w))
    out = w[:, k:].sum(1)
    total = w[:, :k].sum(1) + out
    rest = torch.where(total > 0, out / total, torch.zeros_like(out))
    values = v[:, :k].contiguous()
    classes = torch.where(values > float("-inf"), idx[:, :k], torch.full_like(idx[:, :k], -1))
    return values, classes.to(torch.int32), rest


def plain_listed(state):
    """(mask of the classes that the record lists, the record's places that name a class, safe indices)"""
    named = (state["t_classes"] >= 0) & (state["t_classes"] < state["C"])
    at = torch.where(named, state["t_classes"], torch.zeros_like(state["t_classes"])).long()
    inside = torch.zeros(state["n"], state["C"], dtype=torch.int8, device="cuda")
    inside.scatter_add_(1, at, named.to(torch.int8))
    return inside > 0, named, at


def plain_weights(state, dtype):
    x = state["scores"].to(dtype)
    m = x.amax(1, keepdim=True)
    live = m > float("-inf")
    return m, torch.exp((x - torch.where(live, m, torch.zeros_like(m))) / state["T"])


def plain_stats(state):
    # the loss is what is left when terms with the logarithm of these sums cancel: in 64 bits
    inside, _, _ = plain_listed(state)
    m, w = plain_weights(state, torch.float64)
    s_in = torch.where(inside, w, torch.zeros_like(w)).sum(1)
    s_out = torch.where(inside, torch.zeros_like(w), w).sum(1)
    return torch.stack([m[:, 0], s_in, s_out], 1)


def plain_teacher(state, named, dtype):
    t = torch.where(named, state["t_values"], torch.full_like(state["t_values"], float("-inf"))).to(dtype)
    tm = t.amax(1, keepdim=True)
    has = tm > float("-inf")
    e = torch.exp((t - torch.where(has, tm, torch.zeros_like(tm))) / state["T"])
    z = e.sum(1, keepdim=True)
    r = torch.zeros_like(tm) if state["t_rest"] is None else state["t_rest"][:, None].to(dtype)
    p = (1.0 - r) * e / torch.where(has, z, torch.ones_like(z))
    return p, r, has


def plain_loss(state, stats):
    # a small sum of larger terms that cancel: these few values per row in 64 bits
    _, named, at = plain_listed(state)
    p, r, has = plain_teacher(state, named, torch.float64)
    T = state["T"]
    m, s_in, s_out = stats[:, 0:1], stats[:, 1:2], stats[:, 2:3]
    s = s_in + s_out
    log_q = (state["scores"].gather(1, at).double() - m) / T - torch.log(s)
    zero = torch.zeros_like(p)
    loss = torch.where(p > 0, p * (torch.log(p) - log_q), zero).sum(1, keepdim=True)
    loss = loss + torch.where(r > 0, r * (torch.log(r) - torch.log(s_out / s)), torch.zeros_like(r))
    live = has & (m > float("-inf"))
    return (T * T * torch.where(live, loss, torch.zeros_like(loss)))[:, 0].float()


def plain_grad(state, stats):
    inside, named, at = plain_listed(state)
    p, r, has = plain_teacher(state, named, torch.float32)
    m, w = plain_weights(state, torch.float32)
    s_in, s_out = stats[:, 1:2].float(), stats[:, 2:3].float()
    s = s_in + s_out
    q = w / s
    share = torch.where(s_out > 0, 1.0 - r * s / s_out, torch.zeros_like(r))
    g = torch.where(inside, q, q * share)
    g.scatter_add_(1, at, torch.where(named, -p, torch.zeros_like(p)))
    weight = state["weight"][:, None]
    live = has & (m > float("-inf")) & (weight != 0)
    g = torch.where(live, g * (weight * state["T"]), torch.zeros_like(g))
    return g.to(state["scores"].dtype)


def plain_sample(state):
    v, idx = plain_order(state["scores"])
    # masses in 64 bits: a draw next to a border has to fall on its side
    T = state["temperature"].double()[:, None]
    greedy = T == 0
    m = v[:, :1]
    d = torch.where(v == m, 0.0, v.double() - m.double())
    w = torch.exp(d / torch.where(greedy, torch.ones_like(T), T))
    w = torch.where(v > float("-inf"), w, torch.zeros_like(w))
    place = torch.arange(state["C"], device="cuda")[None]
    k = state["top_k"].long()[:, None]
    k = torch.where(greedy, torch.ones_like(k), torch.where(k <= 0, torch.full_like(k, state["C"]), k))
    w = torch.where(place < k, w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], 1)
    top_p = state["top_p"].double()[:, None]
    keep = (before < top_p * cum[:, -1:]) | (top_p >= 1) | (place == 0)
    keep &= (w >= state["min_p"].double()[:, None]) & (w > 0)
    w = torch.where(keep, w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    W = cum[:, -1:]
    past = keep & (cum > state["u"].double()[:, None] * W)
    n_keep = keep.sum(1, keepdim=True)
    first = torch.where(past.any(1, keepdim=True), past.int().argmax(1, keepdim=True), (n_keep - 1).clamp(min=0))
    live = n_keep > 0
    out = torch.where(live, idx.gather(1, first), torch.full_like(first, -1))
    logp = torch.where(live, torch.log(w.gather(1, first) / W), torch.full_like(W, float("-inf")))
    return out[:, 0].to(torch.int32), logp[:, 0].float()


# --------------------------------------------------------------------- run --

def run(state):
    op = state["op"]
    if own:
        import histogram_split_finding_amd as g
        x, ws = state["scores"], state["ws"]
        if op == "top":
            g.gbdt_top_scores(x, state["k"], state["T"], state["values"], state["classes"], state["rest"], ws)
            return state["values"], state["classes"], state["rest"]
        if op == "sample":
            g.gbdt_sample_classes(x, state["u"], state["temperature"], state["top_k"], state["top_p"],
                                  state["min_p"], state["out"], state["logp"], ws)
            return state["out"], state["logp"]
        teacher = (state["t_values"], state["t_classes"], state["t_rest"])
        if op == "loss":
            g.gbdt_distill_loss(x, *teacher, state["T"], state["loss"], state["stats"], ws)
            return state["loss"], state["stats"]
        if op == "grad":
            g.gbdt_distill_grad(x, *teacher, state["T"], state["stats"], state["weight"], state["grad"], ws)
            return state["grad"]
        g.gbdt_distill_step(x, *teacher, state["T"], state["weight"], state["loss"], state["grad"], ws)
        return state["loss"], state["grad"]
    if op == "top":
        return plain_top(state)
    if op == "sample":
        return plain_sample(state)
    if op == "grad":
        return plain_grad(state, state["stats"])
    stats = plain_stats(state)
    if op == "loss":
        return plain_loss(state, stats), stats.float()
    return plain_loss(state, stats), plain_grad(state, stats)


# --------------------------------------------------------------- in 64 bits --

def exact_keys(x):
    """Integers in the order of the scores: larger for a higher value, and for the lower class among equals."""
    x = x.double()
    x[torch.isnan(x)] = float("-inf")
    bits = x.float().view(torch.int32).long()
    bits = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF))  # -0 and +0 are both 0
    n_classes = x.shape[1]
    return bits * (1 << 20) + torch.arange(n_classes - 1, -1, -1, device=x.device), x


def exact_sorted(x):
    key, x = exact_keys(x)
    key = torch.sort(key, dim=1).values.flip(1)
    at = x.shape[1] - 1 - (key & ((1 << 20) - 1))
    return x.gather(1, at), at


def exact_top(state):
    v, at = exact_sorted(state["scores"])
    k = state["k"]
    z = v / state["T"]
    top = torch.where(z[:, :1] > -math.inf, z[:, :1], torch.zeros_like(z[:, :1]))
    e = torch.exp(z - top)
    inside, outside = e[:, :k].sum(1), e[:, k:].sum(1)
    rest = torch.where(inside > 0, outside / (inside + outside), torch.zeros_like(inside))
    at = torch.where(v > -math.inf, at, torch.full_like(at, -1))
    return v[:, :k], at[:, :k].to(torch.int32), rest


def exact_distill(state, op):
    """Dense over the classes: the teacher's distribution as a full row."""
    x = state["scores"].double()
    n, C = x.shape
    T = state["T"]
    cls = state["t_classes"].long()
    ok = (cls >= 0) & (cls < C)
    # a class beyond the row takes the places that name none
    col = torch.where(ok, cls, torch.full_like(cls, C))
    t = torch.full((n, C + 1), -math.inf, dtype=torch.float64, device=x.device)
    t.scatter_(1, col, state["t_values"].double())
    t = t[:, :C]
    listed_class = torch.zeros(n, C + 1, dtype=torch.bool, device=x.device)
    listed_class.scatter_(1, col, True)
    listed_class = listed_class[:, :C]
    r = torch.zeros(n, dtype=torch.float64, device=x.device) if state["t_rest"] is None else state["t_rest"].double()
    alive = (t.amax(1) > -math.inf) & (x.amax(1) > -math.inf)
    lse_t = torch.logsumexp(t / T, 1)
    p = torch.exp(t / T - torch.where(alive, lse_t, torch.zeros_like(lse_t))[:, None]) * (1.0 - r)[:, None]
    m = x.amax(1)
    e = torch.exp((x - torch.where(m > -math.inf, m, torch.zeros_like(m))[:, None]) / T)
    s_in, s_out = (e * listed_class).sum(1), (e * ~listed_class).sum(1)
    stats = torch.stack([m, s_in, s_out], 1)
    total = s_in + s_out
    q = e / total[:, None]
    loss = grad = None
    if op != "grad":
        terms = torch.where(p > 0, p * (torch.log(p) - torch.log(q)), torch.zeros_like(p)).sum(1)
        terms = terms + torch.where(r > 0, r * (torch.log(r) - torch.log(s_out / total)), torch.zeros_like(r))
        loss = torch.where(alive, T * T * terms, torch.zeros_like(terms))
    if op != "loss":
        cond = torch.where(listed_class | (s_out == 0)[:, None], torch.zeros_like(e), e / s_out[:, None])
        full = p + r[:, None] * cond  # the teacher's mass, its rest spread as the student spreads its own
        q_all = torch.where((s_out == 0)[:, None] & ~listed_class, torch.zeros_like(q), q)
        counts = (alive & (state["weight"] != 0))[:, None]
        grad = torch.where(counts, (q_all - full) * (T * state["weight"].double())[:, None], torch.zeros_like(q))
    return loss, grad, stats


def exact_sample(state):
    v, at = exact_sorted(state["scores"])
    n, C = v.shape
    T = state["temperature"].double()
    cold = T == 0
    top = torch.where(v[:, 0] > -math.inf, v[:, 0], torch.zeros_like(T))
    e = torch.exp((v - top[:, None]) / torch.where(cold, torch.ones_like(T), T)[:, None])
    k = state["top_k"].long()
    limit = torch.where(cold, torch.ones_like(k), torch.where(k > 0, k.clamp(max=C), torch.full_like(k, C)))
    # sums up to each place; the kept classes are the first `limit` of the order, whatever shortens it
    run_sum = torch.cumsum(e, 1)
    mass = run_sum.gather(1, (limit - 1)[:, None])[:, 0]
    p = state["top_p"].double()
    short = torch.searchsorted(run_sum, (p * mass)[:, None], right=False)[:, 0] + 1
    limit = torch.where(p < 1, torch.minimum(limit, short.clamp(max=C)), limit)
    limit = torch.minimum(limit, ((e >= state["min_p"].double()[:, None]) & (e > 0)).sum(1))
    dead = limit == 0
    last = (limit - 1).clamp(min=0)
    total = run_sum.gather(1, last[:, None])[:, 0]
    spot = torch.searchsorted(run_sum, (state["u"].double() * total)[:, None], right=True)[:, 0]
    spot = torch.minimum(spot, last)
    out = torch.where(dead, torch.full_like(spot, -1), at.gather(1, spot[:, None])[:, 0])
    logp = torch.log(e.gather(1, spot[:, None])[:, 0]) - torch.log(total)
    return out.to(torch.int32), torch.where(dead, torch.full_like(logp, -math.inf), logp)


def exact(case, seed):
    state = prepare(case, seed)
    op, n, C = case["op"], case["n"], case["C"]
    per_row = ("scores", "temperature", "top_k", "top_p", "min_p", "u", "t_values", "t_classes", "t_rest", "weight")
    step = max(1, (1 << 26) // C)
    parts = []
    for lo in range(0, n, step):
        part = dict(state)
        for name in per_row:
            if part.get(name) is not None:
                part[name] = part[name][lo:lo + step]
        part["n"] = part["scores"].shape[0]
        if op == "top":
            parts.append(exact_top(part))
        elif op == "sample":
            parts.append(exact_sample(part))
        else:
            loss, grad, stats = exact_distill(part, op)
            parts.append((loss, stats) if op == "loss" else (grad,) if op == "grad" else (loss, grad))
    whole = tuple(torch.cat(column) for column in zip(*parts))
    return whole[0] if op == "grad" else whole
