"""Routing to experts on the GPU against the FP64 reference in learn_ref.py.

Choices are equal: the choice values are FP64 on both sides, and the inputs' equal
values are equal bits.  Weights are FP64 rounded once: 2^-24, with 2^-40 for the
functions.  The gradient's values at the chosen experts are FP64 but for a softmax's
sum of FP32 exponentials, each off by (3 D + 2) 2^-24 with D = max x - x, and so are
the others' own exponentials; the result is rounded once to its type.
"""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import learn_ref as lref
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

STEP = 2.0 ** -24


def to_dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def workspace(n, E):
    return g.new_workspace(g.gbdt_scores_workspace_bytes(n, E))


def check(x, xh, r, bias, dtype, pad=0):
    n, E = xh.shape
    k = r.k
    ws = workspace(n, E)
    classes = torch.full((n, k), 7, dtype=torch.int32, device=DEV)
    weights = torch.full((n, k), 7.0, device=DEV)
    g.gbdt_route_classes(x, r, to_dev(bias), classes, weights, ws)
    assert g.gbdt_read_error(ws) == 0
    dw = np.random.default_rng(n + E).normal(0.0, 1.0, (n, k)).astype(np.float32)
    buf = torch.full((n * (E + pad),), 7.0, dtype=x.dtype, device=DEV)
    grad = buf.as_strided((n, E), (E + pad, 1))
    g.gbdt_route_grad(x, r, classes, to_dev(dw), grad, ws)
    assert g.gbdt_read_error(ws) == 0
    if pad:
        assert bool((buf.view(n, E + pad)[:, E:] == 7.0).all())
    c, w, gr = classes.cpu().numpy(), weights.double().cpu().numpy(), grad.double().cpu().numpy()
    tiny = {"f32": 2.0 ** -126, "bf16": 2.0 ** -126, "f16": 2.0 ** -25}[dtype]
    for i in range(n):
        wc, ww = lref.route(xh[i], r, bias)
        assert np.array_equal(c[i], wc), (i, c[i], wc)
        assert np.all(np.abs(w[i] - ww) <= (STEP + 2.0 ** -40) * np.abs(ww) + 2.0 ** -149), (i, w[i], ww)
        with np.errstate(all="ignore"):
            want = lref.route_grad(xh[i], r, wc, dw[i])
            s = lref.values(xh[i], r.score)
            D = np.where(np.isfinite(xh[i]), xh[i].max() - xh[i], 0.0)
        chosen = wc[wc >= 0]
        size = np.zeros(E)  # of what is added up
        each = abs(r.scale) * np.abs(dw[i][wc >= 0]) * s[chosen]
        if r.renormalise and s[chosen].sum() > 0:
            each = each / s[chosen].sum()
            size[chosen] = each + s[chosen] / s[chosen].sum() * each.sum()
        else:
            size[chosen] = each
            if not r.score:
                size += s * each.sum()
        # (the reference's own terms cancel where the weights are renormalised: s_c d s_e / N twice,
        # a few roundings of 2^-53 each)
        size += 2.0 ** -10 * s * each.sum()
        e = 0.0 if r.score or r.renormalise else 1.0
        tol = (ref.EPS[dtype] / 2 + 2 * STEP) * np.abs(want) + size * (e * (6 * np.minimum(D, 40.0) + 8) * STEP + 2.0 ** -40)
        assert np.all(np.abs(gr[i] - want) <= tol + tiny), (i, np.max(np.abs(gr[i] - want) / (tol + tiny)), gr[i], want)


def scores(n, E, dtype, seed, pad=0, ties=False):
    r = np.random.default_rng(seed)
    b = r.normal(0.0, 1.5, (n, E))
    if ties:
        b = np.round(b)
    t = torch.from_numpy(b).to(ref.TYPES[dtype])
    return ref.place(t, pad), t.double().numpy()


FORMS = [dict(), dict(sigmoid=True), dict(renormalise=False), dict(sigmoid=True, renormalise=False, scale=2.5)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("E", [1, 2, 3, 7, 8, 31, 32, 33, 60, 64, 65, 100, 128, 129, 200, 256, 257, 500, 512, 513,
                               1000, 1024])
def test_sizes(E, dtype):
    for n, form in zip((1, 5, 67, 9), FORMS):
        for k in sorted({1, min(E, 8), min(E, 32)}):
            say("route: %d x %d k=%d %s %s" % (n, E, k, dtype, form))
            x, xh = scores(n, E, dtype, E + n, pad=E % 3)
            bias = np.random.default_rng(E).normal(0.0, 0.2, E).astype(np.float32) if (n + k) % 2 else None
            check(x, xh, g.make_routing(k, **form), bias, dtype, pad=E % 4)


@pytest.mark.parametrize("E,G", [(8, 4), (8, 8), (6, 3), (35, 5), (64, 8), (63, 7), (96, 3), (160, 8), (256, 8), (256, 64),
                                 (198, 9), (1024, 16), (1023, 33), (1023, 3), (1005, 5), (999, 9), (1003, 17), (1024, 64)])
def test_groups(E, G):
    size = E // G
    for kept in sorted({1, (G + 1) // 2, G}):
        for top in (1, 2):
            for form in FORMS[:2] + FORMS[2:3]:
                k = min(6, size * kept)
                say("route groups: %d in %d keep %d top %d %s" % (E, G, kept, top, form))
                x, xh = scores(11, E, "f32", E + kept)
                bias = np.random.default_rng(E).normal(0.0, 0.2, E).astype(np.float32) if top == 2 else None
                check(x, xh, g.make_routing(k, n_groups=G, groups_kept=kept, group_top=top, **form), bias, "f32")


@pytest.mark.parametrize("E,G", [(16, 1), (60, 1), (64, 8), (256, 8), (1000, 1)])
def test_ties_masks_and_odd_rows(E, G):
    """Few values, many of them equal; experts and whole groups out of service; NaN,
    infinities, scores where a sigmoid is 0 or 1 and a softmax underflows."""
    say("route, odd rows: %d in %d" % (E, G))
    r = np.random.default_rng(E)
    b = np.round(r.normal(0.0, 1.5, (14, E)))
    b[0] = -np.inf
    b[1] = 0.0
    b[2] = -np.inf
    b[2, E // 2] = 1.0
    b[3, : E // 2] = -np.inf
    b[4, 1:] = -np.inf
    b[5, r.random(E) < 0.5] = np.nan
    b[6] = np.where(r.random(E) < 0.5, 0.0, -0.0)
    b[7, [1, 3]] = np.inf
    b[8] = 200.0 + np.round(r.normal(0.0, 1.0, E))
    b[9] = -200.0 + np.round(r.normal(0.0, 1.0, E))
    b[10] = -np.inf
    b[10, [0, E - 1]] = [-300.0, 300.0]
    b[11] = np.where(np.arange(E) % 5 == 0, 3.0, -np.inf)
    b[12] = -3.0e38
    b[13] = np.sort(b[13])
    t = torch.from_numpy(b).float()
    x, xh = ref.place(t), t.double().numpy()
    k = 8
    for form in FORMS:
        for top in (1, 2):
            for bias in (None, np.zeros(E, dtype=np.float32)):
                if bias is not None:
                    # (an expert taken out of service by its bias, and one by a NaN)
                    bias[3], bias[7] = -np.inf, np.nan
                rt = g.make_routing(k, n_groups=G, groups_kept=max(1, G // 2), group_top=top, **form)
                n = len(b)
                ws = workspace(n, E)
                classes, weights = torch.zeros(n, k, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
                g.gbdt_route_classes(x, rt, to_dev(bias), classes, weights, ws)
                c, w = classes.cpu().numpy(), weights.double().cpu().numpy()
                for i in range(n):
                    wc, ww = lref.route(xh[i], rt, bias)
                    assert np.array_equal(c[i], wc), (form, top, i, c[i], wc)
                    assert np.all(np.abs(w[i] - ww) <= (STEP + 2.0 ** -40) * np.abs(ww) + 2.0 ** -149), (i, w[i], ww)
                dw = torch.ones(n, k, device=DEV)
                grad = torch.full((n, E), 7.0, device=DEV)
                g.gbdt_route_grad(x, rt, classes, dw, grad, ws)
                assert bool(grad.isfinite().all())
                out = ~np.isfinite(xh) & ~np.isposinf(xh)
                assert bool((grad.cpu().numpy()[out] == 0).all())
                assert g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalise", [False, True])
def test_gradient_against_differences(sigmoid, renormalise):
    """Central differences of the FP64 weights: h^2 times a third derivative of order
    1, and roundings over h."""
    say("route, differences: %s %s" % (sigmoid, renormalise))
    n, E, k, h = 3, 20, 4, 1e-4
    x, xh = scores(n, E, "f32", 3)
    r = g.make_routing(k, sigmoid=sigmoid, renormalise=renormalise, scale=1.5)
    ws = workspace(n, E)
    classes, weights = torch.zeros(n, k, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
    g.gbdt_route_classes(x, r, None, classes, weights, ws)
    dw = np.random.default_rng(1).normal(0.0, 1.0, (n, k)).astype(np.float32)
    grad = torch.zeros(n, E, device=DEV)
    g.gbdt_route_grad(x, r, classes, to_dev(dw), grad, ws)
    c, got = classes.cpu().numpy(), grad.double().cpu().numpy()

    def total(row, i):
        s = lref.values(row, sigmoid)[c[i]]
        return 1.5 * float((s / (s.sum() if renormalise else 1.0)) @ dw[i].astype(np.float64))

    for i in range(n):
        for e in range(E):
            a, b = xh[i].copy(), xh[i].copy()
            a[e] += h
            b[e] -= h
            assert abs((total(a, i) - total(b, i)) / (2 * h) - got[i, e]) <= 10 * h * h + 1e-12 / h * 1e-1 + 1e-6


def lists(classes, E, place=True, ws=None):
    n = classes.numel()
    offsets = torch.full((E + 1,), 7, dtype=torch.int32, device=DEV)
    order = torch.full((n,), -9, dtype=torch.int32, device=DEV)
    pl = torch.full(classes.shape, 7, dtype=torch.int32, device=DEV) if place else None
    g.gbdt_route_lists(classes, E, offsets, order, pl, workspace(1, E) if ws is None else ws)
    return offsets, order, pl


@pytest.mark.parametrize("E", [1, 2, 7, 64, 65, 256, 1000, 1024])
@pytest.mark.parametrize("n", [0, 1, 8, 63, 64, 65, 500, 4096, 4097, 5000, 70001, 600011])
def test_lists(n, E):
    say("lists: %d places, %d experts" % (n, E))
    r = np.random.default_rng(n + E)
    for kind in range(3):
        c = r.integers(-1, E, n).astype(np.int32)
        if kind == 1:
            c = np.where(r.random(n) < 0.9, E // 2, c).astype(np.int32)  # one expert has nearly all
        if kind == 2:
            c[:] = -1 if n % 2 else E - 1
        offsets, order, place = lists(to_dev(c), E)
        key = np.where(c >= 0, c, E)
        want = np.argsort(key, kind="stable")
        cut = np.concatenate([[0], np.cumsum(np.bincount(key, minlength=E + 1)[:E])])
        assert np.array_equal(offsets.cpu().numpy(), cut)
        got = order.cpu().numpy()
        assert np.array_equal(got[: cut[-1]], want[: cut[-1]]) and np.all(got[cut[-1]:] == -9)
        back = np.full(n, -1, dtype=np.int64)
        back[want[: cut[-1]]] = np.arange(cut[-1])
        assert np.array_equal(place.cpu().numpy(), back)
        o2, order2, _ = lists(to_dev(c), E, place=False)
        assert torch.equal(o2, offsets) and torch.equal(order2, order)


@pytest.mark.parametrize("n", [100, 9000])
def test_device_side_checks(n):
    say("route, device checks: %d" % n)
    E, k = 12, 4
    x, xh = scores(n, E, "f32", 5)
    r = g.make_routing(k)
    ws = workspace(n, E)
    classes, weights = torch.zeros(n, k, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
    g.gbdt_route_classes(x, r, None, classes, weights, ws)
    grad, dw = torch.full((n, E), 7.0, device=DEV), torch.ones(n, k, device=DEV)
    for bad in (E, 2 ** 31 - 1):
        worse = classes.clone()
        worse[1, 2] = bad
        g.gbdt_route_grad(x, r, worse, dw, grad, ws)
        assert g.gbdt_read_error(ws) == -3
        padded = classes.cpu().numpy()
        padded[1, 2] = -1
        want = lref.route_grad(xh[1], r, padded[1], np.ones(k, dtype=np.float32))
        assert np.all(np.abs(grad[1].cpu().numpy() - want) <= 1e-6)
        offsets, order, place = lists(worse, E, ws=ws)
        assert g.gbdt_read_error(ws) == -3
        assert place[1, 2].item() == -1 and offsets[E].item() == n * k - 1
    twice = classes.clone()
    twice[2, 1] = twice[2, 0]
    g.gbdt_route_grad(x, r, twice, dw, grad, ws)
    assert g.gbdt_read_error(ws) == -1
    twice[2] = twice[2, 0]
    g.gbdt_route_grad(x, r, twice, dw, grad, ws)
    assert g.gbdt_read_error(ws) == -1 and g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("n", [3, 900, 20000])
def test_streams_graphs_and_repeats(n):
    say("route, graph: %d" % n)
    E, k = 64, 6
    x, _ = scores(n, E, "bf16", 1, ties=True)
    r = g.make_routing(k, sigmoid=True, n_groups=8, groups_kept=3, group_top=2)
    bias = to_dev(np.random.default_rng(2).normal(0.0, 0.1, E).astype(np.float32))
    ws, ws2 = workspace(n, E), workspace(n, E)
    classes, weights = torch.zeros(n, k, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
    offsets, order = torch.zeros(E + 1, dtype=torch.int32, device=DEV), torch.zeros(n * k, dtype=torch.int32, device=DEV)
    place, grad, dw = torch.zeros_like(classes), torch.zeros_like(x), torch.ones(n, k, device=DEV)
    outs = [classes, weights, offsets, order, place, grad]

    def work(ws):
        g.gbdt_route_classes(x, r, bias, classes, weights, ws)
        g.gbdt_route_lists(classes, E, offsets, order, place, ws)
        g.gbdt_route_grad(x, r, classes, dw, grad, ws)

    def taken():
        torch.cuda.synchronize()
        got = [t.cpu() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        return got

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        work(ws)
    taken()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work(ws)
    for q in range(4):
        fresh, _ = scores(n, E, "bf16", 10 + q, ties=True)
        x.copy_(fresh)
        work(ws2)
        want = taken()
        graph.replay()
        for a, b in zip(want, taken()):
            assert torch.equal(a, b), q
        with torch.cuda.stream(s):
            work(ws)
        for a, b in zip(want, taken()):
            assert torch.equal(a, b), q
    assert g.gbdt_read_error(ws) == 0 and g.gbdt_read_error(ws2) == 0


def test_more_rows_than_a_grid():
    """A second launch takes up where the first grid ends."""
    E, n, k = 520, (1 << 22) + 5, 3
    say("route, rows of two grids: %d x %d" % (n, E))
    few, xh = scores(64, E, "bf16", 3)
    x = few.repeat((n + 63) // 64, 1)[:n]
    r = g.make_routing(k, renormalise=False)
    ws = workspace(n, E)
    classes, weights = torch.full((n, k), -7, dtype=torch.int32, device=DEV), torch.zeros(n, k, device=DEV)
    g.gbdt_route_classes(x, r, None, classes, weights, ws)
    assert np.array_equal(classes[:64].cpu().numpy(), np.stack([lref.route(xh[i], r, None)[0] for i in range(64)]))
    assert torch.equal(classes, classes[:64].repeat((n + 63) // 64, 1)[:n])
    grad = torch.full_like(x, 7.0)
    g.gbdt_route_grad(x, r, classes, weights, grad, ws)
    assert torch.equal(grad[64:], grad[:64].repeat((n + 63) // 64, 1)[64:n])
    assert g.gbdt_read_error(ws) == 0


def test_no_rows():
    x = torch.zeros(0, 12, device=DEV)
    ws = workspace(0, 12)
    c, w = torch.zeros(0, 3, dtype=torch.int32, device=DEV), torch.zeros(0, 3, device=DEV)
    r = g.make_routing(3)
    g.gbdt_route_classes(x, r, None, c, w, ws)
    g.gbdt_route_grad(x, r, c, w, x, ws)
    offsets = torch.full((13,), 7, dtype=torch.int32, device=DEV)
    g.gbdt_route_lists(c, 12, offsets, torch.zeros(0, dtype=torch.int32, device=DEV), c, ws)
    assert bool((offsets == 0).all()) and g.gbdt_read_error(ws) == 0
