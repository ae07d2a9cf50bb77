"""The operators on rows of class scores on the GPU against the FP64 reference
in scores_ref.py.

Tolerances.  A score's FP32 exponential exp2((x - m) c): the difference, c and
the product are each off by half a step (2^-24 relative), which moves the
exponent by 3 * 2^-24 * |x - m| / T, and the exponential itself by one step
(2^-23): with D the largest |x - m| / T that matters (40: e^-40 adds nothing a
float would show) a sum of them is off by (3 D + 2) 2^-24, relative.  `rel`
below is that, with 4 more half steps for what follows (sums' and results'
roundings).  Results in a smaller type are off by half its step.  Whole numbers
are equal: the kernels' sums are 64-bit, so a draw differs only where u falls
within 1e-10 of a border.
"""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import scores_ref as ref
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu

SIZES = [1, 2, 7, 8, 9, 16, 17, 32, 33, 63, 64, 65, 100, 128, 129, 257, 1000, 4099, 8192, 8193, 20011, 70001]


def rel(x, T):
    fin = x[np.isfinite(x)]
    D = min(40.0, (fin.max() - fin.min()) / T) if len(fin) else 0.0
    return (3 * D + 6) * 2.0 ** -24


def workspace(x):
    return g.new_workspace(g.gbdt_scores_workspace_bytes(x.shape[0], x.shape[1]))


def run_top(x, k, T):
    n = x.shape[0]
    v = torch.full((n, k), 7.0, device=DEV)
    c = torch.full((n, k), 7, dtype=torch.int32, device=DEV)
    r = torch.full((n,), 7.0, device=DEV)
    ws = workspace(x)
    g.gbdt_top_scores(x, k, T, v, c, r, ws)
    assert g.gbdt_read_error(ws) == 0
    return v.cpu().numpy(), c.cpu().numpy(), r.cpu().numpy()


def check_top(x, xh, k, T):
    v, c, r = run_top(x, k, T)
    for i in range(x.shape[0]):
        wv, wc, wr = ref.top_scores(xh[i], k, T)
        assert np.array_equal(c[i], wc), (i, c[i], wc)
        assert np.array_equal(v[i], wv.astype(np.float32)), i
        assert abs(r[i] - wr) <= 2 * rel(xh[i], T) * wr + 1e-37, (i, r[i], wr)


def to_dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def check_distill(x, xh, tv, tc, tr, T, weight, dtype, pad=0):
    """loss, grad (from the loss's stats) and step, and what lies between the
    gradient's rows."""
    n, C = xh.shape
    ws = workspace(x)
    tvd, tcd, trd, wd = to_dev(tv), to_dev(tc), to_dev(tr), to_dev(weight)
    loss = torch.full((n,), 7.0, device=DEV)
    stats = torch.full((n, 3), 7.0, device=DEV)
    loss2 = torch.full((n,), 7.0, device=DEV)
    buf = [torch.full((n * (C + pad),), 7.0, dtype=x.dtype, device=DEV) for _ in range(2)]
    grad = [b.as_strided((n, C), (C + pad, 1)) for b in buf]
    g.gbdt_distill_loss(x, tvd, tcd, trd, T, loss, stats, ws)
    g.gbdt_distill_grad(x, tvd, tcd, trd, T, stats, wd, grad[0], ws)
    g.gbdt_distill_step(x, tvd, tcd, trd, T, wd, loss2, grad[1], ws)
    assert g.gbdt_read_error(ws) == 0
    half, tiny = ref.EPS[dtype] / 2, {"f32": 1e-37, "bf16": 1e-37, "f16": 2.0 ** -25}[dtype]
    for b in buf:
        if pad:
            assert bool((b.view(n, C + pad)[:, C:] == 7.0).all())
    ls, l2, st = loss.cpu().numpy(), loss2.cpu().numpy(), stats.cpu().numpy()
    gr = [b.double().cpu().numpy() for b in grad]
    for i in range(n):
        w = 1.0 if weight is None else float(weight[i])
        r = None if tr is None else tr[i]
        wl, wg, wst = ref.distill(xh[i], tv[i], tc[i], r, T, w)
        e = rel(xh[i], T)
        for s, t in zip(st[i], wst):
            assert s == t or abs(s - t) <= e * abs(t) + 1e-37 or (np.isnan(s) and np.isnan(t)), (i, st[i], wst)
        for l in (ls[i], l2[i]):
            assert l == wl or (np.isnan(l) and np.isnan(wl)) or \
                abs(l - wl) <= T * T * e + 2.0 ** -24 * abs(wl), (i, l, wl, e)
        rr = 0.0 if r is None else float(r)
        s_all = wst[1] + wst[2]
        amp = 1.0 + (rr * s_all / wst[2] if wst[2] > 0 else 0.0)
        with np.errstate(all="ignore"):
            q = np.where(np.isneginf(xh[i]), 0.0, np.exp((xh[i] - wst[0]) / T)) / (s_all if s_all > 0 else 1.0)
        p = np.zeros(C)
        ok = (tc[i] >= 0) & (tc[i] < C)
        p[tc[i][ok]] = np.abs(wg[tc[i][ok]]) / max(abs(w) * T, 1e-300) + q[tc[i][ok]]
        tol = abs(w) * T * (q * amp * 2 * e + p * 2 * e) + half * np.abs(wg) + tiny
        for got in gr:
            same = (got[i] == wg) | (np.isnan(got[i]) & np.isnan(wg))
            off = np.abs(got[i] - wg)
            assert np.all(same | (off <= tol)), (i, np.nanmax(np.where(same, 0, off / tol)))


def run_sample(x, u, T, k, p, mp):
    n = x.shape[0]
    out = torch.full((n,), 7, dtype=torch.int32, device=DEV)
    logp = torch.full((n,), 7.0, device=DEV)
    ws = workspace(x)
    g.gbdt_sample_classes(x, to_dev(u), to_dev(T), to_dev(k), to_dev(p), to_dev(mp), out, logp, ws)
    assert g.gbdt_read_error(ws) == 0
    return out.cpu().numpy(), logp.cpu().numpy()


def check_sample(x, xh, u, T=None, k=None, p=None, mp=None):
    out, logp = run_sample(x, u, T, k, p, mp)
    for i in range(x.shape[0]):
        at = lambda a, d: float(a[i]) if a is not None else d  # noqa: E731
        wo, wl = ref.sample(xh[i], float(u[i]), at(T, 1.0), int(at(k, 0)), at(p, 1.0), at(mp, 0.0))
        assert out[i] == wo, (i, out[i], wo)
        # logp is computed in FP64 and rounded once
        assert logp[i] == wl or abs(logp[i] - wl) <= 2.0 ** -24 * abs(wl) + 1e-9, (i, logp[i], wl)


def sampling_params(n, C, seed):
    r = np.random.default_rng(seed)
    f = np.float32
    return dict(u=r.random(n).astype(f), T=r.uniform(0.5, 1.5, n).astype(f),
                k=r.integers(1, max(2, min(C, 200)), n).astype(np.int32),
                p=r.uniform(0.3, 0.99, n).astype(f), mp=r.uniform(0.0, 0.2, n).astype(f))


# ----------------------------------------------------------------- shapes --

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", SIZES)
def test_top_sizes(C, dtype):
    for k in sorted({1, min(C, 5), min(C, 64), min(C, 256)}):
        say("top: C=%d k=%d %s" % (C, k, dtype))
        x, xh = ref.rows(5, C, dtype, 100 + C, pad=C % 4)
        check_top(x, xh, k, 1.7)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", SIZES)
def test_distill_sizes(C, dtype):
    for k, rest, T in [(1, True, 1.0), (min(C, 5), True, 2.0), (min(C, 33), False, 1.5), (256, True, 4.0)]:
        say("distill: C=%d k=%d rest=%s T=%s %s" % (C, k, rest, T, dtype))
        x, xh = ref.rows(5, C, dtype, 200 + C, pad=C % 3)
        tv, tc, tr = ref.records(xh, k, C, T, rest)
        weight = np.array([1.0, 0.5, 0.0, -2.0, 3.0], dtype=np.float32)
        check_distill(x, xh, tv, tc, tr, T, weight if C % 2 else None, dtype, pad=C % 5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", SIZES)
def test_sample_sizes(C, dtype):
    n = 6
    x, xh = ref.rows(n, C, dtype, 300 + C, pad=C % 4)
    q = sampling_params(n, C, C)
    for name, kw in [("plain", {}), ("T", dict(T=q["T"])), ("k", dict(k=q["k"])), ("p", dict(p=q["p"])),
                     ("min_p", dict(mp=q["mp"])), ("all", dict(T=q["T"], k=q["k"], p=q["p"], mp=q["mp"])),
                     ("large k", dict(k=np.full(n, max(1, C - 3), dtype=np.int32), p=q["p"])),
                     ("greedy", dict(T=np.zeros(n, dtype=np.float32), k=q["k"]))]:
        say("sample: C=%d %s %s" % (C, name, dtype))
        check_sample(x, xh, q["u"], **kw)


@pytest.mark.parametrize("C,n", [(7, 1000), (64, 517), (1000, 300)])
def test_many_rows(C, n):
    say("many rows: %d x %d" % (n, C))
    x, xh = ref.rows(n, C, "f32", 7)
    check_top(x, xh, min(C, 3), 1.0)
    tv, tc, tr = ref.records(xh, 3, 8, 2.0)
    check_distill(x, xh, tv, tc, tr, 2.0, None, "f32")
    q = sampling_params(n, C, 9)
    check_sample(x, xh, q["u"], q["T"], q["k"], q["p"], q["mp"])


# ------------------------------------------------- masks, ties, odd values --

def odd_rows(C, dtype):
    """Rows where an order, a sum or a range can go wrong."""
    info = torch.finfo(ref.TYPES[dtype])
    r = np.random.default_rng(C)
    base = r.normal(0.0, 1.0, (12, C))
    base[0] = -np.inf                                  # nothing left
    base[1] = 0.5                                      # all equal
    base[2] = -np.inf
    base[2, C // 2] = -3.0                             # one left
    base[3] = info.min                                 # the type's lowest everywhere
    base[4, : C // 2] = -np.inf                        # half masked
    base[5] = np.where(r.random(C) < 0.5, 1.0, 2.0)    # two values
    base[6] = np.where(r.random(C) < 0.5, 0.0, -0.0)   # signed zeros
    base[7, 0], base[7, C - 1] = info.max, info.min    # the whole range
    base[8] = np.sort(base[8])[::-1]                   # high scores side by side
    base[9] *= 1e-3                                    # a narrow row
    base[10] = info.tiny * r.integers(0, 3, C)         # next to zero
    base[11] = np.round(base[11])                      # few values
    return torch.from_numpy(base).to(ref.TYPES[dtype])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("C", [2, 7, 32, 33, 300, 5000, 9001, 33333])
def test_odd_rows(C, dtype):
    say("odd rows: C=%d %s" % (C, dtype))
    t = odd_rows(C, dtype)
    x, xh = ref.place(t), t.double().numpy()
    for k in sorted({1, min(C, 40)}):
        check_top(x, xh, k, 1.0)
    tv, tc, tr = ref.records(xh, min(C, 40), C, 1.0)
    tv[3], tc[3] = -np.inf, np.arange(tc.shape[1]) if tc.shape[1] <= C else -1   # no live entry
    tc[9] = -1                                                                   # no entry at all
    check_distill(x, xh, tv, tc, tr, 1.0, None, dtype)
    n = x.shape[0]
    q = sampling_params(n, C, C)
    # (equal scores make running sums that meet a border exactly: exact there too)
    half = np.full(n, 0.5, dtype=np.float32)
    for kw in [dict(), dict(p=half), dict(k=q["k"], p=half), dict(mp=half), dict(T=np.zeros(n, dtype=np.float32)),
               dict(k=np.full(n, max(1, C // 2), dtype=np.int32))]:
        check_sample(x, xh, q["u"], **kw)
    for u in (0.0, 1.0 - 2.0 ** -24):
        check_sample(x, xh, np.full(n, u, dtype=np.float32))


@pytest.mark.parametrize("C", [7, 33, 9001])
def test_nan_and_inf(C):
    say("NaN and inf: C=%d" % C)
    r = np.random.default_rng(C)
    b = r.normal(0.0, 1.0, (6, C))
    b[0, 1] = np.nan
    b[1, C // 2] = np.inf
    b[2, 0] = b[2, C - 1] = np.inf
    b[3] = np.nan
    b[4, 0], b[4, 1], b[4, 2] = np.nan, np.inf, -np.inf
    b[5, 3] = np.nan
    t = torch.from_numpy(b).float()
    x, xh = ref.place(t), t.double().numpy()
    check_top(x, xh, min(C, 5), 1.0)
    q = sampling_params(6, C, C)
    check_sample(x, xh, q["u"])
    check_sample(x, xh, q["u"], k=np.full(6, 2, dtype=np.int32))
    # distillation: a NaN or +inf score makes its row NaN, weight 0 makes it 0, the other rows stay
    tv, tc, tr = ref.records(b, 3, C, 1.0, holes=False)
    ws = workspace(x)
    loss = torch.zeros(6, device=DEV)
    grad = torch.zeros(6, C, device=DEV)
    weight = torch.tensor([1.0, 1.0, 1.0, 1.0, 1.0, 0.0], device=DEV)
    g.gbdt_distill_step(x, to_dev(tv), to_dev(tc), to_dev(tr), 1.0, weight, loss, grad, ws)
    assert bool(loss.isnan().all()) and bool(grad[:5].isnan().any(1).all())
    assert bool((grad[5] == 0).all())
    # a masked class that the teacher has: loss +inf, gradient finite; a NaN teacher value: NaN
    t = torch.from_numpy(r.normal(0.0, 1.0, (3, C))).float()
    t[0, 2] = -np.inf
    tc = np.array([[1, 2], [1, 2], [1, 2]], dtype=np.int32)
    tv = np.array([[0.5, 1.0], [0.5, np.nan], [0.5, -np.inf]], dtype=np.float32)
    x = ref.place(t)
    loss, grad = torch.zeros(3, device=DEV), torch.zeros(3, C, device=DEV)
    g.gbdt_distill_step(x, to_dev(tv), to_dev(tc), None, 1.0, None, loss, grad, ws)
    assert np.isposinf(loss[0].item()) and bool(grad[0].isfinite().all())
    assert bool(loss[1].isnan()) and bool(grad[1].isnan().any())
    for i in (0, 2):
        wl, wg, _ = ref.distill(t[i].double().numpy(), tv[i], tc[i], None, 1.0, 1.0)
        assert loss[i].item() == wl or abs(loss[i].item() - wl) <= 30 * 2.0 ** -24
        assert np.all(np.abs(grad[i].cpu().numpy() - wg) <= 30 * 2.0 ** -24)


@pytest.mark.parametrize("C", [5, 700])
def test_gradient_against_differences(C):
    """Central differences of the FP64 loss; h^2 times its third derivative
    (at most 1 / T here) and the loss's own rounding over h bound the error."""
    say("differences: C=%d" % C)
    T, h = 2.0, 1e-4
    x, xh = ref.rows(3, C, "f32", 11)
    tv, tc, tr = ref.records(xh, min(C, 4), 12, T)
    n = 3
    ws = workspace(x)
    loss, grad = torch.zeros(n, device=DEV), torch.zeros(n, C, device=DEV)
    g.gbdt_distill_step(x, to_dev(tv), to_dev(tc), to_dev(tr), T, None, loss, grad, ws)
    got = grad.double().cpu().numpy()
    for i in range(n):
        for c in list(range(min(C, 5))) + [int(j) for j in tc[i] if j >= 0]:
            a, b = xh[i].copy(), xh[i].copy()
            a[c] += h
            b[c] -= h
            la = ref.distill(a, tv[i], tc[i], tr[i], T, 1.0)[0]
            lb = ref.distill(b, tv[i], tc[i], tr[i], T, 1.0)[0]
            assert abs((la - lb) / (2 * h) - got[i, c]) <= h * h + 1e-13 / h + T * 2 * rel(xh[i], T), (i, c)


# ------------------------------------- far rows, streams, graphs, records --

def test_offsets_beyond_32_bits():
    """Rows 2^31 + 5 elements apart."""
    C, n, stride = 9001, 3, (1 << 31) + 5
    say("rows %d elements apart" % stride)
    x0, xh = ref.rows(n, C, "bf16", 21)
    buf = torch.empty((n - 1) * stride + C, dtype=torch.bfloat16, device=DEV)
    x = buf.as_strided((n, C), (stride, 1))
    x.copy_(x0)
    check_top(x, xh, 17, 1.0)
    q = sampling_params(n, C, 5)
    check_sample(x, xh, q["u"], p=q["p"])
    tv, tc, tr = ref.records(xh, 9, 5, 1.0)
    check_distill(x, xh, tv, tc, tr, 1.0, None, "bf16")


def test_no_rows():
    x = torch.zeros(0, 12, device=DEV)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(0, 12))
    f, i = torch.zeros(0, device=DEV), torch.zeros(0, dtype=torch.int32, device=DEV)
    v, c = torch.zeros(0, 3, device=DEV), torch.zeros(0, 3, dtype=torch.int32, device=DEV)
    g.gbdt_top_scores(x, 3, 1.0, v, c, f, ws)
    g.gbdt_distill_step(x, v, c, f, 1.0, None, f, torch.zeros(0, 12, device=DEV), ws)
    g.gbdt_sample_classes(x, f, None, None, None, None, i, f, ws)
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("C,n", [(7, 300), (9001, 40), (40000, 2)])
def test_other_stream_and_repeats(C, n):
    """On a stream of its own, and again: the same bits."""
    say("stream: %d x %d" % (n, C))
    x, xh = ref.rows(n, C, "bf16", 31)
    q = sampling_params(n, C, 32)
    tv, tc, tr = ref.records(xh, 5, 33, 1.0)
    dev = [to_dev(a) for a in (tv, tc, tr, q["u"], q["p"])]
    ws = workspace(x)
    s = torch.cuda.Stream()
    seen = []
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s):
            v, c = torch.zeros(n, 5, device=DEV), torch.zeros(n, 5, dtype=torch.int32, device=DEV)
            rest, loss, logp = (torch.zeros(n, device=DEV) for _ in range(3))
            grad, out = torch.zeros(n, C, dtype=x.dtype, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
            g.gbdt_top_scores(x, 5, 1.0, v, c, rest, ws)
            g.gbdt_distill_step(x, dev[0], dev[1], dev[2], 1.0, None, loss, grad, ws)
            g.gbdt_sample_classes(x, dev[3], None, None, dev[4], None, out, logp, ws)
        s.synchronize()
        seen.append([t.cpu() for t in (v, c, rest, loss, grad, out, logp)])
    for other in seen[1:]:
        for a, b in zip(seen[0], other):
            assert torch.equal(a, b)


@pytest.mark.parametrize("C,n", [(7, 300), (300, 20), (40000, 2)])
def test_graph_replays(C, n):
    """Captured once, replayed with other inputs, eager work in between."""
    say("graph: %d x %d" % (n, C))
    x, _ = ref.rows(n, C, "f32", 41)
    ws = workspace(x)
    v, c = torch.zeros(n, 5, device=DEV), torch.zeros(n, 5, dtype=torch.int32, device=DEV)
    rest, loss, logp = (torch.zeros(n, device=DEV) for _ in range(3))
    stats = torch.zeros(n, 3, device=DEV)
    grad, grad2 = torch.zeros(n, C, device=DEV), torch.zeros(n, C, device=DEV)
    out = torch.zeros(n, dtype=torch.int32, device=DEV)
    u, p = torch.zeros(n, device=DEV), torch.full((n,), 0.9, device=DEV)

    def work():
        g.gbdt_top_scores(x, 5, 1.0, v, c, rest, ws)
        g.gbdt_distill_step(x, v, c, rest, 2.0, None, loss, grad, ws)
        g.gbdt_distill_loss(x, v, c, rest, 2.0, loss, stats, ws)
        g.gbdt_distill_grad(x, v, c, rest, 2.0, stats, None, grad2, ws)
        g.gbdt_sample_classes(x, u, None, None, p, None, out, logp, ws)
        return [v, c, rest, loss, stats, grad, grad2, out, logp]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for k in range(4):
        fresh, _ = ref.rows(n, C, "f32", 50 + k)
        x.copy_(fresh)
        u.copy_(torch.from_numpy(np.random.default_rng(k).random(n).astype(np.float32)))
        want = [t.clone() for t in work()]
        torch.cuda.synchronize()
        for t in (v, c, rest, loss, stats, grad, grad2, out, logp):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (v, c, rest, loss, stats, grad, grad2, out, logp)):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("C", [7, 500, 9001])
def test_device_side_checks(C):
    """Values that only the device sees: recorded, in bounds, other rows right."""
    say("device checks: C=%d" % C)
    n = 4
    x, xh = ref.rows(n, C, "f32", 61)
    ws = workspace(x)
    loss, grad = torch.zeros(n, device=DEV), torch.zeros(n, C, device=DEV)

    def step(tv, tc, tr):
        g.gbdt_distill_step(x, to_dev(tv), to_dev(tc), to_dev(tr), 1.0, None, loss, grad, ws)
        with pytest.raises(g.GbdtError) as e:
            g._check(g.gbdt_read_error(ws), "distill")
        assert g.gbdt_read_error(ws) == 0
        return e.value.code

    tv, tc, tr = ref.records(xh, 3, 62, 1.0, holes=False)
    for bad in (C, C + 1000, 2 ** 31 - 1):
        worse = tc.copy()
        worse[1, 2] = bad
        assert step(tv, worse, tr) == -3
        # the entry counts as padding
        padded = tc.copy()
        padded[1, 2] = -1
        for i in range(n):
            wl, _, _ = ref.distill(xh[i], tv[i], padded[i], tr[i], 1.0, 1.0)
            assert abs(loss[i].item() - wl) <= rel(xh[i], 1.0) + 2.0 ** -24 * abs(wl)
    twice = tc.copy()
    twice[2, 1] = twice[2, 0]
    assert step(tv, twice, tr) == -1
    for r in (-0.25, 1.5, np.nan):
        off = tr.copy()
        off[0] = r
        assert step(tv, tc, off) == -3
    f = np.float32
    u = np.full(n, 0.5, dtype=f)
    ones, zeros = np.ones(n, dtype=f), np.zeros(n, dtype=f)
    for which, bad in [("u", 1.0), ("u", -0.1), ("u", np.nan), ("T", -1.0), ("T", np.inf), ("T", np.nan),
                       ("p", 1.5), ("p", np.nan), ("mp", -0.5), ("mp", 2.0)]:
        a = dict(u=u.copy(), T=ones.copy(), p=ones.copy(), mp=zeros.copy())
        a[which][2] = bad
        out, logp = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV)
        g.gbdt_sample_classes(x, to_dev(a["u"]), to_dev(a["T"]), None, to_dev(a["p"]), to_dev(a["mp"]), out, logp,
                              ws)
        with pytest.raises(g.GbdtError) as e:
            g._check(g.gbdt_read_error(ws), "sample")
        assert e.value.code == -3
        assert out[2].item() == -1 and np.isneginf(logp[2].item())
        for i in (0, 1, 3):
            assert out[i].item() == ref.sample(xh[i], 0.5, 1.0, 0, 1.0, 0.0)[0]


# ------------------------------------------ rows that a first pass leaves over --

def long_rows(C, seed):
    """Rows whose first classes tell nothing, or the wrong thing, about the rest."""
    r = np.random.default_rng(seed)
    b = r.normal(0.0, 1.0, (10, C))
    b[0] = np.sort(b[0])[::-1]             # the best first
    b[1] = np.sort(b[1])                   # the best last
    b[2, : C // 2] = -np.inf               # the first half masked
    b[3, C // 2:] = -np.inf                # the second half masked
    b[4, : C // 2] -= 30.0                 # the first half hopeless
    b[5] = np.round(b[5] * 2.0) / 2.0      # a few values, each many times
    b[6] *= 0.01                           # narrow: everything is likely
    b[7] = 0.0                             # equal, but for a few at the end
    b[7, C - 3:] = [1.0, 2.0, 1.0]
    b[8, : C - 2] = -np.inf                # two left
    b[9] *= 4.0                            # wide
    return b


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [2500, 20011, 70001])
def test_long_odd_rows(C, dtype):
    say("long odd rows: C=%d %s" % (C, dtype))
    t = torch.from_numpy(long_rows(C, C)).to(ref.TYPES[dtype])
    x, xh = ref.place(t, 3), t.double().numpy()
    n = x.shape[0]
    for k in (1, 50, 256):
        check_top(x, xh, k, 1.0)
    tv, tc, tr = ref.records(xh, 40, C, 1.0)
    check_distill(x, xh, tv, tc, tr, 1.0, None, dtype, pad=1)
    f = np.float32
    q = sampling_params(n, C, C)
    for name, kw in [("plain", {}), ("p", dict(p=q["p"])), ("deep p", dict(p=np.full(n, 0.9995, dtype=f))),
                     ("min_p", dict(mp=q["mp"])), ("deep min_p", dict(mp=np.full(n, 1e-4, dtype=f))),
                     ("p, min_p", dict(p=q["p"], mp=np.full(n, 1e-3, dtype=f))),
                     ("k", dict(k=np.full(n, 256, dtype=np.int32))),
                     ("large k", dict(k=np.full(n, 257, dtype=np.int32), p=q["p"], mp=np.full(n, 1e-3, dtype=f))),
                     ("cold", dict(T=np.full(n, 0.02, dtype=f))), ("hot", dict(T=np.full(n, 50.0, dtype=f)))]:
        say(name)
        check_sample(x, xh, q["u"], **kw)


@pytest.mark.parametrize("n,C", [(300, 40960), (140, 66001)])
def test_more_rows_than_workgroups_share(n, C):
    """As many long rows as keep a workgroup each, on both sides of the row
    counts that are split or take more threads."""
    say("long rows: %d x %d" % (n, C))
    x, xh = ref.rows(n, C, "bf16", C)
    check_top(x, xh, 20, 2.0)
    q = sampling_params(n, C, n)
    check_sample(x, xh, q["u"], T=q["T"], p=q["p"], mp=q["mp"] * 0.01)
    check_sample(x, xh, q["u"], k=q["k"])
    tv, tc, tr = ref.records(xh, 20, C, 2.0)
    check_distill(x, xh, tv, tc, tr, 2.0, None, "bf16")


@pytest.mark.parametrize("C", [7, 500])
def test_top_without_rest(C):
    x, xh = ref.rows(9, C, "f16", C)
    v, c = torch.zeros(9, 4, device=DEV), torch.zeros(9, 4, dtype=torch.int32, device=DEV)
    ws = workspace(x)
    g.gbdt_top_scores(x, 4, 1.0, v, c, None, ws)
    for i in range(9):
        wv, wc, _ = ref.top_scores(xh[i], 4, 1.0)
        assert np.array_equal(c[i].cpu().numpy(), wc) and np.array_equal(v[i].cpu().numpy(), wv.astype(np.float32))


@pytest.mark.parametrize("C", [9, 40, 3000, 50000])
def test_sample_frequencies(C):
    """Draws with evenly spread u: each class as often as its probability says,
    to within one draw at either end of its interval."""
    n = 4096
    say("frequencies: C=%d" % C)
    row = torch.zeros(C, dtype=torch.float64)
    row[: min(C, 9)] = torch.arange(min(C, 9), dtype=torch.float64) * 0.5 + 6.0
    x = row.float().to(DEV).expand(n, C).contiguous()
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float()
    out, _ = run_sample(x, u.numpy(), None, None, None, None)
    p = torch.softmax(row, 0).numpy()
    for c in range(min(C, 9)):
        assert abs(int((out == c).sum()) - n * p[c]) <= 2.0, c


def test_example():
    """Records, loss, gradient and draws as they are used together."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_classes.py")
    spec = importlib.util.spec_from_file_location("distill_classes", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, agree = m.run(rows=2000, steps=40)
    assert losses[-1] < 0.5 * losses[0] and all(b <= a for a, b in zip(losses, losses[1:]))
    # (a draw from seven classes without learning would agree in one of seven)
    assert agree > 2.0 / 7.0
