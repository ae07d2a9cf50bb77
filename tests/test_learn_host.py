"""Refusals of the operators on drawn classes and of the routing: the C entry
points check what the host can see before any device work, the Python calls the
tensors' types, shapes and strides."""
import ctypes

import pytest
import torch

import histogram_split_finding_amd as g

FAKE = 0x10000  # an aligned address that is never read
WS = 1 << 24


def scores(**kw):
    a = dict(data=FAKE, n_rows=4, row_stride=10, n_classes=10, dtype=0)
    a.update(kw)
    return g.Scores(*[a[k] for k in ("data", "n_rows", "row_stride", "n_classes", "dtype")])


def policy(**kw):
    a = dict(old_logp=FAKE, ref_logp=None, advantage=FAKE, weight=None, clip_low=0.2, clip_high=0.2, kl=0.1)
    a.update(kw)
    return g.Policy(*[a[k] for k in ("old_logp", "ref_logp", "advantage", "weight", "clip_low", "clip_high", "kl")])


def pairs(**kw):
    a = dict(offsets=FAKE, ref_logp=None, weight=None, n_pairs=2, average=0, beta=0.1, smoothing=0.0)
    a.update(kw)
    return g.Pairs(*[a[k] for k in ("offsets", "ref_logp", "weight", "n_pairs", "average", "beta", "smoothing")])


def routing(**kw):
    a = dict(k=3)
    a.update(kw)
    r = g.make_routing(**{k: v for k, v in a.items() if k not in ("score",)})
    if "score" in a:
        r.score = a["score"]
    return r


def ref(v):
    return ctypes.byref(v) if v is not None else None


def logp(x, T=1.0, cls=FAKE, lp=FAKE, st=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_class_logp(ref(x), cls, T, lp, st, ws, nb, None)


def logp_grad(x, T=1.0, cls=FAKE, st=FAKE, d=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_class_logp_grad(ref(x), cls, T, st, d, gr, ld, ws, nb, None)


def policy_loss(x, p, T=1.0, cls=FAKE, lo=FAKE, d=FAKE, st=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_policy_loss(ref(x), cls, T, ref(p), lo, None, d, st, ws, nb, None)


def policy_step(x, p, T=1.0, cls=FAKE, lo=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_policy_step(ref(x), cls, T, ref(p), lo, None, gr, ld, ws, nb, None)


def pref_loss(x, p, T=1.0, cls=FAKE, lo=FAKE, lp=FAKE, d=FAKE, st=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_preference_loss(ref(x), cls, T, ref(p), lo, None, lp, d, st, ws, nb, None)


def pref_step(x, p, T=1.0, cls=FAKE, lo=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_preference_step(ref(x), cls, T, ref(p), lo, None, gr, ld, ws, nb, None)


def route(x, r, c=FAKE, w=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_route_classes(ref(x), ref(r), None, c, w, ws, nb, None)


def route_grad(x, r, c=FAKE, d=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_route_grad(ref(x), ref(r), c, d, gr, ld, ws, nb, None)


def lists(c=FAKE, n=100, E=10, off=FAKE, order=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_route_lists(c, n, E, off, order, None, ws, nb, None)


def all_calls(x, **kw):
    T = {k: v for k, v in kw.items() if k == "T"}
    rest = {k: v for k, v in kw.items() if k != "T"}
    out = [logp(x, **kw), logp_grad(x, **kw), policy_loss(x, policy(), **kw), policy_step(x, policy(), **kw),
           pref_loss(x, pairs(), **kw), pref_step(x, pairs(), **kw)]
    return out if T else out + [route(x, routing(), **rest), route_grad(x, routing(), **rest)]


@pytest.mark.parametrize("kw,code", [
    (dict(data=None), -1), (dict(data=FAKE + 2), -1), (dict(data=FAKE + 1, dtype=1), -1), (dict(n_rows=-1), -1),
    (dict(n_rows=(1 << 31) + 1), -1), (dict(n_classes=0), -1), (dict(n_classes=g.MAX_CLASSES + 1), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(row_stride=9), -2)])
def test_scores_rules(kw, code):
    assert set(all_calls(scores(**kw))) == {code} and g.last_error()


@pytest.mark.parametrize("T", [0.0, -1.0, float("nan"), float("inf"), 1e-31, 1e31])
def test_temperature_rules(T):
    assert set(all_calls(scores(), T=T)) == {-1}


def test_null_rules():
    x, p, q, r = scores(), policy(), pairs(), routing()
    for rc in (logp(None), logp_grad(None), policy_loss(None, p), policy_step(None, p), pref_loss(None, q),
               pref_step(None, q), route(None, r), route_grad(None, r), policy_loss(x, None), policy_step(x, None),
               pref_loss(x, None), pref_step(x, None), route(x, None), route_grad(x, None),
               logp(x, cls=None), logp(x, lp=None), logp_grad(x, cls=None), logp_grad(x, st=None),
               logp_grad(x, d=None), logp_grad(x, gr=None), logp_grad(x, gr=FAKE + 1),
               policy_loss(x, p, cls=None), policy_loss(x, p, lo=None), policy_loss(x, p, d=None),
               policy_loss(x, p, st=None), policy_loss(x, policy(old_logp=None)),
               policy_loss(x, policy(advantage=None)), policy_step(x, p, gr=None), policy_step(x, p, gr=FAKE + 2),
               policy_step(x, p, lo=None), pref_loss(x, q, cls=None), pref_loss(x, q, lo=None),
               pref_loss(x, q, lp=None), pref_loss(x, q, d=None), pref_loss(x, q, st=None),
               pref_loss(x, pairs(offsets=None)), pref_step(x, q, gr=None), pref_step(x, q, lo=None),
               pref_step(x, pairs(offsets=None)), pref_step(x, q, gr=FAKE + 2), pref_step(x, q, cls=None),
               route(x, r, c=None), route(x, r, w=None), route_grad(x, r, c=None), route_grad(x, r, d=None),
               route_grad(x, r, gr=None), lists(c=None), lists(off=None), lists(order=None), lists(n=-1),
               lists(n=1 << 31), lists(E=0), lists(E=1025)):
        assert rc == -1 and g.last_error()
    for rc in (logp_grad(x, ld=9), policy_step(x, p, ld=9), pref_step(x, q, ld=9), route_grad(x, r, ld=9)):
        assert rc == -2


def test_workspace_rules():
    x, p, q, r = scores(), policy(), pairs(), routing()
    need = g.gbdt_scores_workspace_bytes(4, 10)
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(nb=need - 1)):
        assert set(all_calls(x, **kw)) == {-1}
        assert lists(**kw) == -1
    more = g.gbdt_preference_workspace_bytes(4, 10)
    assert more >= need + 4 * 12 and pref_step(x, q, nb=more - 1) == -1
    assert g.gbdt_preference_workspace_bytes(-1, 5) == 0 and g.gbdt_preference_workspace_bytes(5, 0) == 0
    assert g.gbdt_preference_workspace_bytes(1 << 31, 7) >= 12 << 31


@pytest.mark.parametrize("kw", [dict(clip_low=-0.1), dict(clip_low=1.1), dict(clip_low=float("nan")),
                                dict(clip_high=-0.1), dict(clip_high=float("nan")), dict(kl=-1.0),
                                dict(kl=float("inf")), dict(kl=float("nan"))])
def test_policy_rules(kw):
    assert policy_loss(scores(), policy(**kw)) == policy_step(scores(), policy(**kw)) == -1


@pytest.mark.parametrize("kw", [dict(n_pairs=-1), dict(n_pairs=(1 << 21) + 1), dict(beta=float("nan")),
                                dict(beta=float("inf")), dict(smoothing=-0.1), dict(smoothing=0.5),
                                dict(smoothing=float("nan"))])
def test_pair_rules(kw):
    assert pref_loss(scores(), pairs(**kw)) == pref_step(scores(), pairs(**kw)) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(k=0), -1), (dict(k=33), -1), (dict(score=2), -1), (dict(score=-1), -1), (dict(scale=float("inf")), -1),
    (dict(scale=float("nan")), -1), (dict(n_groups=0), -1), (dict(n_groups=65), -1), (dict(groups_kept=0), -1),
    (dict(groups_kept=2), -1), (dict(n_groups=5, groups_kept=6), -1), (dict(group_top=0), -1), (dict(group_top=3), -1),
    (dict(n_groups=3, groups_kept=2), -2), (dict(n_groups=5, groups_kept=1), -2), (dict(k=11), -2)])
def test_routing_rules(kw, code):
    assert route(scores(), routing(**kw)) == route_grad(scores(), routing(**kw)) == code


def test_too_many_experts():
    x = scores(n_classes=1025, row_stride=1025)
    assert route(x, routing()) == route_grad(x, routing(), ld=1025) == -6


def test_no_rows_is_no_work():
    x = scores(n_rows=0, data=None)
    assert logp(x, cls=None, lp=None, ws=None) == logp_grad(x, gr=None) == 0
    assert policy_loss(x, policy(old_logp=None), lo=None) == policy_step(x, policy(), gr=None) == 0
    assert route(x, routing(), c=None) == route_grad(x, routing(), gr=None) == 0
    assert pref_loss(scores(), pairs(n_pairs=0, offsets=None), lo=None) == 0
    assert pref_step(scores(), pairs(n_pairs=0, offsets=None), gr=None) == 0


def test_python_calls_refuse_tensors():
    """A CPU tensor, and a type the operators do not take, raise ValueError."""
    x = torch.zeros(4, 10)
    ws = torch.zeros(1 << 21, dtype=torch.uint8)
    f, i, s = torch.zeros(4), torch.zeros(4, dtype=torch.int32), torch.zeros(4, 2)
    off = torch.zeros(3, dtype=torch.int64)
    r = g.make_routing(2)
    for t in (x, x.double(), x.long(), x[0]):
        with pytest.raises(ValueError):
            g.gbdt_class_logp(t, i, 1.0, f, s, ws)
        with pytest.raises(ValueError):
            g.gbdt_class_logp_grad(t, i, 1.0, s, f, x, ws)
        with pytest.raises(ValueError):
            g.gbdt_policy_loss(t, i, 1.0, f, f, f, f, 0.2, 0.2, 0.0, f, f, f, s, ws)
        with pytest.raises(ValueError):
            g.gbdt_policy_step(t, i, 1.0, f, f, f, f, 0.2, 0.2, 0.0, f, f, x, ws)
        with pytest.raises(ValueError):
            g.gbdt_preference_loss(t, i, 1.0, off, f, None, 0.1, 0.0, False, f[:1], None, f, f, s, ws)
        with pytest.raises(ValueError):
            g.gbdt_preference_step(t, i, 1.0, off, f, None, 0.1, 0.0, False, f[:1], None, x, ws)
        with pytest.raises(ValueError):
            g.gbdt_route_classes(t, r, None, i, f, ws)
        with pytest.raises(ValueError):
            g.gbdt_route_grad(t, r, i, f, x, ws)
    with pytest.raises(ValueError, match="classes"):
        g.gbdt_route_lists(i, 3, i, i, None, ws)


def test_pair_offsets_shape():
    g._load_torch()
    f, cpu = torch.zeros(4), -1
    with pytest.raises(ValueError, match="2 pairs"):
        g._pairs(cpu, (4,), torch.zeros(4, dtype=torch.int64), f, None, 0.1, 0.0, False)
    with pytest.raises(ValueError, match="offsets"):
        g._pairs(cpu, (4,), torch.zeros(3, dtype=torch.int32), f, None, 0.1, 0.0, False)
    with pytest.raises(ValueError, match="weight"):
        g._pairs(cpu, (4,), torch.zeros(3, dtype=torch.int64), f, f, 0.1, 0.0, False)
    with pytest.raises(ValueError, match="ref_logp"):
        g._pairs(cpu, (4,), torch.zeros(3, dtype=torch.int64), f[::2], None, 0.1, 0.0, False)


@pytest.mark.parametrize("bad", [torch.zeros(4).double(), torch.zeros(8)[::2], torch.zeros(3), torch.zeros(4, 1)])
def test_vectors(bad):
    g._load_torch()
    with pytest.raises(ValueError, match="loss"):
        g._at(bad, "loss", torch.float32, (4,), -1)
    with pytest.raises(ValueError, match="loss"):
        g._at(torch.zeros(4), "loss", torch.float32, (4,), 0)  # another device
    with pytest.raises(ValueError, match="loss"):
        g._at(None, "loss", torch.float32, (4,), -1)
