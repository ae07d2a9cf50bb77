"""Refusals of the operators on rows of class scores: the C entry points check
what the host can see before any device work, the Python calls the tensors'
types, shapes and strides."""
import ctypes

import pytest
import torch

import histogram_split_finding_amd as g

FAKE = 0x10000  # an aligned address that is never read


def scores(**kw):
    a = dict(data=FAKE, n_rows=4, row_stride=10, n_classes=10, dtype=0)
    a.update(kw)
    return g.Scores(*[a[k] for k in ("data", "n_rows", "row_stride", "n_classes", "dtype")])


def teacher(**kw):
    a = dict(values=FAKE, classes=FAKE, rest=None, k=3, pad=0)
    a.update(kw)
    return g.Teacher(*[a[k] for k in ("values", "classes", "rest", "k", "pad")])


BAD_SCORES = [
    (dict(data=None), -1), (dict(data=FAKE + 2), -1), (dict(data=FAKE + 1, dtype=1), -1), (dict(n_rows=-1), -1),
    (dict(n_rows=(1 << 31) + 1), -1), (dict(n_classes=0), -1), (dict(n_classes=g.MAX_CLASSES + 1), -1),
    (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(row_stride=9), -2),
]
WS = 1 << 20


def top(x, k=3, T=1.0, v=FAKE, c=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_top_scores(ctypes.byref(x) if x else None, k, T, v, c, None, ws, nb, None)


def loss(x, t, T=1.0, lo=FAKE, st=FAKE, ws=FAKE, nb=WS):
    return g.load().gbdt_distill_loss(ctypes.byref(x) if x else None, ctypes.byref(t) if t else None, T, lo, st,
                                      ws, nb, None)


def grad(x, t, T=1.0, st=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_distill_grad(ctypes.byref(x) if x else None, ctypes.byref(t) if t else None, T, st, None,
                                      gr, ld, ws, nb, None)


def step(x, t, T=1.0, lo=FAKE, gr=FAKE, ld=10, ws=FAKE, nb=WS):
    return g.load().gbdt_distill_step(ctypes.byref(x) if x else None, ctypes.byref(t) if t else None, T, None, lo,
                                      gr, ld, ws, nb, None)


def sample(x, u=FAKE, p=True, out=FAKE, ws=FAKE, nb=WS):
    q = g.Sampling(None, None, None, None)
    return g.load().gbdt_sample_classes(ctypes.byref(x) if x else None, u, ctypes.byref(q) if p else None, out,
                                        None, ws, nb, None)


@pytest.mark.parametrize("kw,code", BAD_SCORES)
def test_scores_rules(kw, code):
    x = scores(**kw)
    assert top(x) == code and g.last_error()
    assert loss(x, teacher()) == code
    assert grad(x, teacher()) == code
    assert step(x, teacher()) == code
    assert sample(x) == code


def test_null_and_size_rules():
    x, t = scores(), teacher()
    for rc in (top(None), loss(None, t), grad(None, t), step(None, t), sample(None), loss(x, None), grad(x, None),
               step(x, None), sample(x, p=False), top(x, v=None), top(x, c=None), loss(x, t, lo=None),
               loss(x, t, st=None), grad(x, t, st=None), grad(x, t, gr=None), grad(x, t, gr=FAKE + 1),
               step(x, t, lo=None), step(x, t, gr=None), step(x, t, gr=FAKE + 2), sample(x, u=None),
               sample(x, out=None), loss(x, teacher(values=None)), loss(x, teacher(classes=None)),
               loss(x, teacher(k=0)), loss(x, teacher(k=g.MAX_LISTED + 1)), top(x, k=0),
               top(scores(n_classes=1000, row_stride=1000), k=g.MAX_LISTED + 1)):
        assert rc == -1 and g.last_error()
    assert top(x, k=11) == -2
    assert grad(x, t, ld=9) == -2 and step(x, t, ld=9) == -2
    need = g.gbdt_scores_workspace_bytes(4, 10)
    assert need >= 256
    for kw in (dict(ws=None), dict(ws=FAKE + 128), dict(nb=need - 1)):
        assert top(x, **kw) == loss(x, t, **kw) == grad(x, t, **kw) == step(x, t, **kw) == sample(x, **kw) == -1


@pytest.mark.parametrize("T", [0.0, -1.0, float("nan"), float("inf")])
def test_temperature_rules(T):
    x, t = scores(), teacher()
    assert top(x, T=T) == loss(x, t, T=T) == grad(x, t, T=T) == step(x, t, T=T) == -1


def test_no_rows_is_no_work():
    x, t = scores(n_rows=0, data=None), teacher(values=None, classes=None)
    assert top(x, v=None, c=None, ws=None) == loss(x, t, lo=None) == grad(x, t, gr=None) == 0
    assert step(x, t, gr=None) == sample(x, u=None, out=None) == 0


def test_workspace_sizes():
    assert g.gbdt_scores_workspace_bytes(-1, 5) == 0
    assert g.gbdt_scores_workspace_bytes(5, 0) == 0
    assert g.gbdt_scores_workspace_bytes(5, g.MAX_CLASSES + 1) == 0
    assert g.gbdt_scores_workspace_bytes(5, g.MAX_CLASSES) > 0


def test_python_calls_refuse_tensors():
    """A CPU tensor, and a type the operators do not take, raise ValueError."""
    x = torch.zeros(4, 10)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    f, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    v, c = torch.zeros(4, 3), torch.zeros(4, 3, dtype=torch.int32)
    for t in (x, x.double(), x.long(), x[0]):
        with pytest.raises(ValueError):
            g.gbdt_top_scores(t, 3, 1.0, v, c, f, ws)
        with pytest.raises(ValueError):
            g.gbdt_distill_step(t, v, c, f, 1.0, None, f, x, ws)
        with pytest.raises(ValueError):
            g.gbdt_sample_classes(t, f, None, None, None, None, i, f, ws)


@pytest.mark.parametrize("name,bad", [
    ("values", torch.zeros(4, 3).double()), ("values", torch.zeros(3, 4).t()), ("classes", torch.zeros(4, 3)),
    ("rest", torch.zeros(5)), ("values", torch.zeros(5, 3))])
def test_python_vectors(name, bad):
    x = torch.zeros(4, 10)
    shape = (4,) if name == "rest" else (4, 3)
    dtype = torch.int32 if name == "classes" else torch.float32
    with pytest.raises(ValueError, match=name):
        g._vector(bad, name, dtype, shape, x)
