"""The same inputs give the same classes, log-probabilities and rests, also
where several waves list a row's likely classes side by side."""
import numpy as np
import pytest
import torch

import histogram_split_finding_amd as g
import scores_ref as ref
from gpu_util import DEV, say, to_dev

pytestmark = pytest.mark.gpu

CLASSES = 65536


def border_rows(n, seed):
    """Rows of 65,536 f32 scores whose top-p cut falls, at top_p = 1/4, between
    the last of some equal best classes and the next of them, to within a few
    of the last bits of an FP64 sum: row i's mass is (i - n / 2) 2^-45 away
    from the border as long double sums tell it.  The mass is in vectors of
    four classes that hold a best class, and in the first vectors' others."""
    r = np.random.default_rng(seed)
    x = np.full(CLASSES, -1000.0, dtype=np.float32)
    best = (np.arange(160) * 102.4).astype(int) * 4
    lower = np.concatenate([best + 1, best + 2, best + 3])
    side = np.setdiff1d(np.arange(2048) * 4, best)[:101]
    free = side[-1] + np.arange(4)
    lower = np.concatenate([lower] + [side[:-1] + q for q in range(4)])
    x[best] = 0.0
    x[lower] = -r.uniform(0.55, 1.6, len(lower)).astype(np.float32)

    def mass(v):
        return np.exp2((v.astype(np.float64) * 1.44269504088896340736).astype(np.longdouble)).sum()

    left = np.longdouble(0.0)
    j = int(np.ceil(mass(x) / 4))
    while True:  # lower ones a little higher until what is left fits the free places
        left = 4 * j - mass(x)
        if left < 0.5:
            break
        x[r.choice(lower)] = -0.55
    for at in free[:3]:
        v = np.float32(np.log(np.float64(left - n * 2.0 ** -45)))  # (some stays for the last place)
        x[at] = np.nextafter(v, np.float32(-np.inf))
        left = 4 * j - mass(x)
    rows = np.repeat(x[None], n, 0)
    for i in range(n):
        up = left + (i - n / 2 + 0.5) * 2.0 ** -45
        rows[i, free[3]] = np.log(np.float64(up))
    return rows, best, j


@pytest.mark.parametrize("n", [128, 300])
def test_cut_next_to_a_border(n):
    """1,024 and 512 threads a row: the draw of the last kept class, again and
    again."""
    say("border: %d rows" % n)
    rows, best, j = border_rows(n, 5)
    x = to_dev(rows)
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(n, CLASSES))
    u = torch.full((n,), 1.0 - 2.0 ** -24, device=DEV)
    top_p, min_p = torch.full((n,), 0.25, device=DEV), torch.full((n,), 0.9, device=DEV)
    out, logp = torch.zeros(n, dtype=torch.int32, device=DEV), torch.zeros(n, device=DEV)
    seen = []
    for _ in range(40):
        g.gbdt_sample_classes(x, u, None, None, top_p, min_p, out, logp, ws)
        seen.append((out.cpu(), logp.cpu()))
    # the border is where it was meant to be: on both sides of it some rows
    first = seen[0][0].numpy()
    assert set(first.tolist()) == {int(best[j - 1]), int(best[j])}
    changed = set()
    for other in seen[1:]:
        changed |= set(np.flatnonzero(other[0].numpy() != first).tolist())
        changed |= set(torch.nonzero(other[1] != seen[0][1])[:, 0].tolist())
    assert not changed, sorted(changed)
    assert g.gbdt_read_error(ws) == 0


@pytest.mark.parametrize("C,n,dtype", [(40001, 2, "f32"), (66001, 300, "bf16"), (66001, 20, "bf16"), (20011, 30, "f16")])
def test_streams_and_graphs(C, n, dtype):
    """On another stream, and captured and replayed with eager work in between:
    draws with top-p and min-p, and records, to the bit."""
    say("repeats: %d x %d %s" % (n, C, dtype))
    x, _ = ref.rows(n, C, dtype, C)
    r = np.random.default_rng(n)
    u = to_dev(r.random(n).astype(np.float32))
    top_p = to_dev(r.uniform(0.5, 0.99, n).astype(np.float32))
    min_p = to_dev(r.uniform(0.001, 0.1, n).astype(np.float32))
    ws = g.new_workspace(g.gbdt_scores_workspace_bytes(n, C))
    v, c = torch.zeros(n, 20, device=DEV), torch.zeros(n, 20, dtype=torch.int32, device=DEV)
    rest, logp = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    out = torch.zeros(n, dtype=torch.int32, device=DEV)

    def work():
        g.gbdt_top_scores(x, 20, 1.0, v, c, rest, ws)
        g.gbdt_sample_classes(x, u, None, None, top_p, min_p, out, logp, ws)

    def taken():
        torch.cuda.synchronize()
        got = [t.cpu() for t in (v, c, rest, out, logp)]
        for t in (v, c, rest, out, logp):
            t.zero_()
        torch.cuda.synchronize()
        return got

    work()
    want = taken()
    s = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s):
            work()
        for a, b in zip(want, taken()):
            assert torch.equal(a, b)
    with torch.cuda.stream(s):
        work()
    taken()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for _ in range(3):
        taken()
        graph.replay()
        for a, b in zip(want, taken()):
            assert torch.equal(a, b)
        work()
        for a, b in zip(want, taken()):
            assert torch.equal(a, b)
    assert g.gbdt_read_error(ws) == 0
