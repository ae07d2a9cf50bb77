"""Pairs of very different lengths: each number of threads a pair, and more rows of a
pair than a thread keeps bits for."""
import numpy as np
import pytest

import scores_ref as ref
from gpu_util import say
from test_gpu_learn import check_pairs, draw_classes

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pairs,long,short", [(2048, 5000, 4), (20, 12000, 10), (1, 40000, 0), (2, 3500, 500),
                                              (512, 900, 3)])
@pytest.mark.parametrize("masked", [False, True])
def test_one_long_pair(pairs, long, short, masked):
    say("pairs: %d, one of %d rows, masked %s" % (pairs, long, masked))
    sizes = [long // 3, long - long // 3] + [short] * (2 * (pairs - 1))
    cuts = np.concatenate([[1], 1 + np.cumsum(sizes)]).tolist()
    n, C = cuts[-1] + 3, 5
    x, xh = ref.rows(n, C, "f32", pairs)
    cls = draw_classes(xh, pairs)
    if masked:  # classes of score -inf, early and late, in the sequence that is preferred
        for i in (cuts[0], cuts[1] - 1, (cuts[0] + cuts[1]) // 2):
            cls[i] = 2
            x[i, 2] = float("-inf")
            xh[i, 2] = -np.inf
    check_pairs(x, xh, cls, 1.0, "f32", cuts, 0.01, 0.1, False)
