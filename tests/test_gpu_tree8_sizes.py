"""GPU tests of tree attention over values of all sizes: finite values that rows do
not see, values far from 1, rows that are computed again from the formula. Against
64 bits within bounds that are derived beside them."""
from __future__ import annotations

import numpy as np
import pytest

from tests import cache8_ref as ref
from tests import tree8_ref as tref
from tests.test_gpu_tree8 import check_tree, drafts, fill, gpu, i32, make, run_tree  # noqa: F401 (gpu: a fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3, INT8, F16, BF16 = torch.float8_e4m3fn, torch.int8, torch.float16, torch.bfloat16
NAN = float("nan")


def check_request(c, out, i, n, parents, q, k, v, nodes, **kw):
    """check_tree for some nodes of request i alone."""
    M = len(parents)
    rows = slice(i * M, (i + 1) * M)
    check_tree(c, out[rows], [n], [parents], q[rows], k[rows], v[rows], [M], slots=[i], nodes=set(nodes), **kw)


# ------------------------------------------------------------------ finite values that rows do not see

def unseen_sizes():
    return [(e, w, x) for e in (F16, BF16) for w in "kv" for x in (1e3, 1e6, 1e9, 1e18, -torch.finfo(e).max)
            if abs(x) <= torch.finfo(e).max]


@pytest.mark.parametrize("elem,what,size", unseen_sizes())
def test_finite_drafts_that_are_not_seen(elem, what, size):
    """A draft of any size beside others in its tile: rows that do not see it keep the
    bound of what they see."""
    rng = np.random.default_rng(31)
    lens, M = [40, 700], 12
    c = make(2, 4, 16, 2, 50, elem, E4M3, M, seed=6, fill=NAN)
    fill(c, rng, lens)
    parents = [[-1, -1, 0, 0, 1, 1, 2, 3, 4, 5, 6, 9], list(range(-1, M - 1))]
    q, k, v = drafts(c, rng, 2, M)
    x = k if what == "k" else v
    x[3, :, 5] = size
    x[M + 8] = size
    out = run_tree(c, lens, parents, q, k, v)
    check_request(c, out, 0, 40, parents[0], q, k, v, [m for m in range(M) if 3 not in tref.seen(parents[0], m, 40, 0, 0)[1]])
    check_request(c, out, 1, 700, parents[1], q, k, v, range(8))


@pytest.mark.parametrize("elem,what,size", unseen_sizes())
@pytest.mark.parametrize("T,n", [(64, 60), (128, 500)])
def test_finite_tail_entries_behind_the_window(elem, what, size, T, n):
    """Stored tokens of any size in tiles of the tail that rows see the rest of: just
    behind the window and between it and the first tokens."""
    rng = np.random.default_rng(32)
    M, window, sinks = 8, 12, 3
    c = make(2, 3, T, 1, n // T + 1, elem, INT8, M, seed=12, fill=NAN)
    k, v = c.vec(rng, n, 2), c.vec(rng, n, 2)
    x = k if what == "k" else v
    x[n - window] = size                  # a root sees those from n - window + 1 on
    if T == 64:
        x[5, 1, 17] = size                # in the tail, beside the first tokens
    c.append([0], [0], [n], k, v)
    parents = [tref.random_tree(rng, M, 4)]
    q, dk, dv = drafts(c, rng, 1, M)
    out = run_tree(c, [n], parents, q, dk, dv, window=window, sinks=sinks)
    check_tree(c, out, [n], parents, q, dk, dv, [M], window=window, sinks=sinks)


def test_queries_of_other_rows_do_not_matter():
    """bf16 queries of the largest and smallest sizes in rows beside each other."""
    rng = np.random.default_rng(33)
    n, M = 100, 8
    c = make(1, 4, 16, 1, 8, BF16, INT8, M, seed=13)
    fill(c, rng, [n])
    q, k, v = drafts(c, rng, 1, M)
    for m, f in ((1, 1e30), (3, 1e-30), (4, 0.0), (6, 1e18)):
        q[m] *= f
    parents = [[-1] * M]
    out = run_tree(c, [n], parents, q, k, v)
    check_tree(c, out, [n], parents, q, k, v, [M], nodes={0, 2, 3, 4, 5, 7})
