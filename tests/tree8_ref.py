"""Plain reference of drafted tokens over the uniform 8-bit cache: rotation by
positions of several axes (fp32, every operation rounded) and attention for trees
in 64 bits, from the definitions in include/dkv.h."""
from __future__ import annotations

import numpy as np

from tests import cache8_ref as ref


def rotate_at(x, pos, pair_axis, rope, rotary_dim, interleaved, dtype):
    """x [n][heads][128] float32, pos [axes][n] -> turned and rounded."""
    y = x.copy()
    for i in range(rotary_dim // 2):
        one, two = (2 * i, 2 * i + 1) if interleaved else (i, i + rotary_dim // 2)
        cs = rope[pos[pair_axis[i]], i].astype(np.float32)
        c, s = cs[:, None, 0], cs[:, None, 1]
        y[..., one] = x[..., one] * c - x[..., two] * s
        y[..., two] = x[..., two] * c + x[..., one] * s
    y[..., :rotary_dim] = ref.round_elem(y[..., :rotary_dim], dtype)
    return y


def depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def seen(parents, m, n, window, sinks):
    """Stored tokens and drafts that node m sees."""
    d = depths(parents)
    p = n + d[m]
    within = lambda j: not window or j > p - window or j < sinks
    stored = [j for j in range(n) if within(j)]
    drafts, x = [], m
    while x >= 0:
        if within(n + d[x]):
            drafts.append(x)
        x = parents[x]
    return stored, sorted(drafts)


def random_tree(rng, m, back=8):
    return [int(rng.integers(max(-1, i - back), i)) for i in range(m)]
