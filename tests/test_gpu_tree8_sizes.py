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


# ------------------------------------------------------------------ values far from 1

def close(got, q, k, v, size, elem):
    """Attention of q [G][128] over k, v [n][128] in 64 bits and its bound: weights rounded
    to fp16 (2^-11), and where they lie under 2^-21 of the row's largest weight times size
    (a token's or its block's largest |v|) off by half of fp16's smallest step: weights
    stand 2^7 above their place beside values of at most 448, the row's largest beside
    one that came to 128 or more, so that is 2^-25 * 448 / (2^7 * 128) < 2^-30 of the largest
    p * size for a token. Logits and exponentials as in cache8_ref.tolerance."""
    s = q @ k.T / np.sqrt(128)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    want, pv = p @ v, p @ np.abs(v)
    qk = (np.abs(q) @ np.abs(k).T).max() / np.sqrt(128)
    d = 2.0 ** -11 + 2 * 128 * 2.0 ** -23 * qk + 2.0 ** -21
    tol = torch.finfo(elem).eps / 2 * np.abs(want) * (1 + d) + d * pv
    tol += len(k) * 2.0 ** -30 * (p * size).max(axis=1, keepdims=True)
    tol += torch.finfo(elem).tiny * torch.finfo(elem).eps / 2           # half of the type's smallest step
    err = np.abs(got - want)
    return (err <= tol).all(), float((err / tol).max())


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("heavy", ["draft", "tail"])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -8, 2.0 ** -11, 2.0 ** -13, 300.0])
@pytest.mark.parametrize("n,T,log", [(4100, 128, 14), (12100, 128, 14), (66, 64, 5.5), (66, 64, 7), (66, 64, 8.3), (65, 16, 7.5), (35, 32, 6)])
def test_light_tokens_beside_a_heavy_one(elem, heavy, size, n, T, log):
    """One token of 16 bits with 2^log times the weight of each of many codes, which hold a
    good part of the mass all the same and round alike, also where they enter the products
    together; values of any size around a mean."""
    rng = np.random.default_rng(41)
    G = 4
    c = make(1, G, T, 1, n // T + 1, elem, E4M3, 1, seed=14)
    q = torch.from_numpy(np.repeat(rng.standard_normal((1, 1, 128)), G, 1).astype(np.float32)).to(elem).cuda()
    own = q[:, :1] * (log * np.log(2) * np.sqrt(128) / float((q[0, 0].double() ** 2).sum()))
    value = lambda m: torch.from_numpy((size * (1 + 0.3 * rng.standard_normal((m, 1, 128)))).astype(np.float32)).to(elem).cuda()
    k, v = torch.from_numpy((0.001 * rng.standard_normal((n, 1, 128))).astype(np.float32)).to(elem).cuda(), value(n)
    if heavy == "tail":
        k[n - 1] = own
    c.append([0], [0], [n], k, v)
    dk = own if heavy == "draft" else torch.zeros_like(own)
    dv = value(1)
    out = run_tree(c, [n], None, q, dk, dv)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    ks, vs = (np.concatenate([x, y.double().cpu().numpy()[0]]) for x, y in zip(c.ref.values(0, n, 0), (dk, dv)))
    block = np.abs(vs).max(axis=1)
    for b in range(n // T):
        block[b * T:(b + 1) * T] = block[b * T:(b + 1) * T].max()
    ok, worst = close(out[0].double().cpu().numpy(), q[0].double().cpu().numpy(), ks, vs, block, elem)
    assert ok, worst


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("where", ["drafts", "tail"])
def test_values_of_many_sizes_side_by_side(elem, where):
    """Neighbouring tokens whose values lie many powers of two apart, seen one by one (chains
    behind a short window): each row within the bound of what it sees."""
    rng = np.random.default_rng(42)
    M, T, n = 24, 64, 56
    c = make(2, 2, T, 1, 1, elem, INT8, M, seed=15)
    low, high = (-12, 12) if elem == F16 else (-90, 90)
    powers = lambda m: torch.from_numpy(2.0 ** rng.integers(low, high, (m, 1, 1)).astype(np.float32)).cuda()
    k, v = c.vec(rng, n, 2), c.vec(rng, n, 2)
    if where == "tail":
        v = (v.float() * powers(n)).to(elem)
    c.append([0], [0], [n], k, v)
    q, dk, dv = drafts(c, rng, 1, M)
    if where == "drafts":
        dv = (dv.float() * powers(M)).to(elem)
    parents = [list(range(-1, M - 1))]
    for window in (1, 2, 5, 0):
        out = run_tree(c, [n], parents, q, dk, dv, window=window).double().cpu().numpy()
        assert c.c.status_words.tolist() == [0, 0]
        for h in range(2):
            ks, vs = c.ref.values(0, n, h)
            for m in range(M):
                st, dr = tref.seen(parents[0], m, n, window, 0)
                kk = np.concatenate([ks[st], dk.double().cpu().numpy()[dr, h]])
                vv = np.concatenate([vs[st], dv.double().cpu().numpy()[dr, h]])
                ok, worst = close(out[m, 2 * h:2 * h + 2], q.double().cpu().numpy()[m, 2 * h:2 * h + 2], kk, vv,
                                  np.abs(vv).max(axis=1), elem)
                assert ok, (window, h, m, worst)


@pytest.mark.parametrize("up", [-100, -108, -114, -119, -123])
@pytest.mark.parametrize("n", [0, 21, 150])
def test_the_smallest_values_stay(up, n):
    """bf16 values near the type's smallest normal number, and nothing else in sight: a window
    of one and two positions over drafts, and what the tail holds."""
    rng = np.random.default_rng(43)
    M = 5
    c = make(2, 3, 128, 1, 2, BF16, E4M3, M, seed=16)
    k, v = c.vec(rng, max(n, 1), 2), c.vec(rng, max(n, 1), 2)
    v[max(n, 128) - 128:] *= 2.0 ** up
    if n:
        c.append([0], [0], [n], k[:n], v[:n])
    q, dk, dv = drafts(c, rng, 1, M)
    dv *= 2.0 ** up
    parents = [[-1, 0, 1, 0, -1]]
    for window in (1, 2, 10):
        out = run_tree(c, [n], parents, q, dk, dv, window=window).double().cpu().numpy()
        assert c.c.status_words.tolist() == [0, 0]
        qn, kn, vn = (x.double().cpu().numpy() for x in (q, dk, dv))
        for h in range(2):
            ks, vs = c.ref.values(0, n, h) if n else (np.zeros((0, 128)),) * 2
            for m in range(M):
                st, dr = tref.seen(parents[0], m, n, window, 0)
                kk, vv = np.concatenate([ks[st], kn[dr, h]]), np.concatenate([vs[st], vn[dr, h]])
                g = slice(3 * h, 3 * h + 3)
                ok, worst = close(out[m, g], qn[m, g], kk, vv, np.abs(vv).max(axis=1), BF16)
                assert ok, (window, h, m, worst)


# ------------------------------------------------------------------ rows that are computed again

def check_again(c, out, lens, parents, q, k, v, feature, window=0, sinks=0, nodes=None):
    """All rows see an infinite V at one feature: infinite there, within the bound of
    cache8_ref.tolerance everywhere else."""
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    M, rest = len(parents[0]), np.arange(128) != feature
    got, qn, kn, vn = (x.double().cpu().numpy() for x in (out, q, k, v))
    assert np.isinf(got[..., feature]).all()
    for i, n in enumerate(lens):
        for h in range(c.hkv):
            ks, vs = c.ref.values(i, n, h) if n else (np.zeros((0, 128)),) * 2
            g = slice(h * c.G, (h + 1) * c.G)
            for m in range(M) if nodes is None else nodes:
                st, dr = tref.seen(parents[i], m, n, window, sinks)
                rows = [i * M + x for x in dr]
                kk, vv = np.concatenate([ks[st], kn[rows, h]]), np.concatenate([vs[st], vn[rows, h]])[:, rest]
                s = qn[i * M + m, g] @ kk.T / np.sqrt(128)
                p = np.exp(s - s.max(axis=1, keepdims=True))
                p /= p.sum(axis=1, keepdims=True)
                want, qk = p @ vv, float((np.abs(qn[i * M + m, g]) @ np.abs(kk).T).max() / np.sqrt(128))
                tol = ref.tolerance(want, p @ np.abs(vv), qk, float(np.abs(vv).max()), len(kk), c.elem, 2.0 ** -11)
                err = np.abs(got[i * M + m, g][:, rest] - want)
                assert (err <= tol).all(), (i, h, m, float((err / tol).max()))


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
@pytest.mark.parametrize("T,window,sinks", [(16, 0, 0), (128, 0, 0), (32, 300, 5), (64, 4200, 20), (128, 70, 0)])
def test_rows_computed_again(elem, code, T, window, sinks):
    """From one token to more than 4096 (a second round of lookups), random logits, trees below
    one root with an infinite feature."""
    rng = np.random.default_rng(51)
    lens, M = [4399, 150, 1, 0], 18
    c = make(2, 3, T, len(lens), 4399 // T + 1, elem, code, M, seed=17, fill=NAN)
    fill(c, rng, lens)
    parents = [[-1] + [max(0, x) for x in tref.random_tree(rng, M)[1:]] for _ in lens]
    q, k, v = drafts(c, rng, len(lens), M)
    v[::M, :, 9] = float("inf")
    out = run_tree(c, lens, parents, q, k, v, window=window, sinks=sinks)
    check_again(c, out, lens, parents, q, k, v, 9, window, sinks, nodes=(0, 1, 5, M - 2, M - 1))


@pytest.mark.parametrize("up", [-116, 116])
def test_huge_and_tiny_logits_computed_again(up):
    """bf16 keys of 2^116 (2^-116) and queries that bring them back, in rows that see the
    infinite value."""
    rng = np.random.default_rng(52)
    n, M = 150, 6
    c = make(1, 4, 32, 1, 8, BF16, E4M3, M, seed=11)
    k, v = c.vec(rng, n, 1), c.vec(rng, n, 1)
    if up > 0:
        k *= 2.0 ** up
    c.append([0], [0], [n], k, v)
    q, dk, dv = drafts(c, rng, 1, M)
    if up > 0:
        q *= 2.0 ** -up
        dk *= 2.0 ** up
    else:
        q[1] *= 2.0 ** up
        dk[3] *= 2.0 ** up
    parents = [[-1, 0, 0, 1, 1, 2]]
    dv[0, :, 9] = float("inf")
    check_again(c, run_tree(c, [n], parents, q, dk, dv), [n], parents, q, dk, dv, 9)


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("sign", ["plus", "both"])
@pytest.mark.parametrize("n", [0, 90, 2000])
def test_largest_values_computed_again(elem, sign, n):
    """V of the type's largest size: means of finite values are finite in rows that are
    computed again, too."""
    rng = np.random.default_rng(53)
    big, M = torch.finfo(elem).max, 7
    c = make(1, 2, 32, 1, 2000 // 32 + 1, elem, INT8, M, seed=18)
    signs = lambda m: torch.from_numpy(rng.choice([-1.0, 1.0], (m, 1, 128)) if sign == "both" else np.ones((m, 1, 128))).to(elem).cuda()
    if n:
        c.append([0], [0], [n], c.vec(rng, n, 1) * 0.05, big * signs(n))
    q, k, v = drafts(c, rng, 1, M)
    k *= 0.05
    v = big * signs(M)
    v[0, :, 9] = float("inf")
    parents = [[-1, 0, 0, 1, 2, 2, 5]]
    out = run_tree(c, [n], parents, q, k, v)
    check_again(c, out, [n], parents, q, k, v, 9)
    assert torch.isfinite(out[..., 10:].float()).all()


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("n,M", [(0, 3), (20, 5), (120, 100)])
def test_rows_of_nothing_but_minus_infinity(elem, n, M):
    """Logits that are all -Inf have no softmax: NaN, in a unit of one block and in one that
    several hold parts of; one finite logit beside them makes that token's value."""
    rng = np.random.default_rng(54)
    c = make(1, 2, 128, 1, 2, elem, E4M3, M, seed=19)
    k, v = c.vec(rng, max(n, 1), 1), c.vec(rng, max(n, 1), 1)
    k[..., 5] = float("-inf")
    if n:
        c.append([0], [0], [n], k, v)
    q, dk, dv = drafts(c, rng, 1, M)
    q[..., 5] = 1.0
    dk[..., 5] = float("-inf")
    dk[M - 1, :, 5] = 1.0
    parents = [list(range(-1, M - 1))]
    out = run_tree(c, [n], parents, q, dk, dv)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    assert torch.isnan(out[:M - 1].float()).all()
    assert torch.equal(out[M - 1].float(), dv[M - 1].float().expand(2, 128))


# ------------------------------------------------------------------ blocks that rows see a part of

def hidden_sizes():
    return [(e, c, w, x) for e in (F16, BF16) for c in (E4M3, INT8) for w, x in
            (("k", 1e18), ("k", 3e4), ("v", 1e4), ("v", 1e9), ("v", 1e18), ("v", -3e38)) if abs(x) <= torch.finfo(e).max]


@pytest.mark.parametrize("T,n,window,sinks", [(64, 300, 151, 0), (128, 700, 300, 20), (32, 200, 90, 40), (16, 333, 40, 3),
                                              (128, 260, 5, 130), (64, 400, 395, 0)])
@pytest.mark.parametrize("elem,code,what,size", hidden_sizes())
def test_finite_codes_that_are_not_seen(elem, code, T, n, window, sinks, what, size):
    """Stored tokens of any size that a window, or the first tokens, leave out of a block whose
    rest rows see: they set the block's scale, with which the rest is stored, and no more. The
    shallow nodes see some of them, which is their own affair."""
    rng = np.random.default_rng(61)
    M = 24
    c = make(2, 3, T, 1, n // T + 1, elem, code, M, seed=20, fill=NAN)
    k, v = c.vec(rng, n, 2), c.vec(rng, n, 2)
    x = k if what == "k" else v
    first = n - window + 1                   # a root sees those from here on
    hidden = [j for j in (first - 1, first - 9, sinks, sinks + 5) if sinks <= j < first]
    assert hidden
    x[hidden] = size
    deep = first + 3                         # seen by nodes of a depth up to 2
    x[deep] = size
    c.append([0], [0], [n], k, v)
    parents = [list(range(-1, 11)) + [-1, 12, 13, 14, 2, 2, 16, 17, 18, 9, 9, 9]]
    q, dk, dv = drafts(c, rng, 1, M)
    out = run_tree(c, [n], parents, q, dk, dv, window=window, sinks=sinks)
    assert c.c.status_words.tolist() == [0, 0]
    depth = np.array(tref.depths(parents[0]))
    check_tree(c, out, [n], parents, q, dk, dv, [M], window=window, sinks=sinks, nodes=set(np.flatnonzero(depth > 2).tolist()))
