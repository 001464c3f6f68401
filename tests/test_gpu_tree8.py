"""GPU tests of drafted tokens over the uniform 8-bit cache (tree attention,
accepted drafts, rotation and append at positions of several axes): stored state
and turned vectors bit for bit, attention against 64 bits within the bound of
cache8_ref.tolerance."""
from __future__ import annotations

import numpy as np
import pytest

from tests import cache8_ref as ref
from tests import tree8_ref as tref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3, INT8, F16, BF16 = torch.float8_e4m3fn, torch.int8, torch.float16, torch.bfloat16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _dkv().build.build()
    _dkv().load()


def _dkv():
    import differentiated_kv_cache_gb300 as dkv
    return dkv


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def make(hkv, G, T, slots, width, elem, code, max_nodes, **kw):
    from tests.test_gpu_cache8 import Cache
    c = Cache(hkv, G, T, slots, width, elem, code, **kw)
    c.c = _dkv().make_cache8(c.pages, c.scales, c.tail, c.table, group_size=G, rotary_dim=c.rot, rotary_interleaved=c.inter,
                             max_nodes=max_nodes)
    return c


def fill(c, rng, lens, slots=None):
    """Store lens[i] tokens in slots[i], a request at a time."""
    for i, n in enumerate(lens):
        if n > 0:
            c.append([i if slots is None else slots[i]], [0], [n], c.vec(rng, n, c.hkv), c.vec(rng, n, c.hkv))


def run_tree(c, lens, parents, q, k, v, n_nodes=None, slots=None, out=None, **kw):
    out = torch.full((q.shape[0], c.hkv * c.G, 128), NAN, dtype=c.elem, device="cuda") if out is None else out
    _dkv().dkv_cache8_tree(c.c, i32(lens), None if parents is None else i32(parents), q, k, v, out,
                           n_nodes=None if n_nodes is None else i32(n_nodes), slots=None if slots is None else i32(slots), **kw)
    return out


def check_tree(c, out, lens, parents, q, k, v, n_nodes, slots=None, window=0, sinks=0, nodes=None):
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    M = q.shape[0] // len(lens)
    got, qn, kn, vn = (x.double().cpu().numpy() for x in (out, q, k, v))
    for i, n in enumerate(lens):
        n = max(n, 0)
        m_i = n_nodes[i]
        for h in range(c.hkv):
            ks, vs = c.ref.values(i if slots is None else slots[i], n, h) if n and m_i > 0 else (np.zeros((0, 128)),) * 2
            g = slice(h * c.G, (h + 1) * c.G)
            for m in range(max(m_i, 0)):
                if nodes is not None and m not in nodes:
                    continue
                st, dr = tref.seen(parents[i], m, n, window, sinks)
                rows = [i * M + x for x in dr]
                kk, vv = np.concatenate([ks[st], kn[rows, h]]), np.concatenate([vs[st], vn[rows, h]])
                want, pv, qk, vm = ref.attend(qn[i * M + m, g], kk, vv)
                tol = ref.tolerance(want, pv, qk, vm, len(kk), c.elem, 2.0 ** -11)
                err = np.abs(got[i * M + m, g] - want)
                assert (err <= tol).all(), (i, h, m, n, float((err / tol).max()), float(np.nanmax(err)))
        if m_i < M:
            assert np.isnan(got[i * M + max(m_i, 0):(i + 1) * M]).all(), "rows behind a request's nodes"


def drafts(c, rng, n_req, M, n_nodes=None):
    q, k, v = c.vec(rng, n_req * M, c.hkv * c.G), c.vec(rng, n_req * M, c.hkv), c.vec(rng, n_req * M, c.hkv)
    if n_nodes is not None:            # rows behind the nodes hold NaN
        for i, m in enumerate(n_nodes):
            for x in (q, k, v):
                x[i * M + max(m, 0):(i + 1) * M] = NAN
    return q, k, v


# ------------------------------------------------------------------ tree attention

@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
@pytest.mark.parametrize("T,G,M", [(16, 4, 9), (32, 3, 17), (64, 8, 16), (128, 5, 26), (64, 1, 1), (32, 7, 2)])
def test_ragged_trees(elem, code, T, G, M):
    """Lengths around the borders of tiles and blocks (none stored among them), trees of
    one node to M, crossed slots; unwritten places hold NaN."""
    rng = np.random.default_rng(T + G)
    lens = [0, 1, 15, 16, T - 1, T, T + 1, 3 * T + 5, 200, 333]
    n = len(lens)
    c = make(2, G, T, n, 400 // T + 1, elem, code, M, seed=T, fill=NAN)
    slots = [int(x) for x in rng.permutation(n)]
    fill(c, rng, lens, slots)
    n_nodes = [M] + [int(rng.integers(1, M + 1)) for _ in range(n - 1)]
    parents = [tref.random_tree(rng, M) for _ in range(n)]
    q, k, v = drafts(c, rng, n, M, n_nodes)
    out = run_tree(c, lens, parents, q, k, v, n_nodes, slots)
    check_tree(c, out, lens, parents, q, k, v, n_nodes, slots)


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 0), (5, 1), (16, 20), (40, 4), (64, 0), (150, 17), (400, 100), (5000, 4)])
def test_windows(elem, window, sinks):
    """Windows shorter than a path, than the stored tokens and beyond all; chains and
    trees."""
    rng = np.random.default_rng(window)
    lens, M = [0, 7, 64, 130, 431], 20
    c = make(2, 3, 32, 5, 14, elem, E4M3, M, seed=1, fill=NAN)
    fill(c, rng, lens)
    parents = [list(range(-1, M - 1)) if i % 2 else tref.random_tree(rng, M, 3) for i in range(5)]
    n_nodes = [20, 20, 13, 20, 20]
    q, k, v = drafts(c, rng, 5, M, n_nodes)
    out = run_tree(c, lens, parents, q, k, v, n_nodes, window=window, sinks=sinks)
    check_tree(c, out, lens, parents, q, k, v, n_nodes, window=window, sinks=sinks)


@pytest.mark.parametrize("elem,code,hkv,G,M,lens", [
    (F16, E4M3, 1, 8, 64, [6000]), (BF16, INT8, 2, 3, 128, [2500, 40]), (F16, INT8, 8, 4, 26, [4100, 3000, 1, 700]),
    (BF16, E4M3, 4, 8, 33, [5001])])
def test_long_and_wide(elem, code, hkv, G, M, lens):
    """Several units of 128 rows, contexts split over the GPU; some nodes are compared."""
    rng = np.random.default_rng(M)
    n = len(lens)
    c = make(hkv, G, 64, n, max(lens) // 64 + 1, elem, code, M, seed=2, fill=NAN)
    fill(c, rng, lens)
    parents = [tref.random_tree(rng, M, 20) for _ in range(n)]
    n_nodes = [M] * (n - 1) + [max(1, M - 7)]
    q, k, v = drafts(c, rng, n, M, n_nodes)
    out = run_tree(c, lens, parents, q, k, v, n_nodes)
    check_tree(c, out, lens, parents, q, k, v, n_nodes, nodes=set(range(0, M, 5)) | {M - 1, M - 8})
    again = run_tree(c, lens, parents, q, k, v, n_nodes)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


def test_chains_and_defaults():
    """No parents: chains; no counts: all nodes; no slots: in order."""
    rng = np.random.default_rng(4)
    lens, M = [100, 33], 6
    c = make(3, 2, 16, 2, 8, F16, E4M3, M, seed=3)
    fill(c, rng, lens)
    q, k, v = drafts(c, rng, 2, M)
    out = run_tree(c, lens, None, q, k, v)
    check_tree(c, out, lens, [list(range(-1, M - 1))] * 2, q, k, v, [M, M])


def test_one_node_is_the_decode_of_its_token():
    rng = np.random.default_rng(5)
    c = make(2, 4, 64, 3, 8, F16, E4M3, 1, seed=4)
    lens = [10, 64 + 62, 300]
    fill(c, rng, lens)
    q, k, v = drafts(c, rng, 3, 1)
    out = run_tree(c, lens, None, q, k, v)
    c.append(None, lens, [1, 1, 1], k, v, step=True)
    c.check()
    dec = c.attend(None, [x + 1 for x in lens], q)
    check_tree(c, out, lens, [[-1]] * 3, q, k, v, [1] * 3)
    c.check_attention(dec, [0, 1, 2], [x + 1 for x in lens], q)


def test_padding_and_strides():
    """Requests of no node (bad slots and lengths there), parts of one projection."""
    rng = np.random.default_rng(6)
    lens, M = [50, -3, 7, 20], 5
    c = make(2, 4, 32, 4, 4, BF16, INT8, M, seed=5)
    fill(c, rng, lens)
    qkv = c.vec(rng, 4 * M, 12)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    n_nodes, slots = [5, 0, -2, 3], [0, 99999, -5, 3]
    parents = [[-1, 0, 1, 0, 3]] * 4
    out = run_tree(c, lens, parents, q, k, v, n_nodes, slots)
    check_tree(c, out, lens, parents, q, k, v, n_nodes, slots)
    # a negative length is none
    out = run_tree(c, [-7, 50], parents[:2], q[:10], k[:10], v[:10], [5, 5], [1, 0])
    check_tree(c, out, [0, 50], parents[:2], q[:10], k[:10], v[:10], [5, 5], [1, 0])


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("bad", [NAN, float("inf"), float("-inf")])
def test_what_is_not_seen_never_enters(elem, what, bad):
    """A draft with values that are not finite: rows that do not see it come out as
    if it were not there, rows that do are not finite."""
    rng = np.random.default_rng(7)
    lens, M = [40, 700], 12
    c = make(2, 4, 16, 2, 50, elem, E4M3, M, seed=6, fill=NAN)
    fill(c, rng, lens)
    parents = [[-1, -1, 0, 0, 1, 1, 2, 3, 4, 5, 6, 9], list(range(-1, M - 1))]
    q, k, v = drafts(c, rng, 2, M)
    clean = run_tree(c, lens, parents, q, k, v)
    check_tree(c, clean, lens, parents, q, k, v, [M, M])
    x = k if what == "k" else v
    x[3, :, 5] = bad             # request 0, node 3: its descendants see it
    x[M + 8, 1, 77] = bad        # request 1, node 8 of a chain, one KV head
    out = run_tree(c, lens, parents, q, k, v).double().cpu().numpy()
    want = clean.double().cpu().numpy()
    assert c.c.status_words.tolist() == [0, 0]
    touched = np.zeros((2 * M, 8, 128), bool)
    hit = [m for m in range(M) if 3 in tref.seen(parents[0], m, 40, 0, 0)[1]]
    touched[hit, :, :] = what == "k"
    touched[hit, :, 5] = True
    touched[M + 8:, 4:, :] |= what == "k"
    touched[M + 8:, 4:, 77] = True
    if what == "k" and np.isinf(bad):
        # the logit's sign decides: +Inf makes NaN, -Inf leaves the token out
        logit = np.full((2 * M, 8), False)
        qn = q.double().cpu().numpy()
        for m in range(2 * M):
            for h in range(8):
                logit[m, h] = (qn[m, h, 5] if m < M else qn[m, h, 77]) * bad > 0
        out_here, want_here = out[touched].copy(), None
        assert np.isnan(out[touched & logit[..., None]]).all()
        assert np.isfinite(out[touched & ~logit[..., None]]).all()
    else:
        assert not np.isfinite(out[touched]).any()
    free = ~touched
    assert np.isfinite(out[free]).all()
    # recomputed rows round their weights otherwise: two roundings of weights and results apart
    tol = 2 * (torch.finfo(elem).eps / 2) * np.abs(want[free]) + 2 * 2.0 ** -10 * 40
    assert (np.abs(out[free] - want[free]) <= tol).all()


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("T,n,chain", [(64, 60, True), (64, 60, False), (16, 70, True), (128, 500, False)])
def test_stored_values_not_finite_behind_the_window(elem, T, n, chain):
    """A stored token (of the tail with T = 64 and 128, a code with T = 16) whose V is NaN: nodes
    whose window does not reach it come out as if it were not there."""
    rng = np.random.default_rng(T)
    M, window, bad = 16, 12, n - 10                 # seen by depths 0 and 1
    c = make(2, 3, T, 1, n // T + 1, elem, E4M3, M, seed=12, fill=NAN)
    fill(c, rng, [n])
    parents = [list(range(-1, M - 1)) if chain else tref.random_tree(rng, M, 8)]
    q, k, v = drafts(c, rng, 1, M)
    par = None if chain else parents
    clean = run_tree(c, [n], par, q, k, v, window=window)
    check_tree(c, clean, [n], parents, q, k, v, [M], window=window)
    feature, token = 39, bad % 16
    place = lambda bits: int(ref.PLACES[bits][1][token, feature])
    if bad // T < n // T:
        c.pages.view(torch.uint8)[int(c.table[0, bad // T]), 0, bad % T // 16, 1, place(8)] = 0x7f
    else:
        c.tail[0, 0, bad % T // 16, 1, place(16)] = NAN
    out = run_tree(c, [n], par, q, k, v, window=window)
    depth = np.array(tref.depths(parents[0]))
    check_tree(c, out, [n], parents, q, k, v, [M], window=window, nodes=set(np.flatnonzero(depth > 1).tolist()))
    hit = out.double().cpu().numpy()[depth <= 1][:, :3]
    assert np.isnan(hit[..., feature]).all()
    rest = np.arange(128) != feature
    want = clean.double().cpu().numpy()[depth <= 1][:, :3][..., rest]
    # recomputed rows round their weights otherwise: two roundings of weights and results apart
    tol = 2 * (torch.finfo(elem).eps / 2) * np.abs(want) + 2 * 2.0 ** -10 * 40
    assert (np.abs(hit[..., rest] - want) <= tol).all()


@pytest.mark.parametrize("elem", [F16, BF16])
def test_infinite_drafts_in_long_contexts_and_many_requests(elem):
    """Leaves with infinite values in some of many requests, whose units are split and lie
    behind one another: only rows that see them change."""
    rng = np.random.default_rng(17)
    lens, M = [1500, 3, 40, 900, 0, 333, 64, 17, 129, 700], 10
    n = len(lens)
    c = make(3, 4, 32, n, 1500 // 32 + 1, elem, INT8, M, seed=13, fill=NAN)
    fill(c, rng, lens)
    parents = [tref.random_tree(rng, M) for _ in range(n)]
    q, k, v = drafts(c, rng, n, M)
    clean = run_tree(c, lens, parents, q, k, v)
    check_tree(c, clean, lens, parents, q, k, v, [M] * n)
    leaf = M - 1
    for i in (0, 3, 4, 7):
        v[i * M + leaf, 1, 20] = float("-inf")
    out = run_tree(c, lens, parents, q, k, v)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    same = torch.ones(n * M, 12, dtype=torch.bool)
    for i in (0, 3, 4, 7):
        same[i * M + leaf, 4:8] = False
    o, w = out.float().cpu(), clean.float().cpu()
    assert torch.isfinite(o[same]).all()
    tol = 2 * (torch.finfo(elem).eps / 2) * w[same].abs() + 2 * 2.0 ** -10 * 40
    assert ((o[same] - w[same]).abs() <= tol).all()
    assert torch.isinf(o[~same][:, 20]).all() and torch.isfinite(o[~same][:, :20]).all()


@pytest.mark.parametrize("elem", [F16, BF16])
def test_values_at_the_edges_of_the_types(elem):
    """Zero blocks beside huge ones, values of the largest size, tiny ones, huge
    queries: finite means, the zero blocks' weights count."""
    rng = np.random.default_rng(8)
    big = torch.finfo(elem).max
    M, n = 6, 90
    c = make(1, 2, 16, 4, 8, elem, E4M3, M, seed=7)
    for s in range(4):
        k, v = c.vec(rng, n, 1) * 0.1, c.vec(rng, n, 1)
        if s == 0:
            v[16:48] = 0
            v[:16] = big
        elif s == 1:
            v[:] = big
        elif s == 2:
            v *= torch.finfo(elem).tiny
        else:
            k[:] = 0
            v[:40] *= 1000
            v[40:] = 0
        c.append([s], [0], [n], k, v)
    q, k, v = drafts(c, rng, 4, M)
    k *= 0.1
    v[M:2 * M] = big
    v[2 * M:3 * M] *= torch.finfo(elem).tiny
    q[3 * M:] *= big / 1e5
    parents = [tref.random_tree(rng, M) for _ in range(4)]
    out = run_tree(c, [n] * 4, parents, q, k, v)
    assert torch.isfinite(out[:3 * M].float()).all()
    with np.errstate(over="ignore"):
        check_tree(c, out[:3 * M], [n] * 3, parents, q[:3 * M], k[:3 * M], v[:3 * M], [M] * 3)


def test_errors_latch():
    rng = np.random.default_rng(9)
    M = 5
    c = make(2, 2, 16, 3, 4, F16, E4M3, M, seed=8)
    fill(c, rng, [60, 20, 10])
    q, k, v = drafts(c, rng, 2, M)
    ok = [[-1, 0, 0, 1, 1]] * 2

    def code(lens, parents, n_nodes, slots):
        c.c.tensors[4].zero_()
        run_tree(c, lens, parents, q, k, v, n_nodes, slots)
        torch.cuda.synchronize()
        return c.c.status_words.tolist()

    ARG, FULL, CHECK = -1, -5, -7
    assert code([60, 20], ok, [5, 5], [0, 1]) == [0, 0]
    assert code([60, 20], ok, [5, 6], [0, 1]) == [ARG, 1]
    assert code([60, 20], ok, [5, 5], [3, 1]) == [ARG, 0]
    assert code([60, 20], ok, [5, 5], [0, -1]) == [ARG, 1]
    assert code([60, 65], ok, [5, 5], [0, 1]) == [FULL, 1]
    assert code([60, 20], [ok[0], [-1, 0, 2, 1, 1]], [5, 5], [0, 1]) == [ARG, 1]
    assert code([60, 20], [[-2, 0, 0, 1, 1], ok[0]], [5, 5], [0, 1]) == [ARG, 0]
    # behind the nodes a parent may be anything
    assert code([60, 20], [ok[0], [-1, 0, 0, 77, -9]], [5, 3], [0, 1]) == [0, 0]
    kept = c.table.clone()
    c.table[1, 0] = 10000
    assert code([60, 20], ok, [5, 5], [0, 1]) == [CHECK, 1]
    c.table.copy_(kept)
    # later calls do nothing until the words are zeroed
    out = torch.full((2 * M, 4, 128), 3.0, dtype=F16, device="cuda")
    run_tree(c, [60, 20], ok, q, k, v, out=out)
    torch.cuda.synchronize()
    assert (out == 3.0).all()
    c.c.tensors[4].zero_()


def test_captured_and_replayed_with_other_contents():
    rng = np.random.default_rng(10)
    M, n = 9, 3
    c = make(2, 4, 32, n, 40, BF16, E4M3, M, seed=9, fill=NAN)
    top = [1200, 700, 40]
    fill(c, rng, top)
    q, k, v = drafts(c, rng, n, M)
    lens, nodes = i32([32, 64, 40]), i32([1, 2, 9])
    parents = [tref.random_tree(rng, M) for _ in range(n)]
    par = i32(parents)
    out = torch.full_like(q, NAN)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _dkv().dkv_cache8_tree(c.c, lens, par, q, k, v, out, n_nodes=nodes)
    for ln, nn in (([32, 64, 40], [1, 2, 9]), (top, [9, 9, 9]), ([0, 690, 38], [4, 1, 0]), ([1200, 0, 0], [9, 0, 0])):
        lens.copy_(i32(ln))
        nodes.copy_(i32(nn))
        out.fill_(NAN)
        g.replay()
        check_tree(c, out, ln, parents, q, k, v, nn)


def test_two_streams_with_workspaces_of_their_own():
    rng = np.random.default_rng(11)
    M = 16
    cs = [make(4, 4, 64, 4, 40, F16, E4M3, M, seed=s) for s in (1, 2)]
    lens = [2300, 100, 900, 5]
    data = []
    for c in cs:
        fill(c, rng, lens)
        data.append(([tref.random_tree(rng, M) for _ in lens], *drafts(c, rng, 4, M)))
    want = [run_tree(c, lens, *d) for c, d in zip(cs, data)]
    outs = [torch.empty_like(w) for w in want]
    par, ln = [i32(d[0]) for d in data], i32(lens)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(10):
        for c, d, o, p, s in zip(cs, data, outs, par, streams):
            _dkv().dkv_cache8_tree(c.c, ln, p, *d[1:], o, stream=s)
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("elem,n,hkv,G,M,longest", [(F16, 300, 4, 3, 3, 60), (BF16, 300, 4, 3, 3, 60), (F16, 1024, 1, 1, 1, 40)])
def test_hundreds_of_short_requests(elem, n, hkv, G, M, longest):
    """Many units of a step or two for each SM, a few long ones among them; some without
    drafts."""
    rng = np.random.default_rng(n + M)
    lens = [int(x) for x in rng.integers(0, longest, n)]
    lens[5], lens[n // 2], lens[n - 1] = 700, 431, 1300
    c = make(hkv, G, 16, n, 1300 // 16 + 1, elem, E4M3, M, seed=3, fill=NAN)
    who = [i for i in range(n) if lens[i] > 0]
    new = [lens[i] for i in who]
    c.append(who, [0] * len(who), new, c.vec(rng, sum(new), hkv), c.vec(rng, sum(new), hkv))
    parents = [tref.random_tree(rng, M) for _ in range(n)]
    n_nodes = [int(x) for x in rng.integers(0, M + 1, n)]
    n_nodes[5] = n_nodes[n - 1] = M
    q, k, v = drafts(c, rng, n, M, n_nodes)
    out = run_tree(c, lens, parents, q, k, v, n_nodes)
    check_tree(c, out, lens, parents, q, k, v, n_nodes)
    again = run_tree(c, lens, parents, q, k, v, n_nodes)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("n", [20, 300])
def test_products_beyond_fp32_that_never_meet(n):
    """bf16 queries and keys of 2^110 in different features: every logit is 0, so the
    result is the mean of the values."""
    rng = np.random.default_rng(12)
    M = 7
    c = make(2, 2, 16, 1, 24, BF16, INT8, M, seed=10)
    k, v = torch.zeros((n, 2, 128), dtype=BF16, device="cuda"), c.vec(rng, n, 2)
    k[:, :, 3] = 2.0 ** 110
    c.append([0], [0], [n], k, v)
    q, _, dv = drafts(c, rng, 1, M)
    q[:] = 0
    q[:, :, 4] = 2.0 ** 110
    q[2] = 0                        # and a query of zeros
    dk = torch.zeros_like(dv)
    dk[:, :, 3] = 2.0 ** 110
    parents = [[-1, 0, 0, 1, 2, -1, 5]]
    out = run_tree(c, [n], parents, q, dk, dv)
    check_tree(c, out, [n], parents, q, dk, dv, [M])


@pytest.mark.parametrize("up", [-116, 116])
def test_huge_keys_and_tiny_queries_computed_again(up):
    """bf16 keys of 2^116 (2^-116) and queries that bring them back, with and without an
    infinite value that rows do not see."""
    rng = np.random.default_rng(13)
    n, M = 150, 6
    c = make(1, 4, 32, 1, 8, BF16, E4M3, M, seed=11)
    k, v = c.vec(rng, n, 1), c.vec(rng, n, 1)
    if up > 0:                      # (a block's smallest scale is 2^-100)
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
    out = run_tree(c, [n], parents, q, dk, dv)
    check_tree(c, out, [n], parents, q, dk, dv, [M])
    dv[5, :, 9] = float("inf")
    out = run_tree(c, [n], parents, q, dk, dv)
    check_tree(c, out, [n], parents, q, dk, dv, [M], nodes=range(5))
    assert torch.isinf(out[5, :, 9].float()).all() and torch.isfinite(out[5, :, :9].float()).all()


def test_two_graphs_of_one_workspace_in_turn():
    """Calls in the order of a stream may share a workspace: it holds nothing between
    them."""
    rng = np.random.default_rng(14)
    M, lens = 9, [900, 70, 0]
    cs, data = [], []
    for s, hkv in ((1, 4), (2, 2)):
        c = make(hkv, 4, 32, 3, 32, F16, INT8, M, seed=s)
        fill(c, rng, lens)
        cs.append(c)
        data.append(([tref.random_tree(rng, M) for _ in lens], *drafts(c, rng, 3, M)))
    cs[1].c = _dkv().make_cache8(cs[1].pages, cs[1].scales, cs[1].tail, cs[1].table, group_size=4, rotary_dim=0,
                                 max_nodes=M, tree_workspace=cs[0].c.tensors[6])
    want = [run_tree(c, lens, *d) for c, d in zip(cs, data)]
    outs, graphs = [torch.full_like(w, NAN) for w in want], []
    ln, par = i32(lens), [i32(d[0]) for d in data]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for c, d, o, p in zip(cs, data, outs, par):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            _dkv().dkv_cache8_tree(c.c, ln, p, *d[1:], o)
        graphs.append(g)
    for order in ((0, 1, 1, 0), (1, 0, 0, 1)):
        for o in outs:
            o.fill_(NAN)
        for x in order:
            graphs[x].replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))


# ------------------------------------------------------------------ accepted drafts

@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
def test_accept_leaves_the_state_of_an_append(elem, code, T):
    """Paths of none to all nodes, across block borders, onto open blocks and onto
    nothing; nodes in any order; other places stay (NaN here)."""
    rng = np.random.default_rng(T)
    before = [0, 1, T - 1, T, 2 * T - 3, T // 2, T + 5, 7]
    n, M, W = len(before), 40, 37
    c = make(2, 3, T, n, 8 if T < 64 else 4, elem, code, 0, seed=T, fill=NAN)
    slots = [int(x) for x in rng.permutation(n)]
    fill(c, rng, before, slots)
    k, v = c.vec(rng, n * M, 2), c.vec(rng, n * M, 2)
    path = [[int(x) for x in rng.integers(0, M, W)] for _ in range(n)]
    n_path = [37, 1, 1, 0, 3, 20, -4, 16]
    before2 = list(before)
    before2[7] = -1                  # padding, its slot may be any number
    slots2 = list(slots)
    slots2[7] = 1 << 30
    _dkv().dkv_cache8_accept(c.c, i32(before2), k, v, i32(path), n_path=i32(n_path), slots=i32(slots2))
    kn, vn = ref.elem_np(k), ref.elem_np(v)
    for i in range(n):
        if before2[i] >= 0 and n_path[i] > 0:
            rows = [i * M + x for x in path[i][:n_path[i]]]
            c.ref.append(slots[i], before[i], kn[rows], vn[rows])
    c.check()


def test_accept_whole_paths_without_counts():
    rng = np.random.default_rng(3)
    c = make(1, 1, 16, 2, 20, F16, INT8, 0, seed=3)
    k, v = c.vec(rng, 256, 1), c.vec(rng, 256, 1)
    path = [list(range(128)), list(range(127, -1, -1))]
    _dkv().dkv_cache8_accept(c.c, i32([0, 0]), k, v, i32(path))
    kn, vn = ref.elem_np(k), ref.elem_np(v)
    for i in range(2):
        rows = [i * 128 + x for x in path[i]]
        c.ref.append(i, 0, kn[rows], vn[rows])
    c.check()


def test_accept_errors_latch():
    rng = np.random.default_rng(4)
    c = make(2, 1, 16, 3, 2, F16, E4M3, 0, seed=4)
    k, v = c.vec(rng, 12, 2), c.vec(rng, 12, 2)

    def code(before, path, n_path, slots):
        c.c.tensors[4].zero_()
        _dkv().dkv_cache8_accept(c.c, i32(before), k, v, i32(path), n_path=i32(n_path), slots=i32(slots))
        torch.cuda.synchronize()
        return c.c.status_words.tolist()

    ARG, FULL, CHECK = -1, -5, -7
    p = [[0, 1, 2], [3, 4, 5]]
    assert code([0, 0], p, [3, 3], [0, 2]) == [0, 0]
    assert code([0, 0], p, [3, 4], [0, 2]) == [ARG, 1]
    assert code([0, 30], p, [3, 3], [0, 2]) == [FULL, 1]
    assert code([0, 0], p, [3, 3], [1, 1])[0] == ARG
    assert code([0, 0], p, [3, 3], [3, 1]) == [ARG, 0]
    assert code([0, 0], [[0, 6, 2], [0, 0, 0]], [3, 3], [0, 1]) == [ARG, 0]
    assert code([0, 0], [[0, 1, -1], [0, 0, 0]], [3, 3], [0, 1]) == [ARG, 0]
    assert code([0, 0], [[0, 1, -1], [0, 0, 99]], [2, 2], [0, 1]) == [0, 0]
    c.table[0, 0] = -1
    assert code([15, 0], p, [1, 1], [0, 1]) == [CHECK, 0]


# ------------------------------------------------------------------ positions of several axes

AXES = [(1, None), (1, "0"), (2, "halves"), (3, "parts"), (3, "mixed"), (4, "mixed")]


def axis_list(kind, axes, pairs):
    if kind is None:
        return None
    if kind == "0":
        return [0] * pairs
    if kind == "mixed":
        return [i % axes for i in range(pairs)]
    cut = sorted({pairs // 5, pairs // 2} if axes == 3 else {pairs // 2})
    return [sum(i >= x for x in cut) for i in range(pairs)]


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("axes,kind", AXES)
@pytest.mark.parametrize("rot,inter", [(16, False), (48, True), (128, False), (128, True), (96, False)])
def test_rotate(elem, axes, kind, rot, inter):
    """Bit for bit; padding rows stay; keys or queries alone; in place; strided."""
    rng = np.random.default_rng(rot + axes)
    c = make(3, 3, 16, 1, 40, elem, E4M3, 0, rot=rot, inter=inter)
    n, L = 37, 640
    pos = rng.integers(0, L, (axes, n))
    pos[:, 0], pos[:, 1] = 0, L - 1
    ax = axis_list(kind, axes, rot // 2)
    x = c.vec(rng, n, 15)
    q, k = x[:, :9], x[:, 9:12]
    want = [tref.rotate_at(ref.elem_np(y), pos, ax or [0] * (rot // 2), c.rope_np, rot, inter, elem) for y in (q, k)]
    dev = pos.copy()
    dev[0, [5, 20]] = [-1, -2 ** 31]      # padding
    dev[1:, 5] = 10 ** 9
    qr, kr = torch.full((n, 9, 128), 7.0, dtype=elem, device="cuda"), torch.full((n, 3, 128), 7.0, dtype=elem, device="cuda")
    _dkv().dkv_cache8_rotate(c.c, i32(dev), c.rope, q=q, k=k, q_rot=qr, k_rot=kr, pair_axis=ax)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    for got, w in ((qr, want[0]), (kr, want[1])):
        w = w.copy()
        w[[5, 20]] = 7.0
        assert np.array_equal(ref.elem_np(got), w)
    q2, k2 = q.contiguous(), k.contiguous()
    _dkv().dkv_cache8_rotate(c.c, i32(pos), c.rope, q=q2, q_rot=q2, pair_axis=ax)
    _dkv().dkv_cache8_rotate(c.c, i32(pos), c.rope, k=k2, k_rot=k2, pair_axis=ax)
    torch.cuda.synchronize()
    assert np.array_equal(ref.elem_np(q2), want[0]) and np.array_equal(ref.elem_np(k2), want[1])


def test_rotate_one_axis_is_the_appends_rotation():
    rng = np.random.default_rng(2)
    c = make(2, 4, 16, 1, 10, F16, E4M3, 0, rot=64)
    k, v, q = c.vec(rng, 100, 2), c.vec(rng, 100, 2), c.vec(rng, 100, 8)
    kr, qr, kr2, qr2 = torch.empty_like(k), torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    c.append(None, [0], [100], k, v, q, kr, qr)
    _dkv().dkv_cache8_rotate(c.c, torch.arange(100, dtype=torch.int32, device="cuda"), c.rope, q=q, k=k, q_rot=qr2, k_rot=kr2)
    torch.cuda.synchronize()
    assert torch.equal(kr, kr2) and torch.equal(qr, qr2)


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (BF16, INT8)])
@pytest.mark.parametrize("axes,kind", AXES)
@pytest.mark.parametrize("T", [16, 64, 128])
def test_append_at(elem, code, axes, kind, T):
    """State, turned keys and queries bit for bit: pieces across blocks, then single
    tokens (the step's kernel), whose positions are not their places."""
    rng = np.random.default_rng(T + axes)
    rot, inter = (128, False) if axes != 3 else (96, True)
    c = make(2, 3, T, 3, 4, elem, code, 0, rot=rot, inter=inter, fill=NAN, seed=T)
    ax = axis_list(kind, axes, rot // 2)
    L = c.rope.shape[0]
    at = [0, 0, 0]
    slots = [2, 0, 1]
    for new, step in (([T + 3, 5, 2 * T], False), ([1, 1, 1], True), ([T - 4, T // 2, 1], False), ([1, 1, 1], True)):
        n = sum(new)
        pos = rng.integers(0, L, (axes, n))
        k, v, q = c.vec(rng, n, 2), c.vec(rng, n, 2), c.vec(rng, n, 6)
        kr, qr = torch.full_like(k, 7.0), torch.full_like(q, 7.0)
        _dkv().dkv_cache8_append_at(c.c, i32(at), i32(pos), k, v, c.rope, pair_axis=ax, n_new=None if step else new,
                                    slots=i32(slots), q=q, k_rot=kr, q_rot=qr)
        turned = [tref.rotate_at(ref.elem_np(y), pos, ax or [0] * (rot // 2), c.rope_np, rot, inter, elem) for y in (k, q)]
        kept, c.ref.rot = c.ref.rot, 0       # the reference stores what is turned already
        row = 0
        for i, m in enumerate(new):
            c.ref.append(slots[i], at[i], turned[0][row:row + m], ref.elem_np(v)[row:row + m])
            row += m
            at[i] += m
        c.ref.rot = kept
        c.check()
        assert np.array_equal(ref.elem_np(kr), turned[0]) and np.array_equal(ref.elem_np(qr), turned[1])


def test_append_at_padding_and_positions_beyond_the_table():
    rng = np.random.default_rng(5)
    c = make(2, 2, 16, 3, 4, F16, E4M3, 0, rot=32)
    k, v = c.vec(rng, 4, 2), c.vec(rng, 4, 2)
    before, pos = i32([0, -1, 3]), torch.tensor([[5, 5, 10 ** 6, 9]], dtype=torch.int32, device="cuda")
    _dkv().dkv_cache8_append_at(c.c, before, pos, k, v, c.rope, n_new=[1, 2, 1])
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    for n_new in ([1, 2, 1], None):
        for bad in (-1, c.rope.shape[0], 2 ** 31 - 1):
            c.c.tensors[4].zero_()
            pos[0, 3 if n_new else 2] = bad
            _dkv().dkv_cache8_append_at(c.c, before, pos if n_new else pos[:, :3].contiguous(), k if n_new else k[:3],
                                        v if n_new else v[:3], c.rope, n_new=n_new)
            torch.cuda.synchronize()
            assert c.c.status_words.tolist() == [-1, 2]
    c.c.tensors[4].zero_()
    qr = torch.empty((2, 4, 128), dtype=F16, device="cuda")
    _dkv().dkv_cache8_rotate(c.c, i32([[1, 70]]), c.rope, q=c.vec(rng, 2, 4), q_rot=qr)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [-1, 1]


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("elem,code", [(F16, E4M3), (BF16, INT8)])
def test_rounds_of_guesses(elem, code):
    """Prompts with images appended at positions of three axes, then rounds of:
    guesses turned at their depths, tree attention, the accepted path appended, in
    one captured step whose contents change; at the end decode attention over what
    is stored."""
    rng = np.random.default_rng(12)
    hkv, G, T, n, M, W, rot = 2, 4, 32, 3, 10, 6, 128
    c = make(hkv, G, T, n, 12, elem, code, M, rot=rot, seed=3, fill=NAN)
    ax = axis_list("parts", 3, rot // 2)
    L = c.rope.shape[0]
    new = [50, 31, 7]
    pos = rng.integers(0, 60, (3, sum(new)))
    k, v = c.vec(rng, sum(new), hkv), c.vec(rng, sum(new), hkv)
    _dkv().dkv_cache8_append_at(c.c, i32([0, 0, 0]), i32(pos), k, v, c.rope, pair_axis=ax, n_new=new)
    turned = tref.rotate_at(ref.elem_np(k), pos, ax, c.rope_np, rot, False, elem)
    c.ref.rot = 0
    row = 0
    for i, m in enumerate(new):
        c.ref.append(i, 0, turned[row:row + m], ref.elem_np(v)[row:row + m])
        row += m
    lens_h = list(new)
    q, k, v = (torch.empty((n * M, h, 128), dtype=elem, device="cuda") for h in (hkv * G, hkv, hkv))
    qr, kr, out = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    lens, nodes, par, p3 = i32([0] * n), i32([M] * n), i32([[-1] * M] * n), i32([[0] * (n * M)] * 3)
    path, n_path = i32([[0] * W] * n), i32([0] * n)

    def step():
        _dkv().dkv_cache8_rotate(c.c, p3, c.rope, q=q, k=k, q_rot=qr, k_rot=kr, pair_axis=ax)
        _dkv().dkv_cache8_tree(c.c, lens, par, qr, kr, v, out, n_nodes=nodes, window=40, sinks=4)
        _dkv().dkv_cache8_accept(c.c, lens, kr, v, path, n_path=n_path)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for r in range(6):
        trees = [tref.random_tree(rng, M, 4) for _ in range(n)]
        counts = [int(x) for x in rng.integers(1, M + 1, n)]
        position = np.array([[60 + lens_h[i] + d for d in tref.depths(trees[i])] for i in range(n)]).reshape(-1)
        paths = []
        for i in range(n):
            x, one = int(rng.integers(0, counts[i])), []
            while x >= 0:
                one.insert(0, x)
                x = trees[i][x]
            paths.append(one[:W])
        for t, x in ((q, c.vec(rng, n * M, hkv * G)), (k, c.vec(rng, n * M, hkv)), (v, c.vec(rng, n * M, hkv)),
                     (lens, i32(lens_h)), (nodes, i32(counts)), (par, i32(trees)), (p3, i32(np.stack([position] * 3))),
                     (path, i32([p + [0] * (W - len(p)) for p in paths])), (n_path, i32([len(p) for p in paths]))):
            t.copy_(x)
        out.fill_(NAN)
        if r % 2:
            step()
        else:
            graph.replay()
        torch.cuda.synchronize()
        want = tref.rotate_at(ref.elem_np(k), np.stack([position] * 3), ax, c.rope_np, rot, False, elem)
        assert np.array_equal(ref.elem_np(kr), want)
        check_tree(c, out, lens_h, trees, qr, kr, v, counts, window=40, sinks=4)
        vn = ref.elem_np(v)
        for i in range(n):
            rows = [i * M + x for x in paths[i]]
            c.ref.append(i, lens_h[i], want[rows], vn[rows])
            lens_h[i] += len(rows)
        c.check()
    q1 = c.vec(rng, n, hkv * G)
    c.check_attention(c.attend(None, lens_h, q1), range(n), lens_h, q1)


def test_offsets_beyond_32_bits():
    """Pages, slots and rows behind the first 4 GB give what near ones give, in all four
    calls."""
    dkv = _dkv()
    hkv, G, T, lens, M, R = 2, 4, 64, [200, 64, 130], 7, 32
    rng = np.random.default_rng(19)
    near = make(hkv, G, T, 3, 4, F16, E4M3, M, rot=R)
    n_pages, n_slots = 2 ** 33 // (hkv * T * 256) + 1, 2 ** 33 // (hkv * T * 512) + 1
    pages = torch.empty((n_pages, hkv, T // 16, 2, 2048), dtype=E4M3, device="cuda")
    tail = torch.empty((n_slots, hkv, T // 16, 2, 2048), dtype=F16, device="cuda")
    scales = torch.empty((n_pages, hkv, 2), device="cuda")
    table = torch.zeros((n_slots, 4), dtype=torch.int32, device="cuda")
    slots = torch.tensor([n_slots - 1, n_slots // 2 + 1, n_slots - 7], dtype=torch.int32, device="cuda")
    table[slots.long()] = torch.arange(n_pages - 12, n_pages, dtype=torch.int32, device="cuda").reshape(3, 4)
    far = dkv.make_cache8(pages, scales, tail, table, group_size=G, rotary_dim=R, max_nodes=M)
    total, rows = sum(lens), 3 * M

    def apart(n, tensors):
        wide = 2 ** 32 // n // 8 * 8 + 8                # rows lie over 8 GB
        space, out = torch.empty((n, wide), dtype=F16, device="cuda"), []
        for i, x in enumerate(tensors):
            y = space[:, 2048 * i:2048 * i + x.shape[1] * 128].view(n, x.shape[1], 128)
            y.copy_(x)
            out.append(y)
        return out

    k, v = near.vec(rng, total, hkv), near.vec(rng, total, hkv)
    qd, kd, vd = near.vec(rng, rows, hkv * G), near.vec(rng, rows, hkv), near.vec(rng, rows, hkv)
    pos = torch.from_numpy(rng.integers(0, 4 * T, (2, total)).astype(np.int32)).cuda()
    dpos = torch.from_numpy(rng.integers(0, 4 * T, (2, rows)).astype(np.int32)).cuda()
    axes = bytes(i % 2 for i in range(R // 2))
    zero, ln, par = i32([0] * 3), i32(lens), i32([tref.random_tree(rng, M) for _ in lens])
    path = i32([[0, 1, 3], [2, 5, 0], [4, 6, 6]])
    kept, got = [apart(total, (k, v)), apart(rows, (qd, kd, vd))], []
    for c, sl, (a, b), (x, y, z) in ((near.c, None, (k, v), (qd, kd, vd)), (far, slots, *kept)):
        dkv.dkv_cache8_append_at(c, zero, pos, a, b, near.rope, pair_axis=axes, n_new=lens, slots=sl)
        qr, kr = torch.empty_like(qd), torch.empty_like(kd)
        dkv.dkv_cache8_rotate(c, dpos, near.rope, q=x, k=y, q_rot=qr, k_rot=kr, pair_axis=axes)
        outs = [torch.empty_like(qd) for _ in range(2)]
        dkv.dkv_cache8_tree(c, ln, par, x, y, z, outs[0], slots=sl)
        dkv.dkv_cache8_accept(c, ln, y, z, path, slots=sl)
        dkv.dkv_cache8_tree(c, ln + 3, par, qr, kr, z, outs[1], window=150, sinks=3, slots=sl)
        torch.cuda.synchronize()
        assert c.status_words.tolist() == [0, 0]
        got.append((qr, kr, *outs))
    for x, y in zip(*got):
        assert torch.isfinite(x.float()).all() and torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert torch.equal(near.pages.view(torch.uint8)[near.table.long()][0, :3], pages.view(torch.uint8)[table[slots.long()].long()][0, :3])


def test_a_slot_of_two_requests():
    """Reading calls may name a slot twice, with other lengths."""
    rng = np.random.default_rng(20)
    M = 5
    c = make(2, 2, 32, 2, 8, BF16, INT8, M, seed=14, fill=NAN)
    fill(c, rng, [192, 50])
    lens, slots = [192, 64, 50, 192], [0, 0, 1, 0]
    parents = [tref.random_tree(rng, M) for _ in lens]
    q, k, v = drafts(c, rng, 4, M)
    out = run_tree(c, lens, parents, q, k, v, slots=slots)
    check_tree(c, out, lens, parents, q, k, v, [M] * 4, slots)


def test_nothing_but_padding_then_something():
    """A call without any draft writes nothing; the next one finds the workspace as it needs it."""
    rng = np.random.default_rng(21)
    M = 4
    c = make(2, 4, 16, 3, 5, F16, E4M3, M, seed=15, fill=NAN)
    fill(c, rng, [70, 0, 16])
    parents = [tref.random_tree(rng, M) for _ in range(3)]
    q, k, v = drafts(c, rng, 3, M, [0, 1, 0])
    out = run_tree(c, [70, 0, 16], parents, q, k, v, [0, 0, -3], slots=[0, 7, -1])
    torch.cuda.synchronize()
    assert torch.isnan(out).all() and c.c.status_words.tolist() == [0, 0]
    out = run_tree(c, [70, 0, 16], parents, q, k, v, [0, 1, 0])
    check_tree(c, out, [70, 0, 16], parents, q, k, v, [0, 1, 0])
    # a node alone sees itself: its value
    assert torch.equal(out[M].view(2, 4, 128), v[M][:, None].expand(2, 4, 128))


def test_requests_that_accept_nothing_need_no_slot():
    """n_path of 0 or less: the slot may be any number, one of another request among them, as
    a request without drafts may have in tree attention."""
    rng = np.random.default_rng(22)
    c = make(2, 2, 16, 3, 4, F16, E4M3, 4, seed=16, fill=NAN)
    fill(c, rng, [20, 15, 9])
    n, M = 6, 4
    k, v = c.vec(rng, n * M, 2), c.vec(rng, n * M, 2)
    before, slots, n_path = [20, 7, 15, 20, 3, 9], [0, -1, 1, 0, 1 << 30, 2], [2, 0, 3, 0, -4, 1]
    path = [[1, 3, 0], [99, 0, 0], [0, 1, 2], [0, 0, 0], [0, 0, 0], [3, 0, 0]]
    _dkv().dkv_cache8_accept(c.c, i32(before), k, v, i32(path), n_path=i32(n_path), slots=i32(slots))
    kn, vn = ref.elem_np(k), ref.elem_np(v)
    for i in range(n):
        if n_path[i] > 0:
            rows = [i * M + x for x in path[i][:n_path[i]]]
            c.ref.append(slots[i], before[i], kn[rows], vn[rows])
    c.check()
    # a whole round with such requests, then one where two that accept share a slot
    q, kd, vd = drafts(c, rng, n, M, [4, 0, 4, 0, 0, 4])
    out = run_tree(c, before, None, q, kd, vd, [4, 0, 4, 0, -1, 4], slots)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0] and torch.isnan(out[M:2 * M].float()).all()
    _dkv().dkv_cache8_accept(c.c, i32(before), k, v, i32(path), n_path=i32([2, 0, 1, 1, 0, 1]), slots=i32(slots))
    torch.cuda.synchronize()
    assert c.c.status_words[0] == -1
    c.c.tensors[4].zero_()


def test_a_workspace_for_fewer_drafts_says_what_it_needs():
    rng = np.random.default_rng(23)
    c = make(2, 4, 16, 2, 4, F16, E4M3, 8, seed=17)
    q, k, v = drafts(c, rng, 2, 20)
    with pytest.raises(_dkv().DkvError, match="max_nodes=20") as e:
        run_tree(c, [0, 0], None, q, k, v)
    assert e.value.code == _dkv().DKV_ERR_SCRATCH
    run_tree(c, [0, 0], None, q[:16], k[:16], v[:16])
