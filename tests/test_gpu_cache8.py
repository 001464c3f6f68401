"""GPU tests of the uniform 8-bit cache (append with rotation, decode attention,
prompt attention) against the plain reference of tests/cache8_ref.py: stored
state bit for bit, attention against 64 bits within the bound derived in
cache8_ref.tolerance."""
from __future__ import annotations

import numpy as np
import pytest

from tests import cache8_ref as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

E4M3, INT8, F16, BF16 = torch.float8_e4m3fn, torch.int8, torch.float16, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    _dkv().build.build()
    _dkv().load()


def _dkv():
    import differentiated_kv_cache_gb300 as dkv
    return dkv


class Cache:
    """Tensors of a layer's cache, the descriptor and the reference beside them."""

    def __init__(self, hkv, G, T, slots, width, elem, code, rot=0, inter=False, seed=0, fill=None, spare=3):
        rng = np.random.default_rng(seed)
        n = slots * width + spare
        self.hkv, self.G, self.T, self.elem, self.slots = hkv, G, T, elem, slots
        self.pages = torch.zeros((n, hkv, T // 16, 2, 2048), dtype=torch.uint8, device="cuda").view(code)
        self.scales = torch.zeros((n, hkv, 2), device="cuda")
        self.tail = torch.zeros((slots, hkv, T // 16, 2, 2048), dtype=elem, device="cuda")
        if fill is not None:
            self.tail.fill_(fill)
        self.table = torch.from_numpy(rng.permutation(n)[:slots * width].astype(np.int32).reshape(slots, width)).cuda()
        self.rot, self.inter = rot, inter
        self.c = _dkv().make_cache8(self.pages, self.scales, self.tail, self.table, group_size=G, rotary_dim=rot,
                                    rotary_interleaved=inter)
        self.ref = ref.RefCache(self.pages, self.scales, self.tail, self.table, rot, inter)
        ang = np.arange(width * T)[:, None] * 10000.0 ** (-np.arange(0, rot, 2) / max(rot, 1))
        self.rope_np = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32) if rot else None
        self.rope = torch.from_numpy(self.rope_np).cuda() if rot else None

    def vec(self, rng, n, heads, scale=1.0):
        x = rng.standard_normal((n, heads, 128)).astype(np.float32) * scale
        x[:, :, rng.integers(0, 128, 3)] *= 8
        return torch.from_numpy(x).to(self.elem).cuda()

    def append(self, slots, before, new, k, v, q=None, k_rot=None, q_rot=None, step=False, **kw):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        rc = _dkv().dkv_cache8_append(self.c, i32(before), k, v, rope=self.rope, n_new=None if step else new,
                                      slots=None if slots is None else i32(slots), q=q, k_rot=k_rot, q_rot=q_rot, **kw)
        at, turned = 0, []
        kn, vn = ref.elem_np(k), ref.elem_np(v)
        for s, b, n in zip(slots if slots is not None else range(len(before)), before, new):
            if b >= 0:
                turned.append(self.ref.append(s, b, kn[at:at + n], vn[at:at + n], self.rope_np))
            else:
                turned.append(None)
            at += n
        return rc, turned

    def check(self):
        torch.cuda.synchronize()
        assert self.c.status_words.tolist() == [0, 0]
        self.ref.check(self.pages, self.scales, self.tail)

    def attend(self, slots, lens, q, window=0, sinks=0, out=None, **kw):
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        out = torch.full_like(q, float("nan"), memory_format=torch.contiguous_format) if out is None else out
        _dkv().dkv_cache8_attention(self.c, i32(lens), q, out, window=window, sinks=sinks,
                                    slots=None if slots is None else i32(slots), **kw)
        return out

    def check_attention(self, out, slots, lens, q, window=0, sinks=0):
        got, qn = out.double().cpu().numpy(), q.double().cpu().numpy()
        for i, (s, n) in enumerate(zip(slots, lens)):
            see = ref.visible(max(n, 0), window, sinks)
            for h in range(self.hkv):
                k, v = self.ref.values(s, max(n, 0), h)
                g = slice(h * self.G, (h + 1) * self.G)
                want, pv, qk, vm = ref.attend(qn[i, g], k[see], v[see])
                tol = ref.tolerance(want, pv, qk, vm, len(see), self.elem, 2.0 ** -11)
                err = np.abs(got[i, g] - want)
                assert (err <= tol).all(), (i, h, n, float((err / tol).max()))


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
@pytest.mark.parametrize("T", [16, 32, 64, 128])
def test_append_in_pieces_gives_the_same_state(elem, code, T):
    """One token, odd pieces across block borders and whole blocks, two requests
    in crossed slots; the other places of the tails (NaN here) stay."""
    rng = np.random.default_rng(T)
    c = Cache(2, 3, T, 4, 5, elem, code, rot=64, inter=T % 64 == 0, fill=float("nan"), seed=T)
    at = {3: 0, 1: 0}
    for a, b in [(1, T - 1), (T // 2 + 1, 1), (1, 2), (2 * T, T), (3, T + 5), (T // 2, 1)]:
        n = a + b
        k, v, q = c.vec(rng, n, 2), c.vec(rng, n, 2), c.vec(rng, n, 6)
        kr, qr = torch.full_like(k, 7.0), torch.full_like(q, 7.0)
        rc, turned = c.append([3, 1], [at[3], at[1]], [a, b], k, v, q, kr, qr)
        assert rc == 0
        assert np.array_equal(ref.elem_np(kr), np.concatenate(turned))
        pos = np.concatenate([np.arange(at[3], at[3] + a), np.arange(at[1], at[1] + b)])
        assert np.array_equal(ref.elem_np(qr), ref.rotate(ref.elem_np(q), pos, c.rope_np, 64, c.inter, elem))
        at[3] += a
        at[1] += b
        c.check()


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (BF16, INT8)])
def test_steps_equal_one_call(elem, code):
    """130 calls of one token and one call of 130 tokens leave the same bits."""
    rng = np.random.default_rng(5)
    a, b = (Cache(3, 2, 32, 2, 6, elem, code, rot=128, seed=9) for _ in range(2))
    k, v = a.vec(rng, 260, 3), a.vec(rng, 260, 3)
    b.append(None, [0, 0], [130, 130], k, v)
    for p in range(130):
        rows = torch.tensor([p, 130 + p], device="cuda")
        a.append(None, [p, p], [1, 1], k[rows], v[rows], step=True)
    a.check()
    b.check()
    # what stays in a tail after its block is complete depends on the calls;
    # the pages, scales and open blocks do not
    assert torch.equal(a.pages.view(torch.uint8), b.pages.view(torch.uint8)) and torch.equal(a.scales, b.scales)
    open_k = [ref.from_tiles(ref.elem_np(x.tail)[1, 2], 16)[:, :130 % 32] for x in (a, b)]
    assert np.array_equal(*open_k)


@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (16, True), (48, False), (96, True), (128, False), (128, True)])
@pytest.mark.parametrize("G", [1, 7])
def test_rotations(rot, inter, G):
    rng = np.random.default_rng(rot)
    for elem in (F16, BF16):
        c = Cache(2, G, 16, 3, 20, elem, E4M3, rot=rot, inter=inter)
        n = [70, 1, 33]
        k, v, q = c.vec(rng, sum(n), 2), c.vec(rng, sum(n), 2), c.vec(rng, sum(n), 2 * G)
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        _, turned = c.append([2, 0, 1], [0, 0, 0], n, k, v, q, kr, qr)
        c.check()
        pos = np.concatenate([np.arange(x) for x in n])
        assert np.array_equal(ref.elem_np(qr), ref.rotate(ref.elem_np(q), pos, c.rope_np, rot, inter, elem))
        assert np.array_equal(ref.elem_np(kr), np.concatenate(turned))


def test_parts_of_one_projection_and_in_place():
    """q, k, v as parts of one [tokens][q | k | v] projection; contiguous q and k
    turned in place."""
    rng = np.random.default_rng(3)
    c = Cache(2, 4, 32, 2, 4, BF16, E4M3, rot=128)
    qkv = c.vec(rng, 50, 12)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    qr = torch.empty((50, 8, 128), dtype=BF16, device="cuda")
    c.append(None, [0, 0], [20, 30], k, v, q, None, qr)
    c.check()
    d = Cache(2, 4, 32, 2, 4, BF16, E4M3, rot=128)
    q2, k2 = q.contiguous(), k.contiguous()
    kn = ref.elem_np(k2)
    before = torch.zeros(2, dtype=torch.int32, device="cuda")
    _dkv().dkv_cache8_append(d.c, before, k2, v, rope=d.rope, n_new=[20, 30], q=q2, k_rot=k2, q_rot=q2)
    torch.cuda.synchronize()
    assert torch.equal(q2, qr)
    assert torch.equal(c.pages.view(torch.uint8), d.pages.view(torch.uint8)) and torch.equal(c.tail, d.tail)
    pos = np.concatenate([np.arange(20), np.arange(30)])
    assert np.array_equal(ref.elem_np(k2), ref.rotate(kn, pos, d.rope_np, 128, False, BF16))


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
def test_special_values(elem, code):
    """Zero blocks, tiny and huge values, infinities and NaN: codes as the header
    says, other tokens of the block undisturbed."""
    c = Cache(1, 1, 16, 1, 8, elem, code)
    big = torch.finfo(elem).max
    x = torch.randn((8 * 16, 1, 128), generator=torch.Generator().manual_seed(1)).to(elem)
    x[16:32] = 0
    x[32:48] *= torch.finfo(elem).tiny
    x[48:64] *= big / 8
    x[70, 0, 3], x[71, 0, 4], x[72, 0, 5] = float("inf"), float("-inf"), float("nan")
    x[80:96] = float("nan")
    x[100] = -0.0
    x[112:] = float("inf")
    y = x.flip(0).contiguous()
    c.append(None, [0], [128], x.cuda(), y.cuda())
    c.check()


def test_padding_rows_are_skipped():
    rng = np.random.default_rng(8)
    c = Cache(2, 2, 16, 5, 4, F16, E4M3, rot=32, fill=3.0)
    n = [4, 1, 20]
    k, v, q = c.vec(rng, 25, 2), c.vec(rng, 25, 2), c.vec(rng, 25, 4)
    qr = torch.full_like(q, 9.0)
    c.append([4, 4, 0], [0, -1, 0], n, k, v, q, None, qr)
    c.check()
    assert (qr[4] == 9).all() and not (qr[5:] == 9).all()
    c.append([4, 4, 0], [4, -1, 20], [1, 1, 1], k[:3], v[:3], step=True)
    c.check()


# ------------------------------------------------------------------ attention

LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 383, 500]


def filled(hkv, G, T, elem, code, lens, seed=0, scale=1.0, fill=float("nan")):
    rng = np.random.default_rng(seed)
    c = Cache(hkv, G, T, len(lens), max(1, -(-max(lens) // T)), elem, code, seed=seed, fill=fill)
    slots = [int(x) for x in rng.permutation(len(lens))]
    some = [i for i, n in enumerate(lens) if n > 0]
    new = [lens[i] for i in some]
    k, v = c.vec(rng, sum(new), hkv, scale), c.vec(rng, sum(new), hkv)
    c.append([slots[i] for i in some], [0] * len(some), new, k, v)
    return c, slots, c.vec(rng, len(lens), hkv * G)


@pytest.mark.parametrize("T,G,elem,code", [(16, 4, F16, E4M3), (32, 1, F16, INT8), (64, 8, BF16, E4M3), (128, 5, BF16, INT8),
                                           (64, 4, F16, E4M3), (128, 7, F16, INT8), (16, 2, BF16, INT8), (32, 3, BF16, E4M3)])
def test_attention_lengths(T, G, elem, code):
    """Every length at block and tile borders, from empty; unwritten tail places
    hold NaN."""
    c, slots, q = filled(2, G, T, elem, code, LENS, seed=G)
    out = c.attend(slots, LENS, q)
    c.check()
    c.check_attention(out, slots, LENS, q)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 3), (16, 0), (17, 4), (64, 64), (100, 16), (100, 33), (250, 200),
                                          (499, 1), (500, 7), (10000, 4), (0, 9)])
def test_attention_window_and_first_tokens(window, sinks):
    for T, G, elem, code in ((32, 4, F16, E4M3), (128, 6, BF16, INT8)):
        c, slots, q = filled(2, G, T, elem, code, LENS, seed=window)
        out = c.attend(slots, LENS, q, window, sinks)
        torch.cuda.synchronize()
        assert c.c.status_words.tolist() == [0, 0]
        c.check_attention(out, slots, LENS, q, window, sinks)


def test_attention_ignores_what_is_not_visible():
    """Tokens outside the window and the first ones hold infinities and NaN, in
    blocks that a visible token shares too: the result does not change."""
    T, lens, window, sinks = 32, [150, 149, 97, 40], 21, 3
    rng = np.random.default_rng(4)
    for elem, code in ((F16, E4M3), (BF16, E4M3), (BF16, INT8)):
        outs = []
        base = Cache(1, 4, T, 4, 5, elem, code)
        k, v, q = base.vec(rng, sum(lens), 1), base.vec(rng, sum(lens), 1), base.vec(rng, 4, 4)
        for bad in (False, True):
            c = Cache(1, 4, T, 4, 5, elem, code)
            kk, vv = k.clone(), v.clone()
            at = 0
            for n in lens:
                hidden = [j for j in range(n) if j not in set(ref.visible(n, window, sinks))]
                if bad:
                    kk[at + np.array(hidden[::2])], vv[at + np.array(hidden[::2])] = float("nan"), float("inf")
                    kk[at + np.array(hidden[1::2])], vv[at + np.array(hidden[1::2])] = float("-inf"), float("nan")
                else:
                    kk[at + np.array(hidden)] = vv[at + np.array(hidden)] = 0.0
                at += n
            c.append(None, [0] * 4, lens, kk, vv)
            outs.append(c.attend(None, lens, q, window, sinks))
            c.check_attention(outs[-1], range(4), lens, q, window, sinks)
        assert torch.equal(*outs)


@pytest.mark.parametrize("scale", [1e-3, 30.0])
def test_attention_of_flat_and_sharp_rows(scale):
    """Near-uniform weights and rows that one token takes alone, with V blocks of
    very different scales and V rows of zeros."""
    for elem, code in ((F16, E4M3), (BF16, INT8)):
        rng = np.random.default_rng(6)
        lens = [700, 64, 333]
        c = Cache(2, 4, 64, 3, 11, elem, code)
        k, v, q = c.vec(rng, sum(lens), 2, scale), c.vec(rng, sum(lens), 2), c.vec(rng, 3, 8)
        f = torch.ones(sum(lens), 1, 1, device="cuda")
        f[64:128], f[128:192], f[200:300], f[300:310] = 1e-4, 0.0, 100.0, 1e-6
        v = (v.float() * f).to(elem)
        c.append(None, [0, 0, 0], lens, k, v)
        out = c.attend(None, lens, q)
        c.check_attention(out, range(3), lens, q)


@pytest.mark.parametrize("amp", [1e-30, 1e-12, 1e12])
def test_attention_bf16_amplitudes(amp):
    """Values far from 1 in every block and in the tail (bf16's range)."""
    rng = np.random.default_rng(2)
    lens = [100, 40, 7]
    c = Cache(1, 3, 32, 3, 4, BF16, E4M3)
    k = c.vec(rng, sum(lens), 1)
    v = (c.vec(rng, sum(lens), 1).float() * amp).to(BF16)
    q = (c.vec(rng, 3, 3).float() * 1e-3).to(BF16)
    k = (k.float() * 1e3).to(BF16)
    c.append(None, [0] * 3, lens, k, v)
    out = c.attend(None, lens, q)
    c.check_attention(out, range(3), lens, q)


def test_attention_strided_queries_same_slot_twice_and_longer_batch():
    """Rows of a projection as q; a slot given twice with other lengths; rows of
    out behind the batch untouched."""
    c, slots, _ = filled(2, 4, 32, F16, E4M3, [300, 90, 10], seed=1)
    rng = np.random.default_rng(1)
    wide = c.vec(rng, 4, 12)
    q = wide[:, :8]
    who, lens = [slots[0], slots[1], slots[0], slots[2]], [300, 77, 256, 10]
    # 256 tokens of the first slot end at a block border; 77 of 90: the tail
    # holds tokens 64..89
    out = torch.full((6, 8, 128), 5.0, dtype=F16, device="cuda")
    c.attend(who, lens, q, out=out[:4])
    c.check_attention(out[:4], who, lens, q)
    assert (out[4:] == 5).all()


def test_long_context_and_many_requests():
    lens = [5000] + [int(x) for x in np.random.default_rng(0).integers(1, 90, 60)]
    c, slots, q = filled(1, 4, 64, F16, INT8, lens, seed=3)
    for window, sinks in ((0, 0), (1000, 5)):
        out = c.attend(slots, lens, q, window, sinks)
        c.check_attention(out, slots, lens, q, window, sinks)


def test_calls_repeat_bit_for_bit():
    lens = [1500, 20, 700, 1, 333]
    c, slots, q = filled(4, 7, 32, BF16, E4M3, lens, seed=3)
    first = c.attend(slots, lens, q)
    for _ in range(20):
        assert torch.equal(first, c.attend(slots, lens, q))


# ------------------------------------------------------------------ errors

def test_device_errors_latch_and_stop_later_calls():
    dkv = _dkv()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(1)

    def fresh():
        c = Cache(2, 2, 16, 3, 3, F16, E4M3, rot=32)
        k, v = c.vec(rng, 9, 2), c.vec(rng, 9, 2)
        return c, k, v

    def state(c):
        torch.cuda.synchronize()
        return c.c.status_words.tolist()

    for slots, before, n_new, want in (([0, 3], [0, 0], [3, 6], [dkv.DKV_ERR_ARG, 1]),
                                       ([-1, 2], [0, 0], [3, 6], [dkv.DKV_ERR_ARG, 0]),
                                       ([0, 1], [0, 43], [3, 6], [dkv.DKV_ERR_TABLE_FULL, 1]),
                                       ([0, 1], [0, 2 ** 31 - 1], [3, 6], [dkv.DKV_ERR_TABLE_FULL, 1])):
        c, k, v = fresh()
        dkv.dkv_cache8_append(c.c, i32(before), k, v, rope=c.rope, n_new=n_new, slots=i32(slots))
        assert state(c) == want
        # nothing else runs until the words are zeroed
        pages, tail = c.pages.clone(), c.tail.clone()
        dkv.dkv_cache8_append(c.c, i32([0]), k[:5], v[:5], rope=c.rope, n_new=[5])
        out = torch.full((1, 4, 128), 3.0, dtype=F16, device="cuda")
        dkv.dkv_cache8_attention(c.c, i32([0]), torch.cat((k[:1], v[:1]), 1), out)
        dkv.dkv_cache8_prefill(c.c, [1], out.clone(), k[:1], v[:1], out)
        assert state(c) == want and (out == 3).all()
        assert torch.equal(c.tail, tail) and torch.equal(c.pages.view(torch.uint8), pages.view(torch.uint8))
        c.c.status_words.zero_()
        dkv.dkv_cache8_attention(c.c, i32([0]), torch.cat((k[:1], v[:1]), 1), out)
        assert state(c) == [0, 0] and (out == 0).all()
    for step in (False, True):
        c, k, v = fresh()
        dkv.dkv_cache8_append(c.c, i32([0, 0]), k[:2], v[:2], rope=c.rope, n_new=None if step else [1, 1], slots=i32([2, 2]))
        assert state(c) == [dkv.DKV_ERR_ARG, state(c)[1]] and state(c)[1] in (0, 1)
    c, k, v = fresh()
    dkv.dkv_cache8_append(c.c, i32([40]), k, v, rope=c.rope[:44], n_new=[9])     # a table of 44 positions
    assert state(c)[0] in (dkv.DKV_ERR_ARG, dkv.DKV_ERR_TABLE_FULL)
    c, k, v = fresh()
    dkv.dkv_cache8_append(c.c, i32([30]), k, v, rope=c.rope[:38], n_new=[9])
    assert state(c) == [dkv.DKV_ERR_ARG, 0]
    for bad in (-1, 12, 2 ** 30):
        c, k, v = fresh()
        c.table[1, 0] = bad
        dkv.dkv_cache8_append(c.c, i32([0, 8]), k[:9], v[:9], rope=c.rope, n_new=[1, 8])
        assert state(c) == [dkv.DKV_ERR_CHECK, 1]
        c.c.status_words.zero_()
        out = torch.empty((2, 4, 128), dtype=F16, device="cuda")
        dkv.dkv_cache8_attention(c.c, i32([1, 20]), torch.randn((2, 4, 128), device="cuda").half(), out)
        assert state(c) == [dkv.DKV_ERR_CHECK, 1]
    for slots, lens, want in (([0, 3], [1, 1], dkv.DKV_ERR_ARG), ([0, 1], [1, 49], dkv.DKV_ERR_TABLE_FULL),
                              ([0, 1], [1, 2 ** 31 - 1], dkv.DKV_ERR_TABLE_FULL)):
        c, k, v = fresh()
        out = torch.empty((2, 4, 128), dtype=F16, device="cuda")
        dkv.dkv_cache8_attention(c.c, i32(lens), torch.randn((2, 4, 128), device="cuda").half(), out, slots=i32(slots))
        assert state(c) == [want, 1]


def test_short_workspace_and_binding_checks():
    dkv = _dkv()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    c = Cache(2, 2, 16, 4, 3, F16, E4M3)
    q = torch.zeros((4, 4, 128), dtype=F16, device="cuda")
    c.c.workspace_bytes -= 1
    assert dkv.dkv_cache8_attention(c.c, i32([0] * 4), q, torch.empty_like(q), check=False) == dkv.DKV_ERR_SCRATCH
    c.c.workspace_bytes += 1
    k = torch.zeros((4, 2, 128), dtype=F16, device="cuda")
    with pytest.raises(TypeError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4), k.bfloat16(), k)
    with pytest.raises(TypeError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4).cpu(), k, k)
    with pytest.raises(TypeError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4).long(), k, k)
    with pytest.raises(ValueError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4), k[:3], k)
    with pytest.raises(ValueError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4), k, k.transpose(0, 1).contiguous().transpose(0, 1))
    with pytest.raises(ValueError):
        dkv.dkv_cache8_append(c.c, i32([0] * 4), k, k, slots=i32([0]))
    with pytest.raises(ValueError):
        dkv.dkv_cache8_attention(c.c, i32([0] * 4), k, torch.empty_like(q))
    with pytest.raises(ValueError):
        dkv.dkv_cache8_attention(c.c, i32([0] * 4), q, torch.empty((4, 8, 128), dtype=F16, device="cuda")[:, ::2])
    with pytest.raises(ValueError):
        dkv.dkv_cache8_prefill(c.c, [2, 1], q, k, k, torch.empty_like(q))
    with pytest.raises(ValueError):
        dkv.make_cache8(c.pages, c.scales[:2], c.tail, c.table, group_size=2)


# ------------------------------------------------------------------ prompt attention

def prefill_case(hkv, G, lens, elem, window, sinks, seed=0, bad=None):
    rng = np.random.default_rng(seed)
    c = Cache(hkv, G, 16, 1, 1, elem, E4M3)
    n = sum(lens)
    q, k, v = c.vec(rng, n, hkv * G), c.vec(rng, n, hkv), c.vec(rng, n, hkv)
    if bad is not None:       # one request's keys and values are not finite
        a = sum(lens[:bad])
        k[a:a + lens[bad]], v[a:a + lens[bad]] = float("nan"), float("inf")
    out = torch.full_like(q, float("nan"))
    _dkv().dkv_cache8_prefill(c.c, lens, q, k, v, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    qn, kn, vn, got = (x.double().cpu().numpy() for x in (q, k, v, out))
    at = 0
    for i, m in enumerate(lens):
        rows = range(m) if m <= 300 else sorted({0, 1, 15, 16, 31, 32, 63, 64, 127, 128, 129, 255, 256, m // 2, m - 129,
                                                 m - 128, m - 2, m - 1, window - 1, window, window + 1} & set(range(m)))
        for p in rows if i != bad else ():
            see = at + ref.visible(p + 1, window, sinks)
            for h in range(hkv):
                g = slice(h * G, (h + 1) * G)
                want, pv, qk, vm = ref.attend(qn[at + p, g], kn[see, h], vn[see, h])
                tol = ref.tolerance(want, pv, qk, vm, len(see), elem, torch.finfo(elem).eps / 2)
                err = np.abs(got[at + p, g] - want)
                assert (err <= tol).all(), (i, p, h, float((err / tol).max()))
        at += m


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("elem", [F16, BF16])
def test_prefill_groups(G, elem):
    prefill_case(2, G, [1, 37, 130, 260], elem, 0, 0, seed=G)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (31, 0), (64, 4), (128, 0), (129, 130), (200, 300), (255, 1),
                                          (400, 16), (5000, 4)])
def test_prefill_windows(window, sinks):
    prefill_case(1, 4, [300, 17, 640, 2], F16, window, sinks, seed=window)
    prefill_case(2, 5, [129, 290], BF16, window, sinks, seed=window)


def test_prefill_long():
    prefill_case(1, 8, [3000, 2049], F16, 0, 0)
    prefill_case(1, 8, [3000, 2049], BF16, 700, 5)


def test_prefill_requests_do_not_touch_each_other():
    for bad in (0, 1, 2):
        prefill_case(1, 4, [100, 77, 150], F16, 0, 0, seed=bad, bad=bad)
        prefill_case(1, 7, [100, 77, 150], BF16, 40, 3, seed=bad, bad=bad)


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3), (130, 70)])
def test_prefill_of_values_that_are_not_finite(elem, window, sinks):
    """Infinite and NaN keys and values reach the rows that see them, feature by
    feature, and no other."""
    rng = np.random.default_rng(window)
    lens, G, hkv = [210, 333, 70], 3, 2
    c = Cache(hkv, G, 16, 1, 1, elem, E4M3)
    n = sum(lens)
    q, k, v = c.vec(rng, n, hkv * G), c.vec(rng, n, hkv), c.vec(rng, n, hkv)
    clean = [x.double().cpu().numpy() for x in (q, k, v)]
    v[5, 0, 17] = float("inf")                 # a first token
    v[100, 0, 3], v[101, 1, 3] = float("-inf"), float("nan")
    v[210 + 64, :, 100] = float("nan")
    v[210 + 200, 1] = float("inf")
    k[210 + 300, 0, 9] = float("nan")
    bad = [x.double().cpu().numpy() for x in (q, k, v)]
    out = torch.full_like(q, 7.0)
    _dkv().dkv_cache8_prefill(c.c, lens, q, k, v, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    got, at = out.double().cpu().numpy(), 0
    for m in lens:
        for p in range(m):
            see = at + ref.visible(p + 1, window, sinks)
            for h in range(hkv):
                g = slice(h * G, (h + 1) * G)
                want, pv, qk, vm = ref.attend(clean[0][at + p, g], clean[1][see, h], clean[2][see, h])
                tol = ref.tolerance(want, pv, qk, vm, len(see), elem, torch.finfo(elem).eps / 2)
                vb, kb = bad[2][see, h], bad[1][see, h]
                hit = ~np.isfinite(vb).all(axis=0) | ~np.isfinite(kb).all()
                x = got[at + p, g]
                assert not np.isfinite(x[:, hit]).any(), (p, h)
                assert (np.abs(x - want) <= tol)[:, ~hit].all(), (p, h)
        at += m


def test_prefill_after_values_that_are_not_finite():
    """While status[2] is on, finite results stay bit for bit; no error latches."""
    rng = np.random.default_rng(1)
    c = Cache(2, 4, 16, 1, 1, BF16, E4M3)
    q, k, v = c.vec(rng, 500, 8), c.vec(rng, 500, 2), c.vec(rng, 500, 2)
    a, b, d = (torch.empty_like(q) for _ in range(3))
    _dkv().dkv_cache8_prefill(c.c, [400, 100], q, k, v, a, window=50, sinks=1)
    torch.cuda.synchronize()
    words = c.c.tensors[4]
    assert words.tolist() == [0, 0, 0, 0]
    bad = v.clone()
    bad[77] = float("inf")
    _dkv().dkv_cache8_prefill(c.c, [400, 100], q, k, bad, b, window=50, sinks=1)
    torch.cuda.synchronize()
    assert words.tolist() == [0, 0, 1, 0]
    sees = torch.zeros(500, dtype=torch.bool, device="cuda")
    sees[77:77 + 50] = True
    assert not torch.isfinite(b[sees].float()).any() and torch.isfinite(b[~sees].float()).all()
    _dkv().dkv_cache8_prefill(c.c, [400, 100], q, k, v, d, window=50, sinks=1)
    assert torch.equal(a, d)


def test_prefill_parts_of_one_projection():
    rng = np.random.default_rng(3)
    c = Cache(2, 4, 16, 1, 1, F16, E4M3)
    qkv = c.vec(rng, 333, 12)
    q, k, v = qkv[:, :8], qkv[:, 8:10], qkv[:, 10:]
    a, b = torch.empty((333, 8, 128), dtype=F16, device="cuda"), torch.empty((333, 8, 128), dtype=F16, device="cuda")
    _dkv().dkv_cache8_prefill(c.c, [300, 33], q, k, v, a, window=100, sinks=2)
    _dkv().dkv_cache8_prefill(c.c, [300, 33], q.contiguous(), k.contiguous(), v.contiguous(), b, window=100, sinks=2)
    assert torch.equal(a, b)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("elem,code,window,sinks", [(F16, E4M3, 0, 0), (BF16, INT8, 90, 4)])
def test_prompt_then_generation(elem, code, window, sinks):
    """Append with rotation, prompt attention over the turned vectors, then 70
    generation steps (append, attention) queued without a wait between them."""
    rng = np.random.default_rng(12)
    hkv, G, T, lens, steps = 2, 4, 32, [150, 64, 31], 70
    c = Cache(hkv, G, T, 3, 8, elem, code, rot=128)
    n = sum(lens)
    q, k, v = c.vec(rng, n, 8), c.vec(rng, n, 2), c.vec(rng, n, 2)
    kr, qr, out = torch.empty_like(k), torch.empty_like(q), torch.empty_like(q)
    slots = [1, 2, 0]
    _, turned = c.append(slots, [0, 0, 0], lens, k, v, q, kr, qr)
    _dkv().dkv_cache8_prefill(c.c, lens, qr, kr, v, out, window=window, sinks=sinks)
    kn, vn, qn, got = (x.double().cpu().numpy() for x in (kr, v, qr, out))
    at = 0
    for m in lens:
        for p in (0, m // 2, m - 1):
            see = at + ref.visible(p + 1, window, sinks)
            for h in range(hkv):
                want, pv, qk, vm = ref.attend(qn[at + p, 4 * h:4 * h + 4], kn[see, h], vn[see, h])
                tol = ref.tolerance(want, pv, qk, vm, len(see), elem, torch.finfo(elem).eps / 2)
                assert (np.abs(got[at + p, 4 * h:4 * h + 4] - want) <= tol).all()
        at += m
    # the steps are queued first, then followed in the reference
    data, outs = [], []
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    for s in range(steps):
        x = [c.vec(rng, 3, 8), c.vec(rng, 3, 2), c.vec(rng, 3, 2)]
        data.append((x, i32([m + s for m in lens]), i32([m + s + 1 for m in lens]), torch.empty_like(x[0])))
        outs.append(torch.empty_like(x[0]))
    sl = i32(slots)
    torch.cuda.synchronize()
    for (x, before, now, q_rot), o in zip(data, outs):
        _dkv().dkv_cache8_append(c.c, before, x[1], x[2], rope=c.rope, slots=sl, q=x[0], q_rot=q_rot)
        _dkv().dkv_cache8_attention(c.c, now, q_rot, o, window=window, sinks=sinks, slots=sl)
    torch.cuda.synchronize()
    for s, ((x, _, _, q_rot), o) in enumerate(zip(data, outs)):
        for i, sl_i in enumerate(slots):
            c.ref.append(sl_i, lens[i] + s, ref.elem_np(x[1])[i:i + 1], ref.elem_np(x[2])[i:i + 1], c.rope_np)
        if s % 9 == 0 or s == steps - 1:
            c.check_attention(o, slots, [m + s + 1 for m in lens], q_rot, window, sinks)
    c.check()


def test_captured_step_replays_with_other_contents():
    """One captured append + attention, replayed over a generation with lengths,
    slots and vectors written between the replays; a padded row skips."""
    dkv = _dkv()
    rng = np.random.default_rng(7)
    c = Cache(2, 4, 16, 4, 6, F16, E4M3, rot=64)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    q, k, v = c.vec(rng, 3, 8), c.vec(rng, 3, 2), c.vec(rng, 3, 2)
    before, now, slots, qr, out = i32([-1] * 3), i32([0] * 3), i32([0, 1, 2]), torch.empty_like(q), torch.empty_like(q)

    def step():
        dkv.dkv_cache8_append(c.c, before, k, v, rope=c.rope, slots=slots, q=q, q_rot=qr)
        dkv.dkv_cache8_attention(c.c, now, qr, out, slots=slots, window=40, sinks=2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    at = {0: 0, 1: 0, 2: 0, 3: 0}
    for s in range(60):
        who = [int(x) for x in rng.permutation(4)[:3]]
        live = [s % 5 != 2, True, s % 7 != 3]
        x = [c.vec(rng, 3, 8), c.vec(rng, 3, 2), c.vec(rng, 3, 2)]
        for dst, src in zip((q, k, v), x):
            dst.copy_(src)
        slots.copy_(i32(who))
        before.copy_(i32([at[w] if a else -1 for w, a in zip(who, live)]))
        now.copy_(i32([at[w] + 1 if a else 0 for w, a in zip(who, live)]))
        g.replay()
        torch.cuda.synchronize()
        for i, (w, a) in enumerate(zip(who, live)):
            if a:
                c.ref.append(w, at[w], ref.elem_np(x[1])[i:i + 1], ref.elem_np(x[2])[i:i + 1], c.rope_np)
                at[w] += 1
            else:
                assert (out[i] == 0).all()
        live_i = [i for i in range(3) if live[i]]
        c.check_attention(out[live_i], [who[i] for i in live_i], [at[who[i]] for i in live_i], qr[live_i], 40, 2)
    c.check()


def test_captured_prompt_attention():
    """A captured prompt attention, replayed over other vectors, beside an append."""
    rng = np.random.default_rng(5)
    c = Cache(2, 4, 32, 2, 8, BF16, E4M3, rot=128)
    lens = [100, 150]
    q, k, v = c.vec(rng, 250, 8), c.vec(rng, 250, 2), c.vec(rng, 250, 2)
    kr, qr, out, before = torch.empty_like(k), torch.empty_like(q), torch.empty_like(q), torch.zeros(2, dtype=torch.int32, device="cuda")

    def run(o):
        _dkv().dkv_cache8_append(c.c, before, k, v, rope=c.rope, n_new=lens, q=q, k_rot=kr, q_rot=qr)
        _dkv().dkv_cache8_prefill(c.c, lens, qr, kr, v, o, window=60, sinks=3)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(out)
    for _ in range(3):
        for t, h in ((q, 8), (k, 2), (v, 2)):
            t.copy_(c.vec(rng, 250, h))
        g.replay()
        again = torch.empty_like(out)
        got = out.clone()
        run(again)
        assert torch.equal(got, again)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 64, 700])
def test_windows_beyond_every_length(window):
    """As no window, whatever the number of first tokens."""
    for sinks in (0, 5, 2 ** 31 - 1):
        prefill_case(1, 4, [300, 17], F16, window, sinks)
        c, slots, q = filled(2, 4, 32, F16, E4M3, [300, 77, 0], seed=2)
        assert torch.equal(c.attend(slots, [300, 77, 0], q), c.attend(slots, [300, 77, 0], q, window, sinks))


def test_first_tokens_beyond_every_length():
    prefill_case(1, 4, [300, 17, 130], BF16, 9, 2 ** 31 - 1)
    c, slots, q = filled(2, 4, 32, F16, E4M3, [300, 77, 0], seed=2)
    assert torch.equal(c.attend(slots, [300, 77, 0], q), c.attend(slots, [300, 77, 0], q, 9, 2 ** 31 - 1))


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (BF16, E4M3), (F16, INT8)])
def test_attention_of_values_that_are_not_finite(elem, code):
    """A visible NaN key makes its heads' rows NaN, an infinite value in the tail
    its feature infinite, and nothing else."""
    rng = np.random.default_rng(9)
    c = Cache(2, 2, 32, 3, 3, elem, code)
    k, v, q = c.vec(rng, 120, 2), c.vec(rng, 120, 2), c.vec(rng, 3, 4)
    k[3, 0, 7] = float("nan")            # request 0, head 0: in a page (e4m3 keeps it, int8 holds 0)
    v[79, 1, 5] = float("inf")           # request 1 (tokens 40..79), head 1: in the tail
    c.append(None, [0, 0, 0], [40, 40, 40], k, v)
    out = c.attend(None, [40, 40, 40], q).float().cpu().numpy()
    assert np.isnan(out[0, :2]).all() == (code == E4M3) and np.isfinite(out[0, 2:]).all()
    assert np.isposinf(out[1, 2:, 5]).all()
    assert np.isfinite(np.delete(out[1], 5, axis=1)).all() and np.isfinite(out[1, :2]).all() and np.isfinite(out[2]).all()


def test_stepping_back_inside_the_open_block():
    """Rejected tokens are written over; the state is that of the tokens kept."""
    rng = np.random.default_rng(2)
    a, b = (Cache(2, 2, 32, 1, 4, BF16, E4M3, rot=32, seed=3) for _ in range(2))
    k, v = a.vec(rng, 90, 2), a.vec(rng, 90, 2)
    bad = a.vec(rng, 12, 2)
    a.append(None, [0], [70], k[:70], v[:70])
    a.append(None, [70], [12], bad, bad)
    a.append(None, [70], [20], k[70:], v[70:])
    b.append(None, [0], [90], k, v)
    torch.cuda.synchronize()
    assert torch.equal(a.pages.view(torch.uint8), b.pages.view(torch.uint8)) and torch.equal(a.scales, b.scales)
    assert np.array_equal(*(ref.from_tiles(ref.elem_np(x.tail)[0, 1], 16)[:, :90 % 32] for x in (a, b)))


def test_largest_batch():
    """1024 requests in one call of each kind, ragged, some padded."""
    rng = np.random.default_rng(4)
    n = 1024
    c = Cache(1, 1, 16, n, 3, F16, INT8, rot=16)
    lens = [int(x) for x in rng.integers(1, 40, n)]
    order = [int(x) for x in rng.permutation(n)]
    k, v, q = c.vec(rng, sum(lens), 1), c.vec(rng, sum(lens), 1), c.vec(rng, n, 1)
    c.append(order, [0] * n, lens, k, v)
    live = [m if i % 7 else 0 for i, m in enumerate(lens)]
    out = c.attend(order, live, q)
    c.check()
    c.check_attention(out, order, live, q)
    step = [m if i % 5 else -1 for i, m in enumerate(lens)]
    c.append(order, step, [1] * n, k[:n], v[:n], step=True)
    c.check()
    got = torch.empty((sum(lens), 1, 128), dtype=F16, device="cuda")
    q2 = c.vec(rng, sum(lens), 1)
    _dkv().dkv_cache8_prefill(c.c, lens, q2, k, v, got, window=11, sinks=2)
    qn, kn, vn, gn = (x.double().cpu().numpy() for x in (q2, k, v, got))
    at = 0
    for m in lens:
        see = at + ref.visible(m, 11, 2)
        want, pv, qk, vm = ref.attend(qn[at + m - 1], kn[see, 0], vn[see, 0])
        assert (np.abs(gn[at + m - 1] - want) <= ref.tolerance(want, pv, qk, vm, len(see), F16, 2.0 ** -11)).all()
        at += m


def test_shared_workspace_of_two_layers():
    """Two layers of one head layout take turns with one workspace."""
    dkv = _dkv()
    lens = [700, 3, 90]
    c, slots, q = filled(2, 4, 32, F16, E4M3, lens, seed=1)
    d, _, q2 = filled(2, 4, 64, BF16, INT8, lens, seed=1)
    want = c.attend(slots, lens, q), d.attend(slots, lens, q2)
    e = dkv.make_cache8(d.pages, d.scales, d.tail, d.table, group_size=4, workspace=c.c.tensors[5])
    d.c = e
    for _ in range(5):
        assert torch.equal(c.attend(slots, lens, q), want[0]) and torch.equal(d.attend(slots, lens, q2), want[1])


@pytest.mark.parametrize("lens", [[40000], [13000, 30001], [24576, 50, 25000]])
def test_unit_over_more_than_32_blocks_of_the_grid(lens):
    c, slots, q = filled(1, 3, 64, BF16, E4M3, lens, seed=3)
    out = c.attend(slots, lens, q)
    c.check_attention(out, slots, lens, q)
    out = c.attend(slots, lens, q, 30000, 5)
    c.check_attention(out, slots, lens, q, 30000, 5)


def test_offsets_beyond_32_bits():
    """Pages, slots and rows behind the first 4 GB give what near ones give."""
    dkv = _dkv()
    hkv, G, T, lens = 2, 4, 64, [200, 64, 130]
    rng = np.random.default_rng(9)
    near = Cache(hkv, G, T, 3, 4, F16, E4M3)
    n_pages, n_slots = 2 ** 33 // (hkv * T * 256) + 1, 2 ** 33 // (hkv * T * 512) + 1
    pages = torch.empty((n_pages, hkv, T // 16, 2, 2048), dtype=E4M3, device="cuda")
    tail = torch.empty((n_slots, hkv, T // 16, 2, 2048), dtype=F16, device="cuda")
    scales = torch.empty((n_pages, hkv, 2), device="cuda")
    table = torch.zeros((n_slots, 4), dtype=torch.int32, device="cuda")
    slots = torch.tensor([n_slots - 1, n_slots // 2 + 1, n_slots - 7], dtype=torch.int32, device="cuda")
    table[slots.long()] = torch.arange(n_pages - 12, n_pages, dtype=torch.int32, device="cuda").reshape(3, 4)
    far = dkv.make_cache8(pages, scales, tail, table, group_size=G)
    total = sum(lens)
    wide = 2 ** 32 // total // 8 * 8 + 8          # rows lie over 8 GB
    space = torch.empty((total, wide), dtype=F16, device="cuda")
    q, k, v = near.vec(rng, total, hkv * G), near.vec(rng, total, hkv), near.vec(rng, total, hkv)
    rows = []
    for i, x in enumerate((q, k, v)):
        y = space[:, 2048 * i:2048 * i + x.shape[1] * 128].view(total, x.shape[1], 128)
        y.copy_(x)
        rows.append(y)
    zero, ln = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.tensor(lens, dtype=torch.int32, device="cuda")
    got = []
    for c, sl, (a, b, d) in ((near.c, None, (q, k, v)), (far, slots, rows)):
        kr, qr, out, dec = torch.empty_like(k), torch.empty_like(q), torch.empty_like(q), torch.empty_like(q[:3])
        dkv.dkv_cache8_append(c, zero, b, d, n_new=lens, slots=sl, q=a, k_rot=kr, q_rot=qr)
        dkv.dkv_cache8_prefill(c, lens, a, b, d, out, window=100, sinks=4)
        dkv.dkv_cache8_attention(c, ln, a[-3:], dec, slots=sl)
        assert c.status_words.tolist() == [0, 0]
        got.append((kr, qr, out, dec))
    for x, y in zip(*got):
        assert torch.isfinite(x).all() and torch.equal(x, y)


def test_padding_rows_with_any_slot():
    dkv = _dkv()
    lens = [70, 0, 33, -5, 16]
    c, slots, q = filled(2, 4, 16, F16, E4M3, [70, 1, 33, 1, 16], seed=6)
    for any_slot in (-1, 5, 2 ** 31 - 1, -2 ** 31):
        who = [s if n > 0 else any_slot for s, n in zip(slots, lens)]
        out = c.attend(who, lens, q)
        c.check_attention(out, slots, lens, q)
        assert (out[1] == 0).all() and (out[3] == 0).all()
        rng = np.random.default_rng(4)
        k, v = c.vec(rng, 5, 2), c.vec(rng, 5, 2)
        tail = c.tail.clone()
        i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
        for n_new in (None, [1] * 5):
            dkv.dkv_cache8_append(c.c, i32([-1] * 5), k, v, n_new=n_new, slots=i32([any_slot] * 5))
        torch.cuda.synchronize()
        assert torch.equal(c.tail.view(torch.int16), tail.view(torch.int16)) and c.c.status_words.tolist() == [0, 0]


def test_workspace_after_a_call_that_latched_an_error():
    """Blocks of a call may begin long apart beside another stream's work: those
    that find an error of their own call already latched still leave the
    workspace as the next call needs it."""
    dkv = _dkv()
    lens = [700, 3000, 1500, 2300]
    c, slots, q = filled(4, 4, 64, F16, E4M3, lens, seed=2)
    apart = dkv.make_cache8(c.pages, c.scales, c.tail, c.table, group_size=4)
    rng = np.random.default_rng(3)
    # one prompt whose blocks hold their multiprocessors for very different times
    p = Cache(1, 8, 64, 1, 1, F16, E4M3)
    pq, pk, pv = (p.vec(rng, 4500, n) for n in (8, 1, 1))
    pout, out = torch.empty_like(pq), torch.empty_like(q)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    sl, ln = i32(slots), i32(lens)
    side = torch.cuda.Stream()
    good = c.table.clone()
    # arrivals lie behind the partial results, two a multiprocessor
    count = c.c.tensors[5][torch.cuda.get_device_properties(0).multi_processor_count * 2 * (4 * 128 + 16) * 4:]
    assert count.numel() >= 16 * len(lens) * 4
    for bad in (0, 1, 2, 3) * 5:
        c.table.copy_(good)
        c.table[slots[bad], 0] = -1
        torch.cuda.synchronize()
        dkv.dkv_cache8_prefill(p.c, [4500], pq, pk, pv, pout, stream=side)
        dkv.dkv_cache8_attention(c.c, ln, q, out, slots=sl)
        torch.cuda.synchronize()
        assert c.c.status_words.tolist() == [dkv.DKV_ERR_CHECK, bad]
        assert not count.any()
        c.table.copy_(good)
        q = c.vec(rng, len(lens), 16)
        want = torch.empty_like(q)
        dkv.dkv_cache8_attention(apart, ln, q, want, slots=sl)
        c.attend(slots, lens, q)          # stopped
        c.c.status_words.zero_()
        assert torch.equal(c.attend(slots, lens, q), want) and c.c.status_words.tolist() == [0, 0]


def test_prompt_attention_of_two_streams_at_once():
    """Blocks share their items out as they come free: whoever takes which, beside
    whatever else runs, alone and replayed, the results are the same bits."""
    dkv = _dkv()
    rng = np.random.default_rng(12)
    cases = []
    for hkv, G, elem, window, sinks in ((4, 4, F16, 0, 0), (2, 7, BF16, 300, 5)):
        c = Cache(hkv, G, 16, 1, 1, elem, E4M3)
        lens = [int(x) for x in rng.integers(1, 3000, 12)] + [64, 1]
        q, k, v = (c.vec(rng, sum(lens), n) for n in (hkv * G, hkv, hkv))
        want = torch.full_like(q, float("nan"))
        dkv.dkv_cache8_prefill(c.c, lens, q, k, v, want, window=window, sinks=sinks)
        assert torch.isfinite(want).all()
        cases.append((c, lens, q, k, v, want, window, sinks))
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(x[5], float("nan")) for _ in range(6)] for x in cases]
    graphs = []
    torch.cuda.synchronize()
    for x, s, o in zip(cases, streams, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            dkv.dkv_cache8_prefill(x[0].c, *x[1:5], o[0], window=x[6], sinks=x[7])
        graphs.append(g)
    torch.cuda.synchronize()
    for i in range(1, 6):
        for x, s, o, g in zip(cases, streams, outs, graphs):
            dkv.dkv_cache8_prefill(x[0].c, *x[1:5], o[i], window=x[6], sinks=x[7], stream=s)
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, o in zip(cases, outs):
        assert x[0].c.status_words.tolist() == [0, 0]
        for y in o:
            assert torch.equal(y, x[5])


def test_generation_on_a_stream_of_higher_priority_beside_prompts():
    """Blocks of the prompt attention that cannot have another block's item (work of
    higher priority waits) end; what they leave begins later."""
    dkv = _dkv()
    rng = np.random.default_rng(21)
    lens = [900, 100, 1300, 5000]
    d, slots, dq = filled(4, 4, 64, F16, E4M3, lens, seed=1)
    dwant = d.attend(slots, lens, dq)
    p = Cache(8, 4, 64, 1, 1, F16, E4M3)
    prompts = [4000, 1500, 2500, 700]
    q, k, v = (p.vec(rng, sum(prompts), n) for n in (32, 8, 8))
    want = torch.empty_like(q)
    dkv.dkv_cache8_prefill(p.c, prompts, q, k, v, want)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    sl, ln = i32(slots), i32(lens)
    low, high = torch.cuda.Stream(priority=0), torch.cuda.Stream(priority=-1)
    outs, douts = [torch.full_like(q, float("nan")) for _ in range(6)], [torch.empty_like(dq) for _ in range(200)]
    torch.cuda.synchronize()
    for o in outs:
        dkv.dkv_cache8_prefill(p.c, prompts, q, k, v, o, stream=low)
    for o in douts:
        dkv.dkv_cache8_attention(d.c, ln, dq, o, slots=sl, stream=high)
    torch.cuda.synchronize()
    assert p.c.status_words.tolist() == [0, 0] and d.c.status_words.tolist() == [0, 0]
    assert all(torch.equal(o, want) for o in outs) and all(torch.equal(o, dwant) for o in douts)


def test_other_streams_and_workspaces():
    """Two caches on two streams at once, and one cache read by two streams with a
    workspace each."""
    dkv = _dkv()
    lens = [900, 100, 1300]
    c, slots, q = filled(4, 4, 64, F16, E4M3, lens, seed=1)
    want = c.attend(slots, lens, q)
    torch.cuda.synchronize()
    other = dkv.make_cache8(c.pages, c.scales, c.tail, c.table, group_size=4)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    sl, ln = i32(slots), i32(lens)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(q) for _ in range(40)] for _ in range(2)]
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        dkv.dkv_cache8_attention(c.c, ln, q, a, slots=sl, stream=streams[0])
        with torch.cuda.stream(streams[1]):
            dkv.dkv_cache8_attention(other, ln, q, b, slots=sl)
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o, want)


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("amp", [1e9, 4e10, 1e12, 1e30, 3e38])
def test_attention_of_zero_values_beside_huge_ones(code, amp):
    """Tokens whose values are zero keep their weight beside blocks of any finite
    size: in pages and in the tail, inside one warp's tiles, over the warps of a
    block and over blocks of the grid."""
    lens = [64, 70, 90, 500, 9000, 5]
    rng = np.random.default_rng(8)
    c = Cache(1, 3, 32, len(lens), 9000 // 32 + 1, BF16, code, fill=float("nan"))
    n = sum(lens)
    k, q = (c.vec(rng, n, 1).float() * 1e-2).to(BF16), c.vec(rng, len(lens), 3)
    v = torch.full((n, 1, 128), amp, device="cuda")
    at = 0
    for i, m in enumerate(lens):
        f = torch.ones(m, 1, 1, device="cuda")
        if i % 2 == 0:
            f[:m // 2 // 32 * 32 or 2] = 0.0           # the first half
        else:
            f[m // 2 // 32 * 32:] = 0.0                # the second, the open block with it
        v[at:at + m] *= f
        at += m
    v = v.to(BF16)
    c.append(None, [0] * len(lens), lens, k, v)
    for window, sinks in ((0, 0), (60, 33)):
        out = c.attend(None, lens, q, window, sinks)
        assert torch.isfinite(out).all()
        c.check_attention(out, range(len(lens)), lens, q, window, sinks)


def test_attention_of_many_light_tokens_of_zero_values():
    """fp16: thousands of zero values, 2^-20 of the largest weight each, beside one
    value of the type's largest size."""
    for lens in ([4200], [4200, 900, 4100]):
        c = Cache(1, 2, 64, len(lens), 70, F16, INT8)
        n = sum(lens)
        k, v = (torch.zeros((n, 1, 128), dtype=F16, device="cuda") for _ in range(2))
        q = torch.zeros((len(lens), 2, 128), dtype=F16, device="cuda")
        q[:, :, 0] = 8.0
        at = 0
        for m in lens:
            p = at + m - 100
            k[p, 0, 0], v[p] = 20.0, 65504.0       # 160 / sqrt(128) is 20.4 in powers of two
            at += m
        c.append(None, [0] * len(lens), lens, k, v)
        out = c.attend(None, lens, q)
        c.check_attention(out, range(len(lens)), lens, q)


def test_group_sizes_on_two_host_threads(tmp_path):
    """Caches of the smallest and the largest group, each served by a host thread and
    a stream of its own: calls of the C entry without Python between them."""
    import ctypes as C
    import subprocess
    dkv = _dkv()
    (tmp_path / "two.c").write_text("""
#include <pthread.h>
#include "dkv.h"
typedef int (*entry)(const dkv_cache8*, int32_t, const int32_t*, const int32_t*, const void*, int64_t, void*, int32_t,
                     int32_t, void*);
struct job { entry f; const dkv_cache8* c; const int32_t *slots, *lens; const void* q; void *out, *stream; int32_t n_req;
             int32_t calls, failed; };
static void* serve(void* p) {
  struct job* j = p;
  for (int i = 0; i < j->calls; i++)
    j->failed += j->f(j->c, j->n_req, j->slots, j->lens, j->q, (int64_t)j->c->n_kv_heads * j->c->group_size * 128, j->out, 0,
                      0, j->stream) != 0;
  return 0;
}
void two(struct job* a, struct job* b) {
  pthread_t t;
  pthread_create(&t, 0, serve, a);
  serve(b);
  pthread_join(t, 0);
}
""")
    so = str(tmp_path / "two.so")
    subprocess.run(["gcc", "-shared", "-fPIC", "-pthread", "-I", str(dkv.build.INCLUDE), "-o", so, str(tmp_path / "two.c")],
                   check=True)

    class Job(C.Structure):
        _fields_ = [(n, C.c_void_p) for n in ("f", "c", "slots", "lens", "q", "out", "stream")] + \
            [(n, C.c_int32) for n in ("n_req", "calls", "failed")]

    lens = [100, 33]
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    keep, jobs = [], []
    for G in (1, 8):
        c, slots, q = filled(1, G, 32, F16, E4M3, lens, seed=G)
        sl, ln, out, stream = i32(slots), i32(lens), torch.empty_like(q), torch.cuda.Stream()
        keep.append((c, sl, ln, q, out, stream, c.attend(slots, lens, q)))
        jobs.append(Job(C.cast(dkv.load().dkv_cache8_attention, C.c_void_p), c.c.address, sl.data_ptr(), ln.data_ptr(),
                        q.data_ptr(), out.data_ptr(), stream.cuda_stream, 2, 50000, 0))
    torch.cuda.synchronize()
    C.CDLL(so).two(C.byref(jobs[0]), C.byref(jobs[1]))
    torch.cuda.synchronize()
    assert [j.failed for j in jobs] == [0, 0]
    for c, _, _, _, out, _, want in keep:
        assert torch.equal(out, want) and c.c.status_words.tolist() == [0, 0]


@pytest.mark.parametrize("elem", [F16, BF16])
def test_prefill_of_own_keys_of_infinite_weight_zero(elem):
    """A row whose own key's logit is -Inf (weight 0) and that does not see the NaN
    beside it has the result of its other keys."""
    rng = np.random.default_rng(3)
    n, G = 150, 2
    c = Cache(1, G, 16, 1, 1, elem, E4M3)
    q, k, v = c.vec(rng, n, G), c.vec(rng, n, 1), c.vec(rng, n, 1)
    q[:, :, 9] = q[:, :, 9].abs() + 0.5
    k[[10, 90], 0, 9] = float("-inf")
    v[[12, 100], 0, ::3] = float("nan")
    out = torch.empty_like(q)
    _dkv().dkv_cache8_prefill(c.c, [n], q, k, v, out, window=30, sinks=2)
    torch.cuda.synchronize()
    got, qn, kn, vn = (x.double().cpu().numpy() for x in (out, q, k, v))
    for p in range(n):
        see = ref.visible(p + 1, 30, 2)
        hit = ~np.isfinite(vn[see, 0]).all(axis=0)
        see = see[np.isfinite(kn[see, 0]).all(axis=1)]      # the others have no weight
        want, pv, qk, vm = ref.attend(qn[p], kn[see, 0], np.nan_to_num(vn[see, 0]))
        tol = ref.tolerance(want, pv, qk, vm, len(see), elem, torch.finfo(elem).eps / 2)
        assert np.isnan(got[p][:, hit]).all() and (np.abs(got[p] - want) <= tol)[:, ~hit].all(), p


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 20)])
def test_prefill_of_infinite_values_of_both_signs(elem, window, sinks):
    """Infinite values give their feature their sign, both signs give NaN, whichever
    is nearer, and a NaN gives NaN."""
    rng = np.random.default_rng(4)
    n, G = 300, 2
    c = Cache(1, G, 16, 1, 1, elem, E4M3)
    q, k, v = c.vec(rng, n, G), c.vec(rng, n, 1), c.vec(rng, n, 1)
    inf = float("inf")
    v[10, 0, 3], v[200, 0, 3] = inf, -inf
    v[5, 0, 4], v[180, 0, 4] = -inf, inf
    v[8, 0, 5], v[100, 0, 5] = float("nan"), inf
    v[[0, 130], 0, 6] = -inf
    out = torch.empty_like(q)
    _dkv().dkv_cache8_prefill(c.c, [n], q, k, v, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    got, vn = out.double().cpu().numpy(), v.double().cpu().numpy()
    for p in range(n):
        x = vn[ref.visible(p + 1, window, sinks), 0]
        up, down, nan = (x == inf).any(axis=0), (x == -inf).any(axis=0), np.isnan(x).any(axis=0)
        nan |= up & down
        g = got[p]
        assert np.isnan(g[:, nan]).all() and (g[:, up & ~nan] == inf).all() and (g[:, down & ~nan] == -inf).all(), p
        assert np.isfinite(g[:, ~(up | down | nan)]).all(), p


def scattered(rng, x, share, kinds=(float("nan"), float("inf"), float("-inf"))):
    """x with a share of its entries not finite."""
    x = x.clone()
    hit = torch.from_numpy(rng.random(tuple(x.shape)) < share).cuda()
    x[hit] = torch.from_numpy(rng.choice(np.float32(kinds), int(hit.sum()))).to(x.dtype).cuda()
    return x


@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("elem,window,sinks,share", [(F16, 0, 0, 2e-4), (BF16, 50, 3, 2e-3), (F16, 129, 200, 2e-4), (BF16, 300, 0, 2e-5),
                                                     (F16, 17, 70, 2e-2), (F16, 64, 1, 0.5)])
def test_prefill_of_scattered_values_that_are_not_finite(G, elem, window, sinks, share):
    """Every row against the definition, feature by feature: NaN, +Inf, -Inf or the
    number that the keys which it sees give."""
    rng = np.random.default_rng(1000 * G + window)
    lens, hkv = [1, 290, 37, 405], 2
    c = Cache(hkv, G, 16, 1, 1, elem, E4M3)
    n = sum(lens)
    q, k, v = c.vec(rng, n, hkv * G), c.vec(rng, n, hkv), c.vec(rng, n, hkv)
    v = scattered(rng, v, share)
    if share < 1e-3:
        k = scattered(rng, k, 2e-5)
        q[[5, 300], 1 % G] = float("nan")
    out = torch.empty_like(q)
    _dkv().dkv_cache8_prefill(c.c, lens, q, k, v, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    got, qn, kn, vn = (x.double().cpu().numpy() for x in (out, q, k, v))
    at = 0
    with np.errstate(invalid="ignore"):
        for m in lens:
            for p in range(m):
                see = at + ref.visible(p + 1, window, sinks)
                for h in range(hkv):
                    x, kk = vn[see, h], kn[see, h]
                    up, down = (x == np.inf).any(axis=0), (x == -np.inf).any(axis=0)
                    for g in range(h * G, (h + 1) * G):
                        s = kk @ qn[at + p, g] / np.sqrt(128)
                        nan = np.isnan(x).any(axis=0) | (up & down) | np.isinf(x[s == -np.inf]).any(axis=0)
                        use = s > -np.inf
                        if np.isnan(s).any() or (s == np.inf).any() or not use.any():
                            nan[:] = True
                        r = got[at + p, g]
                        assert np.isnan(r[nan]).all() and (r[up & ~nan] == np.inf).all() and (r[down & ~nan] == -np.inf).all(), (p, g)
                        rest = ~(nan | up | down)
                        if rest.any():
                            y = np.where(np.isfinite(x[use]), x[use], 0)
                            want, pv, qk, vm = ref.attend(qn[at + p, g:g + 1], kk[use], y)
                            tol = ref.tolerance(want, pv, qk, vm, len(see), elem, torch.finfo(elem).eps / 2)
                            assert (np.abs(r - want[0]) <= tol[0])[rest].all(), (p, g)
            at += m


def test_prefill_cost_of_one_value_that_is_not_finite():
    """One NaN in a first token that every row sees, or in its key: no more than a
    look through the results and the values beside the call itself."""
    rng = np.random.default_rng(0)
    n, hkv, G, window, sinks = 8192, 4, 8, 2048, 16
    c = Cache(hkv, G, 16, 1, 1, F16, E4M3)
    q, k, v = c.vec(rng, n, hkv * G), c.vec(rng, n, hkv), c.vec(rng, n, hkv)
    out = torch.empty_like(q)
    bad_v, bad_k = v.clone(), k.clone()
    bad_v[3, :, 17], bad_k[3, :, 17] = float("nan"), float("nan")

    def time_of(k, v):
        best = []
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            c.c.tensors[4].zero_()
            a.record()
            _dkv().dkv_cache8_prefill(c.c, [n], q, k, v, out, window=window, sinks=sinks)
            b.record()
            torch.cuda.synchronize()
            best.append(a.elapsed_time(b))
        return min(best[1:])

    clean = time_of(k, v)
    for kk, vv in ((k, bad_v), (bad_k, v)):
        assert time_of(kk, vv) < 3 * clean      # by a walk through every row's keys: hundreds
        assert torch.isnan(out[3:]).any(dim=2).all()


def test_prefill_looks_for_values_that_are_not_finite_in_their_own_call_only():
    """A call with an infinite value leaves a mark for the caller and no cost to later
    calls (a look through their results would more than double this shape's time)."""
    rng = np.random.default_rng(1)
    lens, hkv, G = [4096] * 8, 8, 8
    c = Cache(hkv, G, 16, 1, 1, BF16, E4M3)
    q, k, v = (torch.randn((sum(lens), n, 128), device="cuda").to(BF16) for n in (hkv * G, hkv, hkv))
    out, bad = torch.empty_like(q), v.clone()
    bad[77] = float("inf")

    def run(v):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        _dkv().dkv_cache8_prefill(c.c, lens, q, k, v, out, window=32)
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b)

    before = min(run(v) for _ in range(10))
    want = out.clone()
    assert c.c.not_finite.item() == 0
    run(bad)
    assert c.c.not_finite.item() == 1 and c.c.tensors[4].tolist() == [0, 0, 1, 0]
    after = min(run(v) for _ in range(10))
    assert torch.equal(out, want) and c.c.tensors[4].tolist() == [0, 0, 1, 0]
    assert after < 1.15 * before, (before, after)
    c.c.not_finite.zero_()
    run(bad)
    assert c.c.tensors[4].tolist() == [0, 0, 1, 0] and not torch.isfinite(out[77:77 + 32]).any()
    assert torch.isfinite(out[:77]).all() and torch.isfinite(out[77 + 32:]).all()


def test_first_call_on_another_stream_than_the_descriptor_was_made_on():
    """Status words and workspace are zero when make_cache8 returns, whatever the
    stream that it ran on still has to do."""
    dkv = _dkv()
    lens = [3000, 700, 1]
    c, slots, q = filled(4, 4, 64, F16, E4M3, lens, seed=1)
    want = c.attend(slots, lens, q)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    sl, ln, out, side = i32(slots), i32(lens), torch.full_like(q, float("nan")), torch.cuda.Stream()
    size = c.c.tensors[5].numel()
    dirty = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (size, 16)]
    torch.cuda.synchronize()
    del dirty                            # the next allocations of these sizes
    torch.cuda._sleep(100_000_000)       # some 50 ms
    d = dkv.make_cache8(c.pages, c.scales, c.tail, c.table, group_size=4)
    dkv.dkv_cache8_attention(d, ln, q, out, slots=sl, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and d.tensors[4].tolist() == [0] * 4 and not torch.isnan(out).any()


def test_a_device_that_is_not_there_leaves_no_error_behind():
    import ctypes as C
    dkv = _dkv()
    c = Cache(2, 2, 16, 4, 3, F16, E4M3)
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    x, y, ln = (torch.zeros((4, n, 128), dtype=F16, device="cuda") for n in (4, 2, 1))
    out, ln = torch.empty_like(x), i32([1] * 4)
    n = C.c_int64()
    c.c.device = torch.cuda.device_count()
    for call in (lambda: dkv.load().dkv_cache8_workspace(c.c.address, 4, C.byref(n)),
                 lambda: dkv.dkv_cache8_append(c.c, ln, y, y, check=False),
                 lambda: dkv.dkv_cache8_attention(c.c, ln, x, out, check=False),
                 lambda: dkv.dkv_cache8_prefill(c.c, [4], x, y, y, out, check=False)):
        assert call() == dkv.DKV_ERR_CUDA
        assert torch.ones(3, device="cuda").mul(2).sum().item() == 6      # raises what is left behind


def test_which_error_and_which_request():
    """One slot given to several requests, and a position behind the page table and the
    rotation table both: one code each, of a request concerned."""
    dkv = _dkv()
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")
    rng = np.random.default_rng(2)
    for step in (False, True):
        c = Cache(2, 2, 16, 4, 3, F16, E4M3, rot=32)
        k, v = c.vec(rng, 4, 2), c.vec(rng, 4, 2)
        dkv.dkv_cache8_append(c.c, i32([0] * 4), k, v, rope=c.rope, n_new=None if step else [1] * 4, slots=i32([3, 1, 0, 1]))
        torch.cuda.synchronize()
        error, request = c.c.status_words.tolist()
        assert error == dkv.DKV_ERR_ARG and request in (1, 3)
    for before, want in ((40, dkv.DKV_ERR_TABLE_FULL), (39, dkv.DKV_ERR_ARG)):     # 49 and 48 tokens of 48 places, 44 positions
        c = Cache(2, 2, 16, 1, 3, F16, E4M3, rot=32)
        k, v = c.vec(rng, 9, 2), c.vec(rng, 9, 2)
        dkv.dkv_cache8_append(c.c, i32([before]), k, v, rope=c.rope[:44], n_new=[9])
        torch.cuda.synchronize()
        assert c.c.status_words.tolist() == [want, 0]


def test_lengths_below_what_is_stored():
    """The open block holds the newest tokens: any length inside it is good, and any
    end of a block; a slot may occur with several of them."""
    stored, T = 150, 32
    lens = [150, 149, 129, 128, 96, 64, 32, 0]
    c, slots, _ = filled(2, 4, T, BF16, INT8, [stored, 20], seed=5)
    q = c.vec(np.random.default_rng(5), len(lens), 8)
    who = [slots[0]] * len(lens)
    for window, sinks in ((0, 0), (40, 3)):
        out = c.attend(who, lens, q, window, sinks)
        c.check_attention(out, who, lens, q, window, sinks)


@pytest.mark.parametrize("elem,code", [(F16, E4M3), (F16, INT8), (BF16, E4M3), (BF16, INT8)])
def test_attention_of_the_largest_values(elem, code):
    """Means of values of the type's largest size do not round to infinite ones."""
    rng = np.random.default_rng(7)
    lens = [2000, 992, 300, 50]
    c = Cache(1, 4, 64, len(lens), 2000 // 64 + 1, elem, code)
    k = c.vec(rng, sum(lens), 1)
    sign = torch.from_numpy(np.where(rng.random((1, 1, 128)) < 0.5, -1.0, 1.0)).cuda()
    v = (sign * torch.finfo(elem).max).expand(sum(lens), 1, 128).to(elem).contiguous()
    c.append(None, [0] * len(lens), lens, k, v)
    for scale in [0.5, 1.0, 2.0, 4.0] * 25:
        q = c.vec(rng, len(lens), 4, scale)
        out = c.attend(None, lens, q)
        assert torch.isfinite(out).all()
    c.check_attention(out, range(len(lens)), lens, q)


@pytest.mark.parametrize("elem", [F16, BF16])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_prefill_of_the_largest_values(elem, window, sinks):
    """Means of values of the type's largest size do not come out infinite, beside
    infinite ones that are and NaN out of sight."""
    rng = np.random.default_rng(8)
    lens, G = [3000, 40], 4
    c = Cache(1, G, 16, 1, 1, elem, E4M3)
    n, top = sum(lens), torch.finfo(elem).max
    q, k = c.vec(rng, n, G, 1.5), c.vec(rng, n, 1)
    sign = torch.from_numpy(np.where(rng.random((1, 1, 128)) < 0.5, -1.0, 1.0)).cuda()
    v = (sign * top).expand(n, 1, 128).to(elem).contiguous()
    inf = float("inf")
    v[700, 0, 5], v[900, 0, 6], v[1300, 0, 7], v[2999, 0, 8] = inf, -inf, float("nan"), inf
    out = torch.empty_like(q)
    _dkv().dkv_cache8_prefill(c.c, lens, q, k, v, out, window=window, sinks=sinks)
    torch.cuda.synchronize()
    got, vn, sign = out.double().cpu().numpy(), v.double().cpu().numpy(), sign.cpu().numpy()[0]
    at = 0
    for m in lens:
        for p in range(m):
            x = vn[at + ref.visible(p + 1, window, sinks), 0]
            want = np.where(np.isfinite(x).all(axis=0), sign * top, x.max(axis=0) + x.min(axis=0))[0]      # Inf + top, Inf - Inf, NaN
            r = got[at + p]
            fin = np.isfinite(want)
            assert (np.isnan(r) == np.isnan(want)).all() and (r == want)[:, np.isinf(want)].all(), p
            # weights off by half a step each, and half a step of the result
            assert np.isfinite(r[:, fin]).all() and (np.abs(r[:, fin] - want[fin]) <= 1.1 * torch.finfo(elem).eps * top).all(), p
        at += m


def test_prefill_of_the_largest_values_in_many_rows():
    """fp16 weights round up enough in one row of some thousands."""
    rng = np.random.default_rng(0)
    n, G = 3000, 4
    c = Cache(1, G, 16, 1, 1, F16, E4M3)
    v = torch.full((n, 1, 128), 65504.0, dtype=F16, device="cuda")
    for _ in range(12):
        q, k = c.vec(rng, n, G), c.vec(rng, n, 1)
        out = torch.empty_like(q)
        _dkv().dkv_cache8_prefill(c.c, [n], q, k, v, out)
        assert torch.isfinite(out).all() and (out >= 65504 * (1 - 2.0 ** -10)).all()


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("amp", [1e-37, 1e-20, 1e20, 1e35, 3e38])
def test_attention_of_bf16_queries_of_any_size(code, amp):
    """Queries over bf16's whole range beside keys of zero and (where the logits stay in
    fp32's range) others."""
    rng = np.random.default_rng(4)
    lens = [150, 64, 20]
    c = Cache(1, 4, 32, len(lens), 5, BF16, code)
    v, n = c.vec(rng, sum(lens), 1), sum(lens)
    for zero in (True, False):
        if not zero and amp > 1e35:
            continue
        k = torch.zeros((n, 1, 128), dtype=BF16, device="cuda")
        if not zero:
            k = (c.vec(rng, n, 1).float() * min(1.0, 1e30 / amp)).to(BF16)
        q = c.vec(rng, len(lens), 4).float()
        q = (q / q.abs().max() * amp).to(BF16)
        c.append(None, [0] * len(lens), lens, k, v)
        out = c.attend(None, lens, q)
        assert torch.isfinite(out).all()
        c.check_attention(out, range(len(lens)), lens, q)


@pytest.mark.parametrize("code", [E4M3, INT8])
@pytest.mark.parametrize("elem,what,size", [(F16, "k", 6e4), (F16, "v", 6e4), (BF16, "k", 1e18), (BF16, "v", 3e4), (BF16, "v", 1e7),
                                            (BF16, "v", 1e9), (BF16, "v", -3e38)])
@pytest.mark.parametrize("T,G,sinks", [(128, 1, 0), (64, 4, 20), (32, 8, 5)])
def test_decode_of_blocks_that_the_window_cuts(elem, code, what, size, T, G, sinks):
    """Decode attention beside stored tokens of any size that are out of sight, where a warp has
    many tiles (hundreds of requests over one slot)."""
    rng = np.random.default_rng(62)
    n, reqs = 1000, 200
    c = Cache(1, G, T, 1, n // T + 1, elem, code, seed=21, fill=float("nan"))
    k, v = c.vec(rng, n, 1), c.vec(rng, n, 1)
    x = k if what == "k" else v
    hidden = T + 9
    x[[hidden, sinks + 1]] = size
    c.append([0], [0], [n], k, v)
    q = c.vec(rng, reqs, G)
    c.c = _dkv().make_cache8(c.pages, c.scales, c.tail, c.table, group_size=G, max_req=reqs)
    window = n - hidden - 1
    out = c.attend([0] * reqs, [n] * reqs, q, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert c.c.status_words.tolist() == [0, 0]
    rows = [0, 1, 77, 198, 199]
    c.check_attention(out[rows], [0] * 5, [n] * 5, q[rows], window=window, sinks=sinks)
