"""Drafted tokens over the uniform 8-bit cache without a GPU: refused arguments,
and the reference's own trees."""
import ctypes as C

import numpy as np
import pytest

import differentiated_kv_cache_gb300 as dkv
from tests import tree8_ref as tref
from tests.test_cache8 import A, BAD_SHAPE, cache, refused


def tree(c, n_req=2, slots=None, lens=A, nodes=5, n_nodes=None, parents=A, q=A, qs=1024, k=A, ks=256, v=A, vs=256, out=2 * A,
         window=0, sinks=0, ws=A, wb=1 << 30):
    return dkv.load().dkv_cache8_tree(None if c is None else C.byref(c), n_req, slots, lens, nodes, n_nodes, parents, q, qs, k,
                                      ks, v, vs, out, window, sinks, ws, wb, None)


def accept(c, n_req=2, slots=None, before=A, nodes=5, path=A, width=3, n_path=None, k=A, ks=256, v=A, vs=256):
    return dkv.load().dkv_cache8_accept(None if c is None else C.byref(c), n_req, slots, before, nodes, path, width, n_path, k,
                                        ks, v, vs, None)


def rotate(c, n=4, pos=A, axes=1, pair_axis=None, k=A, ks=256, q=None, qs=0, rope=A, rope_len=9, k_rot=A, q_rot=None):
    return dkv.load().dkv_cache8_rotate(None if c is None else C.byref(c), n, pos, axes, pair_axis, k, ks, q, qs, rope, rope_len,
                                        k_rot, q_rot, None)


def append_at(c, n_req=2, n_new=None, slots=None, before=A, pos=A, axes=1, pair_axis=None, k=A, ks=256, v=A, vs=256, q=None,
              qs=0, rope=A, rope_len=9, k_rot=None, q_rot=None):
    nn = None if n_new is None else np.asarray(n_new, np.int32)
    return dkv.load().dkv_cache8_append_at(None if c is None else C.byref(c), n_req, None if nn is None else nn.ctypes.data, slots,
                                           before, pos, axes, pair_axis, k, ks, v, vs, q, qs, rope, rope_len, k_rot, q_rot, None)


@pytest.mark.parametrize("over,code", BAD_SHAPE)
def test_bad_descriptors_are_refused(over, code):
    dkv.build.build()
    refused(tree(cache(**over)), code)
    refused(accept(cache(**over)), code)
    over2 = over if "rotary_dim" in over else dict(over, rotary_dim=64)
    refused(rotate(cache(**over2)), code)
    refused(append_at(cache(**over2)), code)
    if "status" not in over:
        n = C.c_int64()
        refused(dkv.load().dkv_cache8_tree_workspace(C.byref(cache(**over)), 4, C.byref(n)), code)


@pytest.mark.parametrize("over", [dict(pages=None), dict(scales=None), dict(tail=None), dict(page_table=None), dict(pages=A + 8),
                                  dict(tail=A + 2), dict(scales=A + 4), dict(page_table=A + 1)])
def test_storage_is_needed(over):
    dkv.build.build()
    refused(tree(cache(**over)))
    refused(accept(cache(**over)))
    refused(append_at(cache(rotary_dim=32, **over)))


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=1025), dict(n_req=5), dict(lens=None), dict(lens=A + 2), dict(slots=A + 1), dict(nodes=0),
    dict(nodes=129), dict(nodes=-1), dict(n_nodes=A + 2), dict(parents=A + 3), dict(q=None), dict(q=A + 8), dict(qs=1020),
    dict(qs=512), dict(k=None), dict(ks=128), dict(v=None), dict(v=A + 2), dict(vs=260), dict(out=None), dict(out=2 * A + 8),
    dict(out=A), dict(q=2 * A), dict(k=2 * A), dict(v=2 * A), dict(window=-1), dict(sinks=-1), dict(ws=None), dict(ws=A + 8)])
def test_bad_tree_arguments_are_refused(kw):
    dkv.build.build()
    refused(tree(cache(), **kw))


def test_tree_steps_are_numbered_in_32_bits():
    dkv.build.build()
    refused(tree(cache(n_slots=1024, n_kv_heads=4096, table_width=1 << 20), n_req=1024, qs=4096 * 512, ks=4096 * 128, vs=4096 * 128))
    refused(tree(None))
    n = C.c_int64()
    for m in (0, -1, 129):
        refused(dkv.load().dkv_cache8_tree_workspace(C.byref(cache()), m, C.byref(n)))
    refused(dkv.load().dkv_cache8_tree_workspace(C.byref(cache()), 4, None))


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=1025), dict(n_req=5), dict(before=None), dict(before=A + 2), dict(slots=A + 1), dict(nodes=0),
    dict(nodes=129), dict(path=None), dict(path=A + 1), dict(width=0), dict(width=129), dict(n_path=A + 2), dict(k=None),
    dict(k=A + 8), dict(ks=252), dict(v=None), dict(vs=128)])
def test_bad_accept_arguments_are_refused(kw):
    dkv.build.build()
    refused(accept(cache(), **kw))
    refused(accept(None))


@pytest.mark.parametrize("kw", [
    dict(n=0), dict(n=-3), dict(n=2 ** 31 - 1, qs=4096 * 1024), dict(pos=None), dict(pos=A + 2), dict(axes=0), dict(axes=5),
    dict(axes=2), dict(axes=2, pair_axis=bytes([0] * 31 + [2])), dict(pair_axis=bytes([1] * 32)), dict(k=None),
    dict(k_rot=None), dict(k=None, k_rot=None), dict(q=A), dict(q_rot=A), dict(k=A + 2), dict(ks=128),
    dict(q=A, q_rot=A, qs=2048), dict(ks=512), dict(k_rot=A + 8), dict(rope=None), dict(rope=A + 8), dict(rope_len=0)])
def test_bad_rotate_arguments_are_refused(kw):
    dkv.build.build()
    big = "n" in kw and kw["n"] > 5
    refused(rotate(cache(rotary_dim=64, n_kv_heads=4096 if big else 2), **(dict(kw, ks=4096 * 128) if big else kw)))
    refused(rotate(None))
    refused(rotate(cache()))         # nothing turns


@pytest.mark.parametrize("kw", [
    dict(pos=None), dict(pos=A + 2), dict(axes=0), dict(axes=5), dict(axes=3), dict(axes=3, pair_axis=bytes([3] * 32)),
    dict(rope=None), dict(rope_len=0), dict(n_req=0), dict(k=None), dict(vs=0), dict(q=A), dict(n_new=[1, 0]), dict(before=None)])
def test_bad_append_at_arguments_are_refused(kw):
    dkv.build.build()
    refused(append_at(cache(rotary_dim=64), **kw))
    refused(append_at(None))
    refused(append_at(cache()))


def test_reference_trees():
    p = [-1, 0, 0, 1, -1, 4]
    assert tref.depths(p) == [0, 1, 1, 2, 0, 1]
    assert tref.seen(p, 3, 4, 0, 0) == ([0, 1, 2, 3], [0, 1, 3])
    # position 6 with window 3 sees 4, 5, 6: itself and its ancestors at 4 and 5
    assert tref.seen(p, 3, 4, 3, 1) == ([0], [0, 1, 3])
    assert tref.seen(p, 3, 4, 2, 0) == ([], [1, 3])
    assert tref.seen(p, 4, 4, 3, 0) == ([2, 3], [4])
    assert tref.seen(p, 3, 0, 2, 1) == ([], [0, 1, 3])


def test_windows_beyond_32_bits_are_refused():
    with pytest.raises(ValueError):
        dkv.dkv_cache8_tree(None, None, None, None, None, None, None, window=2 ** 32)


def test_pair_axes_are_numbers_one_by_one():
    import torch
    from types import SimpleNamespace
    cache = SimpleNamespace(pairs=8, dev=-1)
    pos = torch.zeros((3, 5), dtype=torch.int32)
    want = bytes([0, 1, 2, 2, 1, 0, 0, 1])
    for given in (want, list(want), tuple(want), np.frombuffer(want, np.uint8).astype(np.int32), torch.tensor(list(want))):
        at, axes, got = dkv.dkv._axes8(cache, pos, given, 5)
        assert (axes, got) == (3, want)
    for bad in (8, [0.5] * 8, [300] * 8, [-1] * 8, [0] * 7, np.zeros(2, np.int32)):
        with pytest.raises((TypeError, ValueError)):
            dkv.dkv._axes8(cache, pos, bad, 5)
    with pytest.raises(ValueError):
        dkv.dkv._axes8(cache, pos, want, 6)


def test_a_cache_without_room_for_drafts_says_what_it_needs():
    import torch
    from types import SimpleNamespace
    dkv.build.build()
    c = cache(group_size=2)
    c.dev, c.elem_dtype, c.heads, c.q_heads, c.pairs = -1, torch.float16, 2, 4, 0
    c.address, c.tree_workspace, c.tree_bytes = C.addressof(c), None, 0
    c.elem_type = dkv.dkv.DKV_F16
    vec = lambda h: torch.zeros((6, h, 128), dtype=torch.float16)
    lens, q, k = torch.zeros(2, dtype=torch.int32), vec(4), vec(2)
    stream = SimpleNamespace(cuda_stream=0)
    with pytest.raises(dkv.DkvError, match="max_nodes=3") as e:
        dkv.dkv_cache8_tree(c, lens, None, q, k, vec(2), vec(4), stream=stream)
    assert e.value.code == dkv.DKV_ERR_ARG
    assert dkv.dkv_cache8_tree(c, lens, None, q, k, vec(2), vec(4), stream=stream, check=False) == dkv.DKV_ERR_ARG
