"""The uniform 8-bit cache without a GPU: descriptor layout, the stored order,
refused arguments."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest

import differentiated_kv_cache_gb300 as dkv
from tests import cache8_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_descriptor_layout_matches_header(tmp_path):
    names = [f for f, _ in dkv.dkv_cache8._fields_]
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "dkv.h"', "int main(void){",
             'printf("%zu\\n", sizeof(dkv_cache8));']
    lines += [f'printf("%zu\\n", offsetof(dkv_cache8, {f}));' for f in names] + ["return 0;}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(tmp_path / "l"), str(tmp_path / "l.c")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True).stdout.split()]
    assert got == [C.sizeof(dkv.dkv_cache8)] + [getattr(dkv.dkv_cache8, f).offset for f in names]


@pytest.mark.parametrize("bits", [8, 16])
def test_tile_order_is_a_permutation(bits):
    for p in ref.PLACES[bits]:
        assert sorted(p.reshape(-1)) == list(range(2048))
    x = np.random.default_rng(1).integers(0, 256, (2, 64, 128)).astype(np.uint8)
    assert (ref.from_tiles(ref.to_tiles(x, bits), bits) == x).all()


A = 1 << 20      # an address that no refused call follows


def cache(**over):
    c = dkv.dkv_cache8()
    v = dict(n_kv_heads=2, group_size=4, head_dim=128, block_tokens=64, elem_type=dkv.DKV_F16, code_type=dkv.DKV_E4M3,
             n_pages=8, n_slots=4, table_width=8, rotary_dim=0, rotary_interleaved=0, device=0, pages=A, scales=A, tail=A,
             page_table=A, status=A, workspace=A, workspace_bytes=1 << 30)
    v.update(over)
    for k, x in v.items():
        setattr(c, k, x)
    return c


def refused(rc, want=dkv.DKV_ERR_ARG):
    assert rc == want, rc


BAD_SHAPE = [(dict(n_kv_heads=0), -1), (dict(n_pages=0), -1), (dict(n_slots=0), -1), (dict(n_slots=(1 << 18) + 1), -1),
             (dict(table_width=0), -1), (dict(table_width=1 << 30), -1), (dict(device=-1), -1), (dict(elem_type=2), -1),
             (dict(code_type=-1), -1), (dict(rotary_dim=8), -1), (dict(rotary_dim=144), -1), (dict(rotary_dim=-16), -1),
             (dict(rotary_interleaved=2), -1), (dict(group_size=0), -8), (dict(group_size=9), -8), (dict(head_dim=64), -8),
             (dict(block_tokens=48), -8), (dict(block_tokens=256), -8), (dict(status=None), -1)]


def append(c, n_req=2, n_new=None, slots=None, before=A, k=A, ks=256, v=A, vs=256, q=None, qs=0, rope=None, rope_len=0,
           k_rot=None, q_rot=None):
    nn = None if n_new is None else np.asarray(n_new, np.int32)
    return dkv.load().dkv_cache8_append(None if c is None else C.byref(c), n_req, None if nn is None else nn.ctypes.data,
                                        slots, before, k, ks, v, vs, q, qs, rope, rope_len, k_rot, q_rot, None)


def attention(c, n_req=2, slots=None, lens=A, q=A, qs=1024, out=2 * A, window=0, sinks=0):
    return dkv.load().dkv_cache8_attention(None if c is None else C.byref(c), n_req, slots, lens, q, qs, out, window,
                                           sinks, None)


def prefill(c, n_req=2, lens=(3, 4), q=A, qs=1024, k=A, ks=256, v=A, vs=256, out=2 * A, window=0, sinks=0):
    ln = None if lens is None else np.asarray(lens, np.int32)
    return dkv.load().dkv_cache8_prefill(None if c is None else C.byref(c), n_req, None if ln is None else ln.ctypes.data,
                                         q, qs, k, ks, v, vs, out, window, sinks, None)


@pytest.mark.parametrize("over,code", BAD_SHAPE)
def test_bad_descriptors_are_refused(over, code):
    dkv.build.build()
    refused(append(cache(**over)), code)
    refused(attention(cache(**over)), code)
    refused(prefill(cache(**over)), code)
    if "status" not in over:
        n = C.c_int64()
        refused(dkv.load().dkv_cache8_workspace(C.byref(cache(**over)), 4, C.byref(n)), code)


@pytest.mark.parametrize("over", [dict(pages=None), dict(scales=None), dict(tail=None), dict(page_table=None),
                                  dict(pages=A + 8), dict(tail=A + 2), dict(scales=A + 4), dict(page_table=A + 1)])
def test_storage_is_needed(over):
    dkv.build.build()
    refused(append(cache(**over)))
    refused(attention(cache(**over)))


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=1025), dict(n_req=5), dict(before=None), dict(before=A + 2), dict(slots=A + 1),
    dict(k=None), dict(v=None), dict(k=A + 2), dict(v=A + 8), dict(ks=255), dict(ks=260), dict(ks=128), dict(vs=0),
    dict(vs=-256), dict(q=A), dict(q_rot=A), dict(q=A, q_rot=A + 4, qs=1024), dict(q=A, q_rot=A * 2, qs=512),
    dict(k_rot=A + 8), dict(k_rot=A, ks=512), dict(q=A, q_rot=A, qs=2048), dict(rope=A, rope_len=5),
    dict(n_new=[1, 0]), dict(n_new=[-3, 4]), dict(n_new=[1, 513])])
def test_bad_append_arguments_are_refused(kw):
    dkv.build.build()
    refused(append(cache(), **kw))


def test_rope_is_given_with_a_rotary_dimension_only():
    dkv.build.build()
    c = cache(rotary_dim=64)
    refused(append(c))
    refused(append(c, rope=A, rope_len=0))
    refused(append(c, rope=A + 8, rope_len=9))
    refused(append(None))


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=1025), dict(n_req=5), dict(lens=None), dict(lens=A + 2), dict(slots=A + 3), dict(q=None),
    dict(q=A + 2), dict(qs=1023), dict(qs=1028), dict(qs=512), dict(out=None), dict(out=A + 4), dict(out=A),
    dict(window=-1, out=2 * A),
    dict(sinks=-1)])
def test_bad_attention_arguments_are_refused(kw):
    dkv.build.build()
    refused(attention(cache(), **kw))


def test_attention_needs_a_workspace_and_32_bit_tile_numbers():
    dkv.build.build()
    refused(attention(cache(workspace=None)))
    refused(attention(cache(workspace=A + 8)))
    refused(attention(cache(n_slots=1024, n_kv_heads=4096, table_width=1 << 20), n_req=1024, qs=4096 * 4 * 128))
    refused(attention(None))


@pytest.mark.parametrize("kw", [
    dict(n_req=0), dict(n_req=1025), dict(lens=None), dict(lens=(3, 0)), dict(lens=(-1, 3)), dict(q=None), dict(k=None),
    dict(v=None), dict(out=None), dict(q=A + 2), dict(qs=1020), dict(ks=252), dict(vs=128), dict(out=A + 8),
    dict(window=-5), dict(sinks=-1), dict(lens=(2 ** 31 - 1, 2 ** 31 - 1)), dict(out=A)])
def test_bad_prefill_arguments_are_refused(kw):
    dkv.build.build()
    refused(prefill(cache(), **kw))
    refused(prefill(None))


def test_bad_workspace_requests_are_refused():
    dkv.build.build()
    n = C.c_int64()
    for r in (0, -1, 1025):
        refused(dkv.load().dkv_cache8_workspace(C.byref(cache()), r, C.byref(n)))
    refused(dkv.load().dkv_cache8_workspace(C.byref(cache()), 4, None))


@pytest.mark.parametrize("given", [[3, 1, 40], (3, 1, 40), np.array([3, 1, 40]), np.array([3, 1, 40], np.int32)[::1],
                                   np.array([3, 9, 1, 9, 40, 9], np.int32)[::2], [np.int64(3), 1, np.int32(40)], [3.0, 1, 40]])
def test_host_lengths(given):
    keep, address, n, total = dkv.dkv._lens8(given)
    assert (n, total) == (3, 44) and list((C.c_int32 * 3).from_address(address)) == [3, 1, 40]


@pytest.mark.parametrize("given", [[2 ** 32 + 2, 1], [2 ** 32 + 2, -2 ** 32 + 1], [3, -2 ** 32 + 1], (2 ** 31, 1), [-2 ** 31 - 1],
                                   np.array([2 ** 32 + 2, 1]), np.array([2.0 ** 31]), [2.5, 1], np.array([1.5])])
def test_host_lengths_beyond_32_bits_are_refused(given):
    with pytest.raises(ValueError):
        dkv.dkv._lens8(given)


@pytest.mark.parametrize("window,sinks", [(2 ** 32, 0), (2 ** 32 + 5, 4), (2 ** 31, 0), (5, 2 ** 32), (-2 ** 32, 0), (5, -2 ** 32 + 1)])
def test_windows_beyond_32_bits_are_refused(window, sinks):
    for call in (lambda: dkv.dkv_cache8_attention(None, None, None, None, window=window, sinks=sinks),
                 lambda: dkv.dkv_cache8_prefill(None, None, None, None, None, None, window=window, sinks=sinks)):
        with pytest.raises(ValueError):
            call()
