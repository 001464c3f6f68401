"""Measured cases of drafted tokens and positions with several axes over the
8-bit block-scaled cache: attention for a tree of drafted tokens, the accepted
path's way into the cache, rotation of queries and keys by time, height and
width, and the append with such positions.

Shapes are those of this repository's workloads (32 query / 8 KV heads, 64/8,
40/8, 28/4, head size 128), its prompt and generation lengths, and generic ones.
"""
import math
import random

import numpy as np
import torch

own = False          # False: plain torch forms; True: the library's kernels

D = 128
SUB = 16             # tokens of one stored tile
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
ELEM = {"fp16": torch.float16, "bf16": torch.bfloat16}
LOG2_FLOOR = -100.0  # smallest block scale: 2^-100
DEV = "cuda"


# ---------------------------------------------------------------- cases

def _tree(name, kv, g, n_req, lens, nodes, elem, code, block, chain=False, window=0, sinks=0, seed=1):
    return {"name": name, "op": "tree", "kv": kv, "group": g, "n_req": n_req, "len_min": lens[0], "len_max": lens[1],
            "nodes_min": nodes[0], "nodes_max": nodes[1], "elem": elem, "code": code, "block": block, "chain": chain,
            "window": window, "sinks": sinks, "lens_seed": seed}


def _accept(name, kv, n_req, before, nodes, path, elem, code, block, seed=1):
    return {"name": name, "op": "accept", "kv": kv, "group": 1, "n_req": n_req, "before_min": before[0],
            "before_max": before[1], "nodes_max": nodes, "path_min": path[0], "path_max": path[1], "elem": elem,
            "code": code, "block": block, "lens_seed": seed}


def _rotate(name, kv, g, n_req, new, axes, elem, rotary=128, inter=False, mixed=False, seed=1):
    return {"name": name, "op": "rotate", "kv": kv, "group": g, "n_req": n_req, "new_min": new[0], "new_max": new[1],
            "axes": axes, "elem": elem, "rotary": rotary, "interleaved": inter, "axes_mixed": mixed, "lens_seed": seed}


def _append(name, kv, g, n_req, new, before, axes, elem, code, block, rotary=128, inter=False, mixed=False, q=True, seed=1):
    return {"name": name, "op": "append", "kv": kv, "group": g, "n_req": n_req, "new_min": new[0], "new_max": new[1],
            "before_min": before[0], "before_max": before[1], "axes": axes, "elem": elem, "code": code, "block": block,
            "rotary": rotary, "interleaved": inter, "axes_mixed": mixed, "with_q": q, "lens_seed": seed}


def listed():
    return [
        # one user's short conversation, a small tree of guesses: pure latency
        _tree("tree_one_small", 8, 4, 1, (300, 300), (8, 8), "fp16", "e4m3", 64),
        # a generation step of a batch with 26 guesses each
        _tree("tree_16x4096_26", 8, 4, 16, (4090, 4170), (26, 26), "fp16", "e4m3", 64, seed=2),
        # few long contexts, many query heads a KV head, wide trees: most of the work is in the products
        _tree("tree_8x32768_64", 8, 8, 8, (32768, 32900), (64, 64), "bf16", "int8", 64, seed=3),
        # ragged batch, odd group, trees of any size, a window with four first tokens
        _tree("tree_window_ragged", 4, 7, 32, (1024, 16384), (1, 17), "bf16", "e4m3", 32, False, 4096, 4, 4),
        # many requests with a chain of five guesses each (no branches), short and long
        _tree("tree_chain_64", 8, 5, 64, (1, 3000), (5, 5), "fp16", "int8", 128, True, seed=5),
        # one user's accepted guesses
        _accept("accept_one", 8, 1, (4100, 4100), 26, (4, 4), "fp16", "e4m3", 64),
        # the accepted guesses of a full batch, from none to all of a path
        _accept("accept_128", 4, 128, (1024, 16384), 64, (0, 9), "bf16", "int8", 32, 2),
        # the guesses of a batch, at their depths
        _rotate("rotate_drafts", 8, 4, 16, (26, 26), 3, "fp16", seed=1),
        # frames of videos, pairs of features dealt out to time, height and width in turn
        _rotate("rotate_video", 8, 5, 8, (7000, 8100), 3, "bf16", 128, False, True, 2),
        # the next token of a batch whose prompts hold images: positions are not places in the cache
        _append("append_at_step_128", 4, 7, 128, (1, 1), (1024, 16384), 3, "bf16", "int8", 32, 128, False, True, True, 3),
        # pieces of prompts with images
        _append("append_at_pieces", 8, 4, 24, (1, 1500), (0, 2000), 3, "fp16", "e4m3", 64, 128, False, False, True, 4),
        # whole prompts with images, two axes on adjacent pairs of half of each head
        _append("append_at_prompts", 8, 5, 8, (8000, 8192), (0, 0), 2, "bf16", "e4m3", 128, 64, True, False, True, 5),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "accept", "rotate", "append"))
    kv, g = rng.choice(((8, 4), (8, 8), (8, 5), (4, 7), (2, 4), (1, 8), (4, 1), (3, 6), (5, 3), (2, 2)))
    elem, code = rng.choice(("fp16", "bf16")), rng.choice(("e4m3", "int8"))
    block, seed = rng.choice((16, 32, 64, 128)), rng.randrange(1 << 20)
    rotary, inter, mixed, axes = rng.choice((128, 128, 64, 32, 16)), rng.random() < 0.5, rng.random() < 0.5, rng.choice((1, 2, 3, 3, 4))
    if op == "tree":
        n_req, nodes = _spread(rng, 1, 100), _spread(rng, 1, 128)
        rows = nodes * g
        hi = _spread(rng, 1, max(1, min(40000, 1000000 // (n_req * kv), 400000000 // (n_req * kv * rows))))
        window = rng.choice((0, 0, _spread(rng, 1, 8000)))
        c = _tree("", kv, g, n_req, (max(1, hi // rng.choice((1, 3, 20))), hi), (max(1, nodes // rng.choice((1, 2, 9))), nodes),
                  elem, code, block, rng.random() < 0.25, window, rng.choice((0, 1, 4, 37, 200)) if window else 0, seed)
    elif op == "accept":
        n_req, nodes = _spread(rng, 1, 128), _spread(rng, 1, 128)
        path = rng.randint(1, min(nodes, 20))
        c = _accept("", kv, n_req, (0, _spread(rng, 1, 6000)), nodes, (rng.randint(0, path), path), elem, code, block, seed)
    else:
        n_req = _spread(rng, 1, 128)
        hi = rng.choice((1, _spread(rng, 1, max(1, min(8000, 40000 // n_req)))))
        new = (max(1, hi // rng.choice((1, 2, 9))), hi)
        if op == "rotate":
            c = _rotate("", kv, g, n_req, new, axes, elem, rotary, inter, mixed, seed)
        else:
            c = _append("", kv, g, n_req, new, (0, _spread(rng, 1, 6000)), axes, elem, code, block, rotary, inter, mixed,
                        rng.random() < 0.7, seed)
    del c["name"]
    return c


def _numbers(case, lo, hi, salt):
    r = random.Random(case["lens_seed"] * 1000003 + salt)
    return [r.randint(lo, hi) for _ in range(case["n_req"])]


def _lens(case):
    return _numbers(case, case["len_min"], case["len_max"], 1)


def _nodes(case):
    return _numbers(case, case["nodes_min"], case["nodes_max"], 3)


def _appended(case):
    """Tokens that each request gets, and had before."""
    if case["op"] == "accept":
        return _numbers(case, case["path_min"], case["path_max"], 1), _numbers(case, case["before_min"], case["before_max"], 2)
    new = _numbers(case, case["new_min"], case["new_max"], 1)
    return new, _numbers(case, case["before_min"], case["before_max"], 2) if "before_min" in case else [0] * len(new)


def _parents(case, seed):
    """[n_req][nodes_max] list: node m hangs on an earlier node or (-1) on the last stored token."""
    if case["chain"]:
        return [list(range(-1, case["nodes_max"] - 1)) for _ in range(case["n_req"])]
    r = random.Random(seed * 7919 + case["lens_seed"])
    return [[r.randint(max(-1, m - 12), m - 1) for m in range(case["nodes_max"])] for _ in range(case["n_req"])]


def _cached(n, depth, window, sinks):
    """Stored tokens of n that a node at this depth sees (position n + depth)."""
    if window <= 0:
        return n
    lo = max(n + depth - window + 1, 0)
    return n if lo <= sinks else max(n - lo, 0) + min(sinks, n)


def work(case):
    kv, g = case["kv"], case["group"]
    if case["op"] == "tree":
        t, nbytes, pairs = case["block"], 0, 0
        for n, m, par in zip(_lens(case), _nodes(case), _parents(case, 0)):
            see = _cached(n, 0, case["window"], case["sinks"])
            in_tail = min(see, n % t)
            nbytes += kv * ((see - in_tail) * 2 * D + in_tail * 4 * D + -(-(see - in_tail) // t) * 8)
            nbytes += m * (kv * 4 * D + 2 * kv * g * 2 * D + 4)
            depth = []
            for p in par[:m]:
                depth.append(0 if p < 0 else depth[p] + 1)
                pairs += _cached(n, depth[-1], case["window"], case["sinks"]) + depth[-1] + 1
        return {"bytes": nbytes, "flops": 4 * D * kv * g * pairs}
    new, before = _appended(case)
    total = sum(new)
    nbytes = flops = 0
    if case["op"] != "accept":
        heads = kv * (1 + (g if case.get("with_q", True) else 0))
        nbytes += 2 * total * heads * D * 2 + total * case["axes"] * 4         # vectors read and written, positions
        flops += 3 * total * heads * case["rotary"]
        # every position of every axis' part of the table once
        pos, _ = _positions(case, 0)
        axis = np.array(_pair_axis(case))
        for a in range(case["axes"]):
            nbytes += len(np.unique(pos[a])) * int((axis == a).sum()) * 8
    else:
        nbytes += total * (kv * D * 2 + 4)                                     # keys read, places in the tree
    if case["op"] != "rotate":
        t = case["block"]
        nbytes += total * kv * D * 2                                            # values read
        for n, b in zip(new, before):
            blocks = (b + n) // t - b // t
            nbytes += blocks * kv * (t * 2 * D + 8)                             # codes and scales
            nbytes += (b % t) * kv * D * 4 if blocks else 0                     # tokens already in the open block
            nbytes += ((b + n) % t if blocks else n) * kv * D * 4               # tokens left in it
        flops += 4 * total * kv * D
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- positions

def _pair_axis(case):
    """Which axis each pair of features turns by: parts of the head, or in turn."""
    pairs, n = case["rotary"] // 2, case["axes"]
    if case["axes_mixed"]:
        return [i % n for i in range(pairs)]
    # the first axis (time) has half a share of what the others have
    ends = [round(pairs * (2 * a + 1) / (2 * n - 1)) for a in range(n)]
    return [next(a for a in range(n) if i < ends[a]) for i in range(pairs)]


def _positions(case, seed):
    """[axes][tokens] positions of each request's new tokens back to back, and the table's length."""
    new, before = _appended(case)
    rng = np.random.default_rng(seed * 7919 + case["lens_seed"])
    parts, n_axes = [], case["axes"]
    for n, b in zip(new, before):
        at, have, mine = b // 2 + int(rng.integers(0, 50)), 0, []
        while have < n:
            text = int(rng.integers(1, 60)) if n > 1 else 1
            mine.append(np.repeat((at + np.arange(text))[None], n_axes, 0))
            at += text
            have += text
            if have < n:      # a picture or a few frames: rows and columns on the last axes
                side = [int(x) for x in rng.integers(1, 20, n_axes)]
                side[0] = min(side[0], 4) if n_axes > 2 else side[0]
                grid = np.stack(np.meshgrid(*[np.arange(s) for s in side], indexing="ij")).reshape(n_axes, -1)
                mine.append(at + grid)
                at += max(side)
                have += grid.shape[1]
        parts.append(np.concatenate(mine, 1)[:, :n])
    pos = np.concatenate(parts, 1).astype(np.int32)
    return pos, int(pos.max()) + 1


# ---------------------------------------------------------------- stored order
# A tile holds 16 tokens of one head: 2048 key values, then 2048 value entries,
# in the order that the matrix instructions' registers take them.

def _order(bits):
    """For each place of a tile: where its key value and its value entry lie in [16 tokens][128]."""
    p = torch.arange(SUB * D, device=DEV)
    w = p % 8
    if bits == 8:
        s, lane = 2 * (p // 512) + p // 8 % 2, p // 16 % 32
    else:
        s, lane = p // 256, p // 8 % 32
    row, col = 8 * (w // 4) + lane // 4, 8 * (w // 2 % 2) + 2 * (lane % 4) + w % 2
    return torch.stack((row * D + 16 * s + col, col * D + 16 * s + row))


def _store(x, bits):
    """[..., 2, T, 128] token-major -> [..., T/16, 2, 2048] in stored order."""
    t = x.shape[-2]
    x = x.reshape(*x.shape[:-3], 2, t // SUB, SUB * D).transpose(-2, -3)
    order = _order(bits)
    return torch.stack((x[..., 0, :][..., order[0]], x[..., 1, :][..., order[1]]), dim=-2)


def _restore(x, bits):
    """The inverse of _store."""
    c = x.shape[-3]
    back = _order(bits).argsort(dim=1)
    x = torch.stack((x[..., 0, :][..., back[0]], x[..., 1, :][..., back[1]]), dim=-3)
    return x.reshape(*x.shape[:-3], 2, c * SUB, D)


def _quantise(x, code):
    """Codes and scales of blocks x: [..., T, 128] 16-bit values."""
    f = x.float()
    amax = torch.where(torch.isfinite(f), f.abs(), torch.zeros_like(f)).amax(dim=(-1, -2))
    scale = (amax / QMAX[code]).clamp_min(2.0 ** LOG2_FLOOR)
    inv = 1.0 / scale
    y = (f * inv[..., None, None]).clamp(-QMAX[code], QMAX[code])
    if code == "int8":
        return torch.nan_to_num(y, nan=0.0).round().to(torch.int8), scale
    return y.to(torch.float8_e4m3fn), scale


# ---------------------------------------------------------------- inputs

def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + salt)
    return g


def _vectors(shape, gen, elem, outliers):
    """Normal vectors; keys and values have four channels of eight times the size in each head."""
    x = torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)
    if outliers:
        heads = shape[-2]
        ch = torch.rand((heads, D), generator=gen, device=DEV).argsort(dim=1)[:, :4]
        x *= 1.0 + 7.0 * torch.zeros((heads, D), device=DEV).scatter_(1, ch, 1.0)
    return x.to(elem)


def _pages_for(tokens, block, gen):
    """A page table over shuffled page numbers for requests that end at `tokens`."""
    width = max(1, max(-(-n // block) for n in tokens))
    n = len(tokens) * width
    ids = torch.rand(n + 3, generator=gen, device=DEV).argsort()[:n].to(torch.int32)
    return ids.reshape(len(tokens), width).contiguous(), n + 3


def prepare(case, seed):
    gen = _gen(seed, 1)
    kv, g, elem, op = case["kv"], case["group"], ELEM[case["elem"]], case["op"]
    st = {"case": case}
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    if op == "rotate":
        # the head layout is all that the call takes of a cache
        table, n_pages, block, code, n_slots = torch.zeros((1, 1), dtype=torch.int32, device=DEV), 1, 16, "e4m3", 1
    else:
        block, code, n_slots = case["block"], case["code"], case["n_req"]
        if op == "tree":
            ends = _lens(case)
        else:
            new, before = _appended(case)
            ends = [a + b for a, b in zip(new, before)]
        table, n_pages = _pages_for(ends, block, gen)
    c = block // SUB
    st["pages"] = torch.zeros((n_pages, kv, c, 2, SUB * D), dtype=CODE[code], device=DEV)
    st["scales"] = torch.zeros((n_pages, kv, 2), dtype=torch.float32, device=DEV)
    st["tail"] = torch.zeros((n_slots, kv, c, 2, SUB * D), dtype=elem, device=DEV)
    st["table"] = table
    if op != "rotate":
        # requests lie in slots of another order than the call's
        st["slots"] = torch.rand(n_slots, generator=gen, device=DEV).argsort().to(torch.int32)
        x = _vectors((n_slots, 2, block, kv, D), gen, elem, True).permute(0, 3, 1, 2, 4)
        st["tail"].copy_(_store(x, 16))
    if op in ("rotate", "append"):
        new, before = _appended(case)
        total, r = sum(new), case["rotary"]
        pos, rope_len = _positions(case, seed)
        st["positions"] = torch.from_numpy(pos).to(DEV)
        inv_freq = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
        ang = torch.arange(rope_len, device=DEV, dtype=torch.float64)[:, None] * inv_freq
        st["rope"] = torch.stack((ang.cos(), ang.sin()), dim=-1).float().contiguous()
        st["pair_axis"] = _pair_axis(case)
        st["k"] = _vectors((total, kv, D), gen, elem, True)
        st["k_rot"] = torch.zeros_like(st["k"])
        st["q"] = st["q_rot"] = None
        if case.get("with_q", True):
            st["q"] = _vectors((total, kv * g, D), gen, elem, False)
            st["q_rot"] = torch.zeros_like(st["q"])
    if op == "append":
        st["n_new"], st["before"] = new, i32(before)
        st["v"] = _vectors((total, kv, D), gen, elem, True)
    if op in ("tree", "accept"):
        m = case["nodes_max"]
        st["k"] = _vectors((n_slots * m, kv, D), gen, elem, True)
        st["v"] = _vectors((n_slots * m, kv, D), gen, elem, True)
    if op == "accept":
        # nodes of a path come in rising order, at places that another seed has elsewhere
        r = random.Random(seed * 7919 + case["lens_seed"])
        st["path"] = i32([sorted(r.sample(range(m), min(m, case["path_max"]))) for _ in range(n_slots)])
        st["n_path"], st["before"] = i32(new), i32(before)
    if op == "tree":
        st["q"] = _vectors((n_slots * m, kv * g, D), gen, elem, False)
        st["out"] = torch.zeros_like(st["q"])
        st["lens"], st["n_nodes"], st["parents"] = i32(ends), i32(_nodes(case)), i32(_parents(case, seed))
        # earlier tokens, quantised block by block
        x = _vectors((n_pages, 2, block, kv, D), gen, torch.float32, True).permute(0, 3, 1, 2, 4)
        codes, scale = _quantise(x, code)
        del x
        byte = codes.view(torch.uint8)
        st["pages"].view(torch.uint8).copy_(_store(byte, 8))
        st["scales"].copy_(scale)
    if own:
        # the descriptor of a layer's cache, made once by a user's program
        import differentiated_kv_cache_gb300 as dkv
        st["cache"] = dkv.make_cache8(st["pages"], st["scales"], st["tail"], st["table"], group_size=g,
                                      rotary_dim=case.get("rotary", 0), rotary_interleaved=case.get("interleaved", False),
                                      max_nodes=case["nodes_max"] if op == "tree" else 0)
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        import differentiated_kv_cache_gb300 as dkv
        c = st["case"]
        if op == "tree":
            dkv.dkv_cache8_tree(st["cache"], st["lens"], None if c["chain"] else st["parents"], st["q"], st["k"], st["v"],
                                st["out"], n_nodes=st["n_nodes"], window=c["window"], sinks=c["sinks"], slots=st["slots"])
        elif op == "accept":
            dkv.dkv_cache8_accept(st["cache"], st["before"], st["k"], st["v"], st["path"], n_path=st["n_path"],
                                  slots=st["slots"])
        elif op == "rotate":
            dkv.dkv_cache8_rotate(st["cache"], st["positions"], st["rope"], q=st["q"], k=st["k"], q_rot=st["q_rot"],
                                  k_rot=st["k_rot"], pair_axis=st["pair_axis"])
        else:
            dkv.dkv_cache8_append_at(st["cache"], st["before"], st["positions"], st["k"], st["v"], st["rope"],
                                     pair_axis=st["pair_axis"], n_new=None if c["new_max"] == 1 else st["n_new"],
                                     slots=st["slots"], q=st["q"], k_rot=st["k_rot"], q_rot=st["q_rot"])
    elif op == "tree":
        _plain_tree(st)
    elif op == "accept":
        _plain_accept(st)
    elif op == "rotate":
        _plain_rotate(st)
    else:
        _plain_append(st)
    if op == "tree":
        return {"out": st["out"]}
    if op == "rotate":
        return {"k_rot": st["k_rot"], "q_rot": st["q_rot"]}
    stored = {"pages": st["pages"], "scales": st["scales"], "tail": st["tail"]}
    return stored if op == "accept" else {**stored, "k_rot": st["k_rot"], "q_rot": st["q_rot"]}


def _turned(x, cos_sin, case):
    """x [n, heads, 128] turned by the angles of its pairs [n, rotary/2, 2]; 32 bits, rounded once."""
    r = case["rotary"]
    f = x.float()
    cos, sin = cos_sin[:, None, :, 0], cos_sin[:, None, :, 1]
    a, b = (f[..., 0:r:2], f[..., 1:r:2]) if case["interleaved"] else (f[..., :r // 2], f[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), dim=-1).flatten(-2) if case["interleaved"] else torch.cat((y, z), dim=-1)
    return torch.cat((turned, f[..., r:]), dim=-1).to(x.dtype)


def _plain_rotate(st):
    axis = torch.tensor(st["pair_axis"], device=DEV)
    rows = st["positions"].long()[axis].T                                          # [n][pairs]
    cos_sin = st["rope"][rows, torch.arange(len(axis), device=DEV)]
    st["k_rot"].copy_(_turned(st["k"], cos_sin, st["case"]))
    if st["q"] is not None:
        st["q_rot"].copy_(_turned(st["q"], cos_sin, st["case"]))


def _plain_store(st, k, v, req, nth, new, most):
    """Tokens (rows k, v; the nth of a request's) into the cache; rows past a request's `new` are no tokens."""
    case, t, kv = st["case"], st["case"]["block"], st["case"]["kv"]
    before, slots = st["before"].long(), st["slots"].long()
    n_req = len(new)
    # the touched blocks of every request, the open block's tokens first; a place behind them for rows that are no tokens
    first = before // t
    nb = (t - 1 + most + t - 1) // t
    x = torch.zeros((n_req, nb * t + 1, kv, 2, D), dtype=k.dtype, device=DEV)
    x[:, :t] = _restore(st["tail"][slots], 16).permute(0, 3, 1, 2, 4)
    at = torch.where(nth < new[req], before[req] % t + nth, torch.full_like(nth, nb * t))
    x[req, at, :, 0] = k
    x[req, at, :, 1] = v
    blocks = x[:, :nb * t].reshape(n_req, nb, t, kv, 2, D).permute(0, 1, 3, 4, 2, 5)        # [req][block][kv][2][t][128]
    end = before + new
    i, j = torch.nonzero(first[:, None] + torch.arange(nb, device=DEV) < (end // t)[:, None], as_tuple=True)
    codes, scale = _quantise(blocks[i, j], case["code"])
    page = st["table"][slots[i], first[i] + j].long()
    st["pages"].view(torch.uint8)[page] = _store(codes.view(torch.uint8), 8)
    st["scales"][page] = scale
    # the tokens left in the open block; its other places keep what they held
    kept = torch.where(end // t > first, end % t, before % t + new)
    lo = torch.where(end // t > first, torch.zeros_like(end), before % t)
    place = torch.arange(t, device=DEV)
    mine = ((place >= lo[:, None]) & (place < kept[:, None]))[:, None, None, :, None]
    last = blocks[torch.arange(n_req, device=DEV), (end // t - first).clamp_max(nb - 1)]
    st["tail"][slots] = _store(torch.where(mine, last, _restore(st["tail"][slots], 16)), 16)


def _plain_append(st):
    _plain_rotate(st)
    new = torch.tensor(st["n_new"], device=DEV)
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), new, output_size=sum(st["n_new"]))
    nth = torch.arange(len(req), device=DEV) - (new.cumsum(0) - new)[req]
    _plain_store(st, st["k_rot"], st["v"], req, nth, new, max(st["n_new"]))


def _plain_accept(st):
    n_req, width = st["path"].shape
    req = torch.arange(n_req, device=DEV).repeat_interleave(width)
    nth = torch.arange(width, device=DEV).repeat(n_req)
    row = req * st["case"]["nodes_max"] + st["path"].long().reshape(-1)
    _plain_store(st, st["k"][row], st["v"][row], req, nth, st["n_path"].long(), width)


def _plain_tree(st):
    case, t, kv, g, m = st["case"], st["case"]["block"], st["case"]["kv"], st["case"]["group"], st["case"]["nodes_max"]
    n, slots = st["lens"].long(), st["slots"].long()
    ids = st["table"][slots].long()                                                # [req][width]
    x = _restore(st["pages"].view(torch.uint8)[ids], 8).view(CODE[case["code"]])   # [req][width][kv][2][t][128]
    x = x.float() * st["scales"][ids][..., None, None]
    x = x.permute(0, 2, 3, 1, 4, 5).reshape(len(n), kv, 2, -1, D)
    open_at = n // t * t
    x = torch.cat((x, torch.zeros((len(n), kv, 2, t, D), device=DEV)), dim=3)
    at = (open_at[:, None] + torch.arange(t, device=DEV))[:, None, None, :, None].expand(-1, kv, 2, -1, D)
    x = x.scatter(3, at, _restore(st["tail"][slots], 16).float())
    stored = x.shape[3]
    drafts = torch.stack((st["k"], st["v"]), dim=1).reshape(len(n), m, 2, kv, D).permute(0, 3, 2, 1, 4).float()
    x = torch.cat((x, drafts), dim=3)
    # a node's ancestors and itself: powers of (1 + "is the parent of")
    node = torch.arange(m, device=DEV)
    link = (st["parents"].long()[:, :, None] == node).double() + torch.eye(m, device=DEV, dtype=torch.float64)
    over = torch.linalg.matrix_power(link, m) > 0                                  # [req][node][its ancestors]
    depth = over.sum(dim=-1) - 1
    here = n[:, None] + depth                                                      # positions
    pos = torch.arange(stored, device=DEV)
    see = (pos < n[:, None])[:, None, :].expand(-1, m, -1)
    if case["window"]:
        see = see & ((pos > (here - case["window"])[..., None]) | (pos < case["sinks"]))
        over = over & ((here[:, None, :] > (here - case["window"])[..., None]) | (here < case["sinks"])[:, None, :])
    see = torch.cat((see, over), dim=2)[:, None, :, None, :]                       # [req][1][node][1][key]
    q = st["q"].float().reshape(len(n), m, kv, g, D).transpose(1, 2)
    s = (q.reshape(len(n), kv, m * g, D) @ x[:, :, 0].transpose(-1, -2)).div_(math.sqrt(D))
    s = s.reshape(len(n), kv, m, g, -1).masked_fill_(~see, -math.inf)
    p = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
    v = x[:, :, 1]
    o = (p.reshape(len(n), kv, m * g, -1) @ v).reshape(len(n), kv, m, g, D) / p.sum(dim=-1, keepdim=True)
    o = o.transpose(1, 2).reshape(len(n), m, kv * g, D).to(st["out"].dtype)
    real = (node < st["n_nodes"][:, None])[:, :, None, None]
    st["out"].copy_(torch.where(real, o, st["out"].reshape(o.shape)).reshape(st["out"].shape))


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definition in 64 bits, request by request, from the same inputs."""
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    return {"tree": _exact_tree, "accept": _exact_accept, "rotate": _exact_rotate, "append": _exact_append}[case["op"]](case, st)


def _tile_places(bits):
    """(place of a key value, place of a value entry) for [16 tokens][128 features], from the register layout."""
    i = torch.arange(SUB, device=DEV)[:, None]
    f = torch.arange(D, device=DEV)[None, :]

    def place(row, col, s):
        lane, w = 4 * (row % 8) + col % 8 // 2, 4 * (row // 8) + 2 * (col // 8) + col % 2
        return s // 2 * 512 + lane * 16 + s % 2 * 8 + w if bits == 8 else s * 256 + lane * 8 + w

    return place(i, f % 16, f // 16), place(f % 16, i, f // 16)


def _read(tiles, bits):
    """[n tiles][2][2048] -> keys and values [16 n tokens][128]."""
    pk, pv = _tile_places(bits)
    return tiles[:, 0][:, pk].reshape(-1, D), tiles[:, 1][:, pv].reshape(-1, D)


def _exact_turned(case, st, x):
    y, r = x.double().clone(), case["rotary"]
    table = st["rope"].double()
    for i, a in enumerate(st["pair_axis"]):
        one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
        c, s = (table[st["positions"][a].long(), i, e][:, None] for e in range(2))
        u, w = x[..., one].double(), x[..., two].double()
        y[..., one] = u * c - w * s
        y[..., two] = w * c + u * s
    return y


def _exact_rotate(case, st):
    return {"k_rot": _exact_turned(case, st, st["k"]), "q_rot": _exact_turned(case, st, st["q"])}


def _exact_stored(case, st, keys, values):
    """keys, values: for each request its new tokens [n][kv][128], the keys in 64 bits."""
    kv, t, elem = case["kv"], case["block"], ELEM[case["elem"]]
    bytes_of = st["pages"].view(torch.uint8)
    pk8, pv8 = _tile_places(8)
    pk16, pv16 = _tile_places(16)
    tail = st["tail"].double()
    for i, (k, v) in enumerate(zip(keys, values)):
        slot, b, n = int(st["slots"][i]), int(st["before"][i]), len(k)
        used = b % t
        olds = [_read(st["tail"][slot, h], 16) for h in range(kv)]
        kk = torch.cat((torch.stack([o[0][:used] for o in olds], 1), k.to(elem)))
        vv = torch.cat((torch.stack([o[1][:used] for o in olds], 1), v))
        full = (used + n) // t
        if full:
            both = torch.stack((kk[:full * t], vv[:full * t]), 2).double().reshape(full, t, kv, 2, D)
            scale = (both.abs().amax(dim=(1, 4)) / QMAX[case["code"]]).clamp_min(2.0 ** LOG2_FLOOR)      # [full][kv][2]
            y = both / scale[:, None, :, :, None]
            y = y.round().to(torch.int8) if case["code"] == "int8" else y.clamp(-448, 448).float().to(torch.float8_e4m3fn)
            y = y.view(torch.uint8).reshape(full, t // SUB, SUB, kv, 2, D).permute(0, 3, 1, 4, 2, 5)
            tiles = torch.zeros((full, kv, t // SUB, 2, SUB * D), dtype=torch.uint8, device=DEV)
            tiles[..., 0, :][..., pk8] = y[..., 0, :, :]
            tiles[..., 1, :][..., pv8] = y[..., 1, :, :]
            pages = st["table"][slot, b // t:b // t + full].long()
            bytes_of[pages] = tiles
            st["scales"][pages] = scale.float()
        # what stays in the open block; its earlier tokens lie there already
        whole_k = torch.cat((torch.stack([o[0][:used] for o in olds], 1).double(), k))
        lo = 0 if full else used
        for x in range(lo, used + n - full * t):
            tail[slot, :, x // SUB, 0][:, pk16[x % SUB]] = whole_k[full * t + x]
            tail[slot, :, x // SUB, 1][:, pv16[x % SUB]] = vv[full * t + x].double()
    return {"pages": st["pages"], "scales": st["scales"].double(), "tail": tail}


def _exact_accept(case, st):
    keys, values = [], []
    for i, n in enumerate(_appended(case)[0]):
        rows = i * case["nodes_max"] + st["path"][i, :n].long()
        keys.append(st["k"][rows].double())
        values.append(st["v"][rows])
    return _exact_stored(case, st, keys, values)


def _exact_append(case, st):
    k_rot = _exact_turned(case, st, st["k"])
    q_rot = _exact_turned(case, st, st["q"]) if st["q"] is not None else None
    sizes = _appended(case)[0]
    return {**_exact_stored(case, st, k_rot.split(sizes), st["v"].split(sizes)), "k_rot": k_rot, "q_rot": q_rot}


def _exact_tree(case, st):
    kv, g, t, m = case["kv"], case["group"], case["block"], case["nodes_max"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    parents = st["parents"].tolist()
    for i, (n, nodes) in enumerate(zip(_lens(case), _nodes(case))):
        slot, full = int(st["slots"][i]), n // t
        depth, see = [], torch.zeros((nodes, n + nodes), dtype=torch.bool)
        key = torch.arange(n)
        for x in range(nodes):
            depth.append(0 if parents[i][x] < 0 else depth[parents[i][x]] + 1)
            here = n + depth[x]
            within = lambda p: not case["window"] or p > here - case["window"] or p < case["sinks"]  # noqa: E731
            see[x, :n] = (key > here - case["window"]) | (key < case["sinks"]) if case["window"] else True
            y = x
            while y >= 0:
                see[x, n + y] = within(n + depth[y])
                y = parents[i][y]
        see = see.to(DEV).repeat_interleave(g, 0)
        pages = st["table"][slot, :full].long()
        for h in range(kv):
            k, v = _read(st["tail"][slot, h], 16)
            k, v = k[:n - full * t].double(), v[:n - full * t].double()
            if full:
                ck, cv = _read(st["pages"][pages, h].reshape(-1, 2, SUB * D).view(torch.uint8), 8)
                sc = st["scales"][pages, h].double().repeat_interleave(t, 0)
                ck, cv = (x.contiguous().view(CODE[case["code"]]).double() * sc[:, j:j + 1] for j, x in enumerate((ck, cv)))
                k, v = torch.cat((ck, k)), torch.cat((cv, v))
            rows = slice(i * m, i * m + nodes)
            k, v = torch.cat((k, st["k"][rows, h].double())), torch.cat((v, st["v"][rows, h].double()))
            q = st["q"][rows, h * g:(h + 1) * g].double().reshape(nodes * g, D)
            p = torch.softmax((q @ k.T / math.sqrt(D)).masked_fill(~see, -math.inf), dim=-1)
            out[rows, h * g:(h + 1) * g] = (p @ v).reshape(nodes, g, D)
    return {"out": out}
