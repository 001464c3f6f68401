"""Measured cases of the 8-bit block-scaled cache: append with rotation, decode
attention and prompt attention with a sliding window and first tokens that stay
visible.

Shapes are those of this repository's workloads (32 query / 8 KV heads, 64/8,
40/8, 28/4, head size 128), its prompt and generation lengths, and generic ones.
"""
import math
import random

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

def _append(name, kv, g, n_req, new, before, elem, code, block, rotary=128, inter=False, q=True, seed=1):
    return {"name": name, "op": "append", "kv": kv, "group": g, "n_req": n_req, "new_min": new[0], "new_max": new[1],
            "before_min": before[0], "before_max": before[1], "elem": elem, "code": code, "block": block,
            "rotary": rotary, "interleaved": inter, "with_q": q, "lens_seed": seed}


def _decode(name, kv, g, n_req, lens, elem, code, block, window=0, sinks=0, seed=1):
    return {"name": name, "op": "decode", "kv": kv, "group": g, "n_req": n_req, "len_min": lens[0], "len_max": lens[1],
            "elem": elem, "code": code, "block": block, "window": window, "sinks": sinks, "lens_seed": seed}


def _prompt(name, kv, g, n_req, lens, elem, window, sinks, seed=1):
    return {"name": name, "op": "prompt", "kv": kv, "group": g, "n_req": n_req, "len_min": lens[0], "len_max": lens[1],
            "elem": elem, "window": window, "sinks": sinks, "lens_seed": seed}


def listed():
    return [
        # one user's next token: pure latency
        _append("append_one_token", 8, 4, 1, (1, 1), (4100, 4100), "fp16", "e4m3", 64),
        # a generation step of a full batch, ragged, bf16 with adjacent-pair rotation of half of each head
        _append("append_step_128", 4, 7, 128, (1, 1), (1024, 16384), "bf16", "int8", 32, 64, True, True, 2),
        # pieces of prompts put in between generation steps, odd sizes at odd places
        _append("append_pieces_ragged", 8, 5, 24, (1, 1500), (0, 2000), "bf16", "e4m3", 128, 128, False, True, 3),
        # the prompts of a whole batch
        _append("append_prompts_32x4096", 8, 4, 32, (4096, 4096), (0, 0), "fp16", "e4m3", 64),
        # one user in a short conversation
        _decode("decode_one_short", 8, 4, 1, (300, 300), "fp16", "e4m3", 64),
        # a generation step of the batch above
        _decode("decode_32x4096", 8, 4, 32, (4090, 4170), "fp16", "e4m3", 64),
        # few long contexts, many query heads a KV head
        _decode("decode_8x32768", 8, 8, 8, (32768, 32900), "bf16", "int8", 64),
        # ragged batch, odd group, a window with four first tokens
        _decode("decode_window_128", 4, 7, 128, (1024, 16384), "bf16", "e4m3", 32, 4096, 4, 4),
        # many short requests: most of what is read is the open block
        _decode("decode_short_200", 8, 5, 200, (1, 160), "fp16", "int8", 128, 0, 0, 5),
        # short ragged prompts
        _prompt("prompt_short_ragged", 8, 4, 12, (17, 700), "fp16", 256, 4, 6),
        # the prompts of a whole batch, streaming
        _prompt("prompt_32x4096_w1024", 8, 4, 32, (4096, 4096), "fp16", 1024, 4),
        # one long prompt with a wide window
        _prompt("prompt_16384_w4096", 8, 8, 1, (16384, 16384), "bf16", 4096, 64),
    ]


def _spread(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "decode", "prompt"))
    kv, g = rng.choice(((8, 4), (8, 8), (8, 5), (4, 7), (2, 4), (1, 8), (4, 1), (3, 6), (5, 3), (2, 2)))
    elem, code = rng.choice(("fp16", "bf16")), rng.choice(("e4m3", "int8"))
    block, seed = rng.choice((16, 32, 64, 128)), rng.randrange(1 << 20)
    if op == "append":
        n_req = _spread(rng, 1, 128)
        most = max(1, min(8192, 60000 // n_req))
        hi = rng.choice((1, _spread(rng, 1, most)))
        c = _append("", kv, g, n_req, (max(1, hi // rng.choice((1, 2, 9))), hi), (0, _spread(rng, 1, 6000)), elem, code,
                    block, rng.choice((128, 128, 64, 32, 16, 0)), rng.random() < 0.5, rng.random() < 0.7, seed)
    elif op == "decode":
        n_req = _spread(rng, 1, 200)
        hi = _spread(rng, 1, max(1, min(60000, 1000000 // (n_req * kv))))
        window = rng.choice((0, 0, _spread(rng, 1, 8000)))
        c = _decode("", kv, g, n_req, (max(1, hi // rng.choice((1, 3, 20))), hi), elem, code, block, window,
                    rng.choice((0, 1, 4, 37, 200)) if window else 0, seed)
    else:
        n_req = _spread(rng, 1, 32)
        hi = _spread(rng, 1, max(1, min(9000, 24000 // n_req)))
        window = rng.choice((0, _spread(rng, 1, 5000), _spread(rng, 1, 5000)))
        if window == 0:
            hi = min(hi, 4500)
        c = _prompt("", kv, g, n_req, (max(1, hi // rng.choice((1, 2, 9))), hi), elem, window,
                    rng.choice((0, 1, 4, 37, 200)) if window else 0, seed)
    del c["name"]
    return c


def _numbers(case, lo, hi, salt):
    r = random.Random(case["lens_seed"] * 1000003 + salt)
    return [r.randint(lo, hi) for _ in range(case["n_req"])]


def _lens(case):
    return _numbers(case, case["len_min"], case["len_max"], 1)


def _appended(case):
    return _numbers(case, case["new_min"], case["new_max"], 1), _numbers(case, case["before_min"], case["before_max"], 2)


def _visible(n, window, sinks):
    """Tokens that the query at position n - 1 sees."""
    if window <= 0 or window >= n:
        return n
    return window + min(sinks, n - window)


def _visible_sum(n, window, sinks):
    """Sum of _visible over the n positions of a prompt."""
    if window <= 0 or window >= n:
        return n * (n + 1) // 2
    rest = n - window
    s = min(sinks, rest)
    return window * (window + 1) // 2 + rest * window + s * (s + 1) // 2 + (rest - s) * s


def work(case):
    kv, g = case["kv"], case["group"]
    if case["op"] == "append":
        new, before = _appended(case)
        total, t = sum(new), case["block"]
        nbytes = total * kv * D * 2 * 2                                      # k and v read
        nbytes += total * kv * D * 2 if case["rotary"] else 0               # rotated k
        nbytes += 2 * total * kv * g * D * 2 if case["with_q"] else 0       # q read, rotated q
        if case["rotary"]:
            rows = set()
            for n, b in zip(new, before):
                rows.update(range(b, b + n))
            nbytes += len(rows) * case["rotary"] * 4
        for n, b in zip(new, before):
            blocks = (b + n) // t - b // t
            nbytes += blocks * kv * (t * 2 * D + 8)                          # codes and scales
            nbytes += (b % t) * kv * D * 4 if blocks else 0                  # tokens already in the open block
            nbytes += ((b + n) % t if blocks else n) * kv * D * 4            # tokens left in it
        vecs = total * kv * (1 + (g if case["with_q"] else 0))
        return {"bytes": nbytes, "flops": 3 * vecs * case["rotary"] + 4 * total * kv * D}
    lens = _lens(case)
    if case["op"] == "decode":
        t, nbytes, keys = case["block"], 0, 0
        for n in lens:
            see = _visible(n, case["window"], case["sinks"])
            in_tail = min(see, n % t)
            nbytes += kv * ((see - in_tail) * 2 * D + in_tail * 4 * D + -(-(see - in_tail) // t) * 8)
            keys += see
        nbytes += 2 * len(lens) * kv * g * D * 2
        return {"bytes": nbytes, "flops": 4 * D * kv * g * keys}
    total = sum(lens)
    return {"bytes": total * D * 2 * (2 * kv * g + 2 * kv),
            "flops": 4 * D * kv * g * sum(_visible_sum(n, case["window"], case["sinks"]) for n in lens)}


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
    kv, g, elem = case["kv"], case["group"], ELEM[case["elem"]]
    st = {"case": case}
    if case["op"] == "prompt":
        lens = _lens(case)
        n = sum(lens)
        st["lens"] = lens
        st["q"] = _vectors((n, kv * g, D), gen, elem, False)
        st["k"] = _vectors((n, kv, D), gen, elem, True)
        st["v"] = _vectors((n, kv, D), gen, elem, True)
        st["out"] = torch.zeros((n, kv * g, D), dtype=elem, device=DEV)
        table, n_pages, block, code, n_slots = torch.zeros((1, 1), dtype=torch.int32, device=DEV), 1, 16, "e4m3", 1
    else:
        block, code, n_slots = case["block"], case["code"], case["n_req"]
        if case["op"] == "append":
            new, before = _appended(case)
            ends = [a + b for a, b in zip(new, before)]
        else:
            ends = _lens(case)
        table, n_pages = _pages_for(ends, block, gen)
    c = block // SUB
    st["pages"] = torch.zeros((n_pages, kv, c, 2, SUB * D), dtype=CODE[code], device=DEV)
    st["scales"] = torch.zeros((n_pages, kv, 2), dtype=torch.float32, device=DEV)
    st["tail"] = torch.zeros((n_slots, kv, c, 2, SUB * D), dtype=elem, device=DEV)
    st["table"] = table
    if case["op"] != "prompt":
        # requests lie in slots of another order than the call's
        st["slots"] = torch.rand(n_slots, generator=gen, device=DEV).argsort().to(torch.int32)
        x = _vectors((n_slots, 2, block, kv, D), gen, elem, True).permute(0, 3, 1, 2, 4)
        st["tail"].copy_(_store(x, 16))
    if case["op"] == "append":
        total = sum(new)
        st["n_new"] = new
        st["before"] = torch.tensor(before, dtype=torch.int32, device=DEV)
        st["k"] = _vectors((total, kv, D), gen, elem, True)
        st["v"] = _vectors((total, kv, D), gen, elem, True)
        st["rope"] = st["k_rot"] = st["q"] = st["q_rot"] = None
        r = case["rotary"]
        if r:
            inv_freq = 10000.0 ** (-torch.arange(0, r, 2, device=DEV, dtype=torch.float64) / r)
            # another seed stands at another place of a longer text
            ang = (torch.arange(max(ends), device=DEV, dtype=torch.float64) + seed % 1000)[:, None] * inv_freq
            st["rope"] = torch.stack((ang.cos(), ang.sin()), dim=-1).float().contiguous()
            st["k_rot"] = torch.zeros_like(st["k"])
        if case["with_q"]:
            st["q"] = _vectors((total, kv * g, D), gen, elem, False)
            st["q_rot"] = torch.zeros_like(st["q"])
    if case["op"] == "decode":
        st["q"] = _vectors((n_slots, kv * g, D), gen, elem, False)
        st["out"] = torch.zeros((n_slots, kv * g, D), dtype=elem, device=DEV)
        st["lens"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
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
                                      rotary_dim=case.get("rotary", 0), rotary_interleaved=case.get("interleaved", False))
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        import differentiated_kv_cache_gb300 as dkv
        c = st["case"]
        if op == "append":
            dkv.dkv_cache8_append(st["cache"], st["before"], st["k"], st["v"], rope=st["rope"],
                                  n_new=None if c["new_max"] == 1 else st["n_new"], slots=st["slots"], q=st["q"],
                                  k_rot=st["k_rot"], q_rot=st["q_rot"])
        elif op == "decode":
            dkv.dkv_cache8_attention(st["cache"], st["lens"], st["q"], st["out"], window=c["window"], sinks=c["sinks"],
                                     slots=st["slots"])
        else:
            dkv.dkv_cache8_prefill(st["cache"], st["lens"], st["q"], st["k"], st["v"], st["out"], window=c["window"],
                                   sinks=c["sinks"])
    elif op == "append":
        _plain_append(st)
    elif op == "decode":
        _plain_decode(st)
    else:
        _plain_prompt(st)
    if op == "append":
        return {"pages": st["pages"], "scales": st["scales"], "tail": st["tail"], "k_rot": st["k_rot"], "q_rot": st["q_rot"]}
    return {"out": st["out"]}


def _rotate(x, rows, case):
    """x [n, heads, 128] turned by the angles of its rows [n, rotary/2, 2]; 32 bits, rounded once."""
    r = case["rotary"]
    if not r:
        return x
    f = x.float()
    cos, sin = rows[:, None, :, 0], rows[:, None, :, 1]
    a, b = (f[..., 0:r:2], f[..., 1:r:2]) if case["interleaved"] else (f[..., :r // 2], f[..., r // 2:r])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((y, z), dim=-1).flatten(-2) if case["interleaved"] else torch.cat((y, z), dim=-1)
    return torch.cat((turned, f[..., r:]), dim=-1).to(x.dtype)


def _plain_append(st):
    case, t, kv = st["case"], st["case"]["block"], st["case"]["kv"]
    new = torch.tensor(st["n_new"], device=DEV)
    before, slots = st["before"].long(), st["slots"].long()
    req = torch.repeat_interleave(torch.arange(len(new), device=DEV), new, output_size=sum(st["n_new"]))
    pos = before[req] + torch.arange(len(req), device=DEV) - (new.cumsum(0) - new)[req]
    rows = st["rope"][pos] if st["rope"] is not None else None
    k = _rotate(st["k"], rows, case)
    if st["k_rot"] is not None:
        st["k_rot"].copy_(k)
    if st["q"] is not None:
        st["q_rot"].copy_(_rotate(st["q"], rows, case))
    # the touched blocks of every request, the open block's tokens first
    first = before // t
    nb = max((b % t + n + t - 1) // t for n, b in zip(st["n_new"], _appended(case)[1]))
    x = torch.zeros((len(new), nb * t, kv, 2, D), dtype=k.dtype, device=DEV)
    x[:, :t] = _restore(st["tail"][slots], 16).permute(0, 3, 1, 2, 4)
    at = pos - first[req] * t
    x[req, at, :, 0] = k
    x[req, at, :, 1] = st["v"]
    blocks = x.reshape(len(new), nb, t, kv, 2, D).permute(0, 1, 3, 4, 2, 5)        # [req][block][kv][2][t][128]
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
    last = blocks[torch.arange(len(new), device=DEV), (end // t - first).clamp_max(nb - 1)]
    st["tail"][slots] = _store(torch.where(mine, last, _restore(st["tail"][slots], 16)), 16)


def _plain_decode(st):
    case, t, kv, g = st["case"], st["case"]["block"], st["case"]["kv"], st["case"]["group"]
    n, slots = st["lens"].long(), st["slots"].long()
    ids = st["table"][slots].long()                                                # [req][width]
    x = _restore(st["pages"].view(torch.uint8)[ids], 8).view(CODE[case["code"]])   # [req][width][kv][2][t][128]
    x = x.float() * st["scales"][ids][..., None, None]
    x = x.permute(0, 2, 3, 1, 4, 5).reshape(len(n), kv, 2, -1, D)
    place = torch.arange(t, device=DEV)
    open_at = n // t * t
    x = torch.cat((x, torch.zeros((len(n), kv, 2, t, D), device=DEV)), dim=3)
    at = (open_at[:, None] + place)[:, None, None, :, None].expand(-1, kv, 2, -1, D)
    x = x.scatter(3, at, _restore(st["tail"][slots], 16).float())
    pos = torch.arange(x.shape[3], device=DEV)
    see = pos < n[:, None]
    if case["window"]:
        see &= (pos >= (n - case["window"])[:, None]) | (pos < case["sinks"])
    q = st["q"].float().reshape(len(n), kv, g, D)
    s = (q @ x[:, :, 0].transpose(-1, -2) / math.sqrt(D)).masked_fill(~see[:, None, None, :], -math.inf)
    p = (s - s.amax(dim=-1, keepdim=True)).exp()
    v = x[:, :, 1].masked_fill(~see[:, None, :, None], 0.0)
    st["out"].copy_((p @ v / p.sum(dim=-1, keepdim=True)).reshape(len(n), kv * g, D))


def _plain_prompt(st):
    """Query blocks of 128 tokens against the keys of the window before them and the first tokens."""
    case, kv, g = st["case"], st["case"]["kv"], st["case"]["group"]
    lens = torch.tensor(st["lens"], device=DEV)
    most, b = max(st["lens"]), 128
    w = case["window"] if 0 < case["window"] < most else most
    nq, back = -(-most // b), -(-(w - 1) // b) * b
    req = torch.repeat_interleave(torch.arange(len(lens), device=DEV), lens, output_size=sum(st["lens"]))
    pos = torch.arange(len(req), device=DEV) - (lens.cumsum(0) - lens)[req]

    def padded(x, front):
        y = torch.zeros((len(lens), x.shape[1], front + nq * b, D), device=DEV)
        y[req, :, front + pos] = x.float()
        return y

    q = padded(st["q"], 0).reshape(len(lens), kv, g, nq, b, D).transpose(2, 3).reshape(len(lens), kv, nq, g * b, D)
    k, v = padded(st["k"], back), padded(st["v"], back)
    first = min(case["sinks"], most) if case["window"] else 0
    row = torch.arange(nq * b, device=DEV).reshape(nq, b, 1)
    key = (torch.arange(nq, device=DEV) * b - back)[:, None, None] + torch.arange(back + b, device=DEV)
    see = (key <= row) & (key > row - w) & (key >= 0)
    early = torch.arange(first, device=DEV)
    see = torch.cat((see, (early <= row - w).expand(nq, b, first)), dim=2).repeat(1, g, 1)
    s = torch.cat((q @ k.unfold(2, back + b, b), q @ k[:, :, None, back:back + first].transpose(-1, -2)), dim=-1)
    s = s.div_(math.sqrt(D)).masked_fill_(~see, -math.inf)
    p = s.sub_(s.amax(dim=-1, keepdim=True)).exp_()
    o = p[..., :back + b] @ v.unfold(2, back + b, b).transpose(-1, -2) + p[..., back + b:] @ v[:, :, None, back:back + first]
    o = o / p.sum(dim=-1, keepdim=True)
    o = o.reshape(len(lens), kv, nq, g, b, D).permute(0, 2, 4, 1, 3, 5).reshape(len(lens), nq * b, kv * g, D)
    st["out"].copy_(o[req, pos])


# ---------------------------------------------------------------- 64 bits

def exact(case, seed):
    """The definition in 64 bits, request by request, from the same inputs."""
    global own
    was, own = own, False
    st = prepare(case, seed)
    own = was
    return {"append": _exact_append, "decode": _exact_decode, "prompt": _exact_prompt}[case["op"]](case, st)


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


def _exact_append(case, st):
    kv, t, r = case["kv"], case["block"], case["rotary"]
    elem = ELEM[case["elem"]]
    new, before = _appended(case)

    def turn(x, p):
        y = x.double().clone()
        if r:
            ang = st["rope"].double()[p]
            c, s = ang[:, None, :, 0], ang[:, None, :, 1]
            one = torch.arange(0, r, 2, device=DEV) if case["interleaved"] else torch.arange(r // 2, device=DEV)
            two = one + (1 if case["interleaved"] else r // 2)
            y[..., one] = x.double()[..., one] * c - x.double()[..., two] * s
            y[..., two] = x.double()[..., two] * c + x.double()[..., one] * s
        return y

    bytes_of = st["pages"].view(torch.uint8)
    pk8, pv8 = _tile_places(8)
    pk16, pv16 = _tile_places(16)
    krot = torch.zeros(st["k"].shape, dtype=torch.float64, device=DEV)
    qrot = torch.zeros(st["q"].shape, dtype=torch.float64, device=DEV) if st["q"] is not None else None
    tail = st["tail"].double()
    at = 0
    for i, (n, b) in enumerate(zip(new, before)):
        slot = int(st["slots"][i])
        p = torch.arange(b, b + n, device=DEV)
        k = turn(st["k"][at:at + n], p)
        v = st["v"][at:at + n]
        krot[at:at + n] = k
        if qrot is not None:
            qrot[at:at + n] = turn(st["q"][at:at + n], p)
        at += n
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
    return {"pages": st["pages"], "scales": st["scales"].double(), "tail": tail,
            "k_rot": krot if st["k_rot"] is not None else None, "q_rot": qrot}


def _exact_decode(case, st):
    kv, g, t = case["kv"], case["group"], case["block"]
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    for i, n in enumerate(_lens(case)):
        slot, full = int(st["slots"][i]), n // t
        seen = torch.arange(n, device=DEV)
        seen = seen[(seen < case["sinks"]) | (seen >= n - case["window"])] if case["window"] else seen
        pages = st["table"][slot, :full].long()
        for h in range(kv):
            k, v = _read(st["tail"][slot, h], 16)
            if full:
                ck, cv = _read(st["pages"][pages, h].reshape(-1, 2, SUB * D).view(torch.uint8), 8)
                sc = st["scales"][pages, h].double().repeat_interleave(t, 0)
                ck, cv = (x.contiguous().view(CODE[case["code"]]).double() * sc[:, j:j + 1] for j, x in enumerate((ck, cv)))
                k, v = torch.cat((ck, k.double())), torch.cat((cv, v.double()))
            p = torch.softmax(st["q"][i, h * g:(h + 1) * g].double() @ k.double()[seen].T / math.sqrt(D), dim=-1)
            out[i, h * g:(h + 1) * g] = p @ v.double()[seen]
    return {"out": out}


def _exact_prompt(case, st):
    kv, g, step = case["kv"], case["group"], 1024
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device=DEV)
    if work(case)["flops"] > 8e12:
        return None
    at = 0
    for n in st["lens"]:
        k, v = (st[x][at:at + n].double().transpose(0, 1) for x in ("k", "v"))
        for a in range(0, n, step):
            rows = torch.arange(a, min(n, a + step), device=DEV)
            keys = torch.arange(0, int(rows[-1]) + 1, device=DEV)
            if case["window"]:
                keys = keys[(keys < case["sinks"]) | (keys > a - case["window"])]
            see = keys <= rows[:, None]
            if case["window"]:
                see &= (keys > rows[:, None] - case["window"]) | (keys < case["sinks"])
            q = st["q"][at + a:at + a + len(rows)].double().reshape(len(rows), kv, g, D).permute(1, 2, 0, 3)
            s = (q @ k[:, keys].transpose(-1, -2)[:, None] / math.sqrt(D)).masked_fill(~see, -math.inf)
            o = torch.softmax(s, dim=-1) @ v[:, keys][:, None]
            out[at + a:at + a + len(rows)] = o.permute(2, 0, 1, 3).reshape(len(rows), kv * g, D)
        at += n
    return {"out": out}
