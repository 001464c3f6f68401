"""Plain reference of the uniform 8-bit cache: the stored state bit by bit
(numpy, fp32 with every operation rounded) and attention in 64 bits, from the
definitions in include/dkv.h."""
from __future__ import annotations

import numpy as np
import torch

SUB, D = 16, 128
QMAX = {torch.float8_e4m3fn: np.float32(448.0), torch.int8: np.float32(127.0)}


def tile_places(bits):
    """Places of K and of V entries of a tile, each [16 tokens][128 features]."""
    i, f = np.meshgrid(np.arange(SUB), np.arange(D), indexing="ij")
    out = []
    for r, c, m in ((i, f % 16, f // 16), (f % 16, i, f // 16)):
        lane, w = 4 * (r % 8) + (c % 8) // 2, 4 * (r // 8) + 2 * (c // 8) + c % 2
        out.append((m // 2) * 512 + 16 * lane + 8 * (m % 2) + w if bits == 8 else 256 * m + 8 * lane + w)
    return out


PLACES = {8: tile_places(8), 16: tile_places(16)}


def to_tiles(x, bits):
    """[2][T][128] -> [T/16][2][2048]"""
    t = x.shape[1]
    out = np.zeros((t // SUB, 2, SUB * D), x.dtype)
    for s in range(t // SUB):
        for o in range(2):
            out[s, o, PLACES[bits][o]] = x[o, s * SUB:(s + 1) * SUB]
    return out


def from_tiles(x, bits):
    """[T/16][2][2048] -> [2][T][128]"""
    return np.stack([np.concatenate([x[s, o][PLACES[bits][o]] for s in range(x.shape[0])]) for o in range(2)])


def elem_np(t):
    """16-bit tensor -> exact float32 array."""
    return t.detach().cpu().float().numpy()


def round_elem(x, dtype):
    """float32 array rounded to the 16-bit type, as float32."""
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dtype).float().numpy()


def rotate(x, pos, rope, rotary_dim, interleaved, dtype):
    """x [n][heads][128] float32 (exact 16-bit values) at positions pos."""
    if not rotary_dim:
        return x
    y = x.copy()
    half = rotary_dim // 2
    cos, sin = (rope[pos][:, None, :, e].astype(np.float32) for e in range(2))
    one = np.arange(0, rotary_dim, 2) if interleaved else np.arange(half)
    two = one + (1 if interleaved else half)
    a, b = x[..., one], x[..., two]
    y[..., one] = a * cos - b * sin
    y[..., two] = b * cos + a * sin
    return round_elem(y, dtype)


def quantise(x, code):
    """One operand's block [T][128] float32 -> (code bytes, scale)."""
    fin = np.where(np.isfinite(x), np.abs(x), np.float32(0))
    s = np.float32(max(np.float32(fin.max()) * (np.float32(1) / QMAX[code]), np.float32(2.0 ** -100)))
    inv = np.float32(1.0) / s
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.clip(x * inv, -QMAX[code], QMAX[code])
    if code == torch.int8:
        c = np.where(np.isnan(y), 0, np.rint(y)).astype(np.int8)
        return c.view(np.uint8), s
    return torch.from_numpy(y).to(code).view(torch.uint8).numpy(), s


class RefCache:
    """Every token of every slot as exact 16-bit values; the state that a cache
    must hold follows from them."""

    def __init__(self, pages, scales, tail, table, rotary_dim=0, interleaved=False):
        self.code, self.elem = pages.dtype, tail.dtype
        self.pages = pages.view(torch.uint8).cpu().numpy().copy()
        self.scales, self.tail = scales.cpu().numpy().copy(), elem_np(tail).copy()
        self.table, self.rot, self.inter = table.cpu().numpy(), rotary_dim, interleaved
        self.hkv, self.T = self.pages.shape[1], self.pages.shape[2] * SUB
        self.tok = {}            # slot -> [n][hkv][2][128]

    def append(self, slot, before, k, v, rope=None):
        """k, v [n][hkv][128] float32 -> the turned keys."""
        n = k.shape[0]
        k = rotate(k, np.arange(before, before + n), rope, self.rot, self.inter, self.elem)
        old = self.tok.get(slot, np.zeros((0, self.hkv, 2, D), np.float32))
        assert len(old) >= before
        now = np.concatenate([old[:before], np.stack([k, v], 2)])
        self.tok[slot] = now
        T = self.T
        for b in range(before // T, (before + n - 1) // T + 1):
            lo, hi = max(before - b * T, 0), min(before + n - b * T, T)
            for h in range(self.hkv):
                x = now[b * T:(b + 1) * T, h].transpose(1, 0, 2)
                if hi == T:
                    page = self.table[slot, b]
                    codes = [quantise(x[o], self.code) for o in range(2)]
                    self.pages[page, h] = to_tiles(np.stack([c[0] for c in codes]), 8)
                    self.scales[page, h] = [c[1] for c in codes]
                else:
                    t = from_tiles(self.tail[slot, h], 16)
                    t[:, lo:hi] = x[:, lo:hi]
                    self.tail[slot, h] = to_tiles(t, 16)
        return k

    def values(self, slot, n, h):
        """Stored K and V [n][128] in 64 bits."""
        out = np.zeros((2, n, D))
        full = n // self.T
        for b in range(full):
            p = self.table[slot, b]
            c = from_tiles(self.pages[p, h], 8)
            c = c.view(np.int8).astype(np.float64) if self.code == torch.int8 else \
                torch.from_numpy(c.copy()).view(self.code).double().numpy()
            out[:, b * self.T:(b + 1) * self.T] = c * self.scales[p, h].astype(np.float64)[:, None, None]
        out[:, full * self.T:] = from_tiles(self.tail[slot, h], 16)[:, :n - full * self.T]
        return out

    def check(self, pages, scales, tail):
        """The GPU's state, bit for bit (NaN codes and values where the reference has them)."""
        got = pages.view(torch.uint8).cpu().numpy()
        if self.code == torch.float8_e4m3fn:
            nan = (self.pages & 0x7f) == 0x7f
            assert ((got & 0x7f) == 0x7f)[nan].all()
            assert (got == self.pages)[~nan].all(), "codes"
        else:
            assert (got == self.pages).all(), "codes"
        assert np.array_equal(scales.cpu().numpy(), self.scales), "scales"
        assert np.array_equal(elem_np(tail), self.tail, equal_nan=True), "tail"


def visible(n, window, sinks):
    j = np.arange(n)
    return j[(j >= n - window) | (j < sinks)] if window else j


def attend(q, k, v):
    """q [G][128], k, v [n][128] in 64 bits -> (out, sum p |v|, largest sum |q k| / sqrt(128), largest |v|)."""
    if not len(k):
        z = np.zeros((q.shape[0], D))
        return z, z, 0.0, 0.0
    s = q @ k.T / np.sqrt(D)
    p = np.exp(s - s.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    return p @ v, p @ np.abs(v), float((np.abs(q) @ np.abs(k).T).max() / np.sqrt(D)), float(np.abs(v).max())


def tolerance(ref, pv, qk, vmax, n, elem, p_eps):
    """Bound of |out - ref|: weights rounded to a relative p_eps (and, where they
    are under 2^-14 of the largest, off by at most 2^-24 of it), logits off by
    at most 128 half steps of fp32 of sum |q k| / sqrt(128) (a tensor-core sum of
    128 products, truncating: a whole step, 2^-23) in every one of the two
    sums, 2^-21 for the exponentials, and half a step of the output's type."""
    eps = torch.finfo(elem).eps / 2
    d = p_eps + 2 * 128 * 2.0 ** -23 * qk + 2.0 ** -21
    return eps * np.abs(ref) * (1 + d) + d * pv + n * 2.0 ** -24 * vmax + torch.finfo(elem).tiny
