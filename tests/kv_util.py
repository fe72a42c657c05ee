"""Plain 64-bit forms of the paged cache and its attention, and their inputs.

Everything here is numpy on the host, written from the definitions in
include/qgemv.h and sharing no code with the library: quantisation by searching
the nearest value in a table of every code, attention as a softmax over the
positions that a token sees.
"""
from __future__ import annotations

import numpy as np

import oracle as O

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)) for e in range(16) for m in range(8)])
E4M3[127] = np.nan


def nearest(x, grid):
    """Index of the value of the ascending grid nearest to |x| (ties to the even index, saturating)."""
    a = np.minimum(np.abs(x), grid[-1])
    hi = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo = hi - 1
    down, up = a - grid[lo], grid[hi] - a
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x, fmt, g):
    """(codes, scales) of x [..., D] (float64 values of bf16). The quotients
    are 32-bit numbers by definition (a 64-bit quotient of 32-bit numbers
    rounded to 32 bits is the 32-bit quotient)."""
    if fmt == "bf16":
        return O.bf16_bits(x), None
    with np.errstate(all="ignore"):
        y = (x / np.float64(np.float32(g))).astype(np.float32).astype(np.float64)
        sign = np.signbit(y).astype(np.int64)
        if fmt == "fp8":
            top = np.max(np.where(np.isnan(y), 0.0, np.abs(y)), -1)
            s = np.full(top.shape, 22)
            for b in range(21, 0, -1):
                s = np.where(top <= 448.0 * 2.0 ** (b - 15), b, s)
            r = y * 2.0 ** (15.0 - s)[..., None]
            code = nearest(np.nan_to_num(r, nan=0.0, posinf=1e9, neginf=-1e9), E4M3[:127]) + 128 * sign
            code = np.where(np.isnan(r), 127, code)
            return code.astype(np.uint8), s.astype(np.uint8)
        blocks = y.reshape(y.shape[:-1] + (y.shape[-1] // 16, 16))
        top = np.max(np.abs(blocks), -1)                           # NaN stays
        q = (top / 6.0).astype(np.float32).astype(np.float64)
        scale = np.where(np.isnan(q), 127, nearest(np.nan_to_num(q, nan=0.0, posinf=1e9), E4M3[:127]))
        f = np.where(scale == 127, 0.0, E4M3[np.minimum(scale, 126)])[..., None]
        r = np.where(f > 0, (blocks / np.where(f > 0, f, 1.0)).astype(np.float32).astype(np.float64), 0.0)
        code = nearest(np.nan_to_num(r, nan=0.0, posinf=1e9, neginf=-1e9), E2M1) + 8 * np.where(f > 0, np.signbit(r), 0)
        code = code.reshape(y.shape).astype(np.uint8)
        return code[..., 0::2] | (code[..., 1::2] << 4), scale.astype(np.uint8)


def values(codes, scales, fmt, g):
    """The 64-bit values of stored codes [..., row]."""
    if fmt == "bf16":
        return O.bf16_array(codes)
    g = np.float64(np.float32(g))
    if fmt == "fp8":
        v = np.where(codes & 128, -1.0, 1.0) * E4M3[codes & 127]
        return v * 2.0 ** (scales.astype(np.float64) - 15)[..., None] * g
    pair = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[:-1] + (2 * codes.shape[-1],))
    v = np.where(pair & 8, -1.0, 1.0) * E2M1[pair & 7]
    sc = np.where(scales & 128, -1.0, 1.0) * E4M3[scales & 127]
    return v * np.repeat(sc, 16, -1) * g


def attention(q, k, v, seen, scale):
    """(out, lse, a, ds) of one sequence: q [T][Hq][D], k, v [L][Hkv][D],
    seen [T][L]; for the error bounds a = (sum p |v|, sum |v|) per output and
    ds = sum |q k| scale, the largest over the keys a row sees."""
    T, Hq, D = q.shape
    H = k.shape[1]
    G = Hq // H
    out, a = np.zeros((T, Hq, D)), np.zeros((2, T, Hq, D))
    lse, ds = np.full((T, Hq), -np.inf), np.zeros((T, Hq))
    for t in range(T):
        keys = np.nonzero(seen[t])[0]
        if not len(keys):
            continue
        for h in range(Hq):
            kk, vv = k[keys, h // G], v[keys, h // G]
            s = (kk @ q[t, h]) * scale
            m = s.max()
            w = np.exp(s - m)
            total = w.sum()
            lse[t, h] = m + np.log(total)
            out[t, h] = (w @ vv) / total
            a[0, t, h] = (w @ np.abs(vv)) / total
            a[1, t, h] = np.abs(vv).sum(0)
            ds[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
    return out, lse, a, ds


def attention_bounds(a, ds, lse, n_keys, D, fmt):
    """Error bounds of (out before its bf16 rounding, lse).

    A score sums D products in fp32; a tensor core may truncate, each addition
    off by up to 2^-22 of the partial sums' largest magnitude, at most ds:
    |ds| (D + 8) 2^-22, and 2^-22 |s| more for the scaling to base 2 and the
    exponential's argument (|s| <= ds). A weight is therefore off by a factor
    within e^(+-e_s), and by half a step of its 16-bit type when it enters the
    second product (f16 2^-11; bf16 2^-8), plus 2^-21 for the exponential
    itself. Sums of n weights: n 2^-22 relative. The same relative error is in
    the sum that divides, but for the 16-bit rounding. Below f16's normal
    range half a step is 2^-25, whatever the weight: weights are held times
    2^7 or more of the row's largest (its maximum is kept within 2^8 above),
    so the sum of weights is at least 2^7 and a weight is off by up to 2^-32 of
    it there: 2^-32 sum |v| in all. bf16 has the range of 32-bit numbers.
    """
    e_s = ds * (D + 10) * 2.0 ** -22
    rel = 2 * (e_s + 2.0 ** -21 + n_keys * 2.0 ** -22) + 2.0 ** (-8 if fmt == "bf16" else -11)
    with np.errstate(invalid="ignore"):
        b_lse = e_s + 2.0 ** -20 + n_keys * 2.0 ** -22 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0.0)
    low = 0.0 if fmt == "bf16" else 2.0 ** -32
    return a[0] * rel[..., None] + a[1] * low + 1e-30, b_lse


def ancestor_masks(r, counts):
    """64-bit masks of random trees: each draft sees its ancestors and itself."""
    out = []
    for t in counts:
        m = []
        for i in range(t):
            m.append((m[int(r.integers(max(0, i - 4), i))] if i else 0) | (1 << i))
        out += m
    return np.array(out, dtype=np.uint64).view(np.int64)


class Paged:
    """A host copy of a paged cache of quantised normal values, with the
    sequences' page tables (pages anywhere in the pool, unused table entries
    out of range, unused slots NaN where the format has one)."""

    def __init__(self, seed, fmt, dim, page, heads, lens, counts, kg=1.0, vg=1.0, extra_pages=3, std=1.0):
        r = np.random.default_rng(seed)
        self.fmt, self.dim, self.page, self.heads, self.g = fmt, dim, page, heads, (kg, vg)
        self.lens, self.counts = list(lens), list(counts)
        need = [(n + t + page - 1) // page for n, t in zip(lens, counts)]
        self.max_pages = max(need + [1]) + 1
        ids = r.permutation(sum(need) + extra_pages)
        self.pages = len(ids)
        self.table = np.full((len(lens), self.max_pages), -7, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.start = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
        self.total = int(self.start[-1])
        shape = (self.pages, heads, page, dim)
        self.parts = []
        used = np.zeros((self.pages, page), bool)
        for b in range(len(lens)):
            for p in range(lens[b] + counts[b]):
                used[self.table[b, p // page], p % page] = True
        for g in self.g:
            x = O.round_bf16(r.standard_normal(shape) * std)
            codes, scales = quantise(x, fmt, g)
            hole = ~used[:, None, :, None] & np.ones(codes.shape, bool)
            if fmt == "bf16":
                codes[hole] = 0x7FC0
            elif fmt == "fp8":
                codes[hole] = 0x7F
            else:
                scales[~used[:, None, :, None] & np.ones(scales.shape, bool)] = 0x7F
            self.parts.append([codes, scales])

    def at(self, b, first, n):
        p = np.arange(first, first + n)
        return self.table[b, p // self.page], p % self.page

    def stored(self, kv, b, first, n):
        """Values of positions first .. first + n of sequence b: [n][heads][dim]."""
        pg, off = self.at(b, first, n)
        codes, scales = self.parts[kv]
        return values(codes[pg, :, off], None if scales is None else scales[pg, :, off], self.fmt, self.g[kv])

    def device(self, torch, q):
        """(KVCache, KVBatch) over copies on the device."""
        t = []
        for codes, scales in self.parts:
            c = torch.from_numpy(codes.view(np.int16)).cuda().view(torch.bfloat16) if self.fmt == "bf16" else \
                torch.from_numpy(codes).cuda()
            t.append((c, None if scales is None else torch.from_numpy(scales).cuda()))
        cache = q.KVCache(self.fmt, t[0][0], t[1][0], t[0][1], t[1][1], *self.g)
        return cache, self.batch(torch, q)

    def batch(self, torch, q, n_tokens=None):
        return q.KVBatch(torch.from_numpy(self.table).cuda(),
                         torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                         torch.from_numpy(self.start).cuda(), self.total if n_tokens is None else n_tokens)

    def host_part(self, cache, kv):
        """(codes, scales) of a device cache as numpy arrays."""
        import torch
        c = cache.v if kv else cache.k
        s = cache.v_scales if kv else cache.k_scales
        c = c.view(torch.int16).cpu().numpy().view(np.uint16) if self.fmt == "bf16" else c.cpu().numpy()
        return c, None if s is None else s.cpu().numpy()
