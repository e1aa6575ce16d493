"""The serving operators over an 8-bit cache from their definition, in 64 bits, sequence by sequence, on the CPU; and
the random caches that the tests run them on."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3, I8 = torch.float8_e4m3fn, torch.int8
MAX = {E4M3: 448.0, I8: 127.0}


def round8(x, kind):
    """float64 -> the stored values (as float64): nearest even on the type's grid, saturating, NaN kept or 0."""
    x = np.clip(np.asarray(x, np.float64), -MAX[kind], MAX[kind])
    if kind == I8:
        return np.rint(np.nan_to_num(x, nan=0.0))
    step = np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6))) - 3)
    return np.rint(x / step) * step


def pow2_scale(amax, kind):
    """The least 2^e >= 2^-100 with amax <= MAX * 2^e."""
    e = -100
    while amax > MAX[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def stored(t):
    return t.double().numpy()


class Cache:
    """k, v as stored values [P, H, page, D] and their scales [P, H], all float64 numpy."""

    def __init__(self, k, v, k_scale, v_scale):
        self.kind = k.dtype
        self.pool = {"k": stored(k), "v": stored(v)}
        self.scale = {"k": k_scale.double().numpy().copy(), "v": v_scale.double().numpy().copy()}
        self.page = k.shape[2]

    def tokens(self, name, pages, h, n):
        x = self.pool[name][pages, h] * self.scale[name][pages, h][:, None, None]
        return x.reshape(-1, x.shape[-1])[:n]


def append(c, new, table, lens, n_new):
    """new: {"k": [B, H, n, D], "v": ...} torch CPU tensors.  Changes c."""
    for name, x in new.items():
        x = x.double().numpy()
        for b in range(x.shape[0]):
            for h in range(x.shape[1]):
                t = 0
                while t < n_new[b]:
                    pos = lens[b] + t
                    at, slot = table[b][pos // c.page], pos % c.page
                    m = min(c.page - slot, n_new[b] - t)
                    val = x[b, h, t:t + m]
                    s = pow2_scale(np.max(np.abs(val[np.isfinite(val)]), initial=0.0), c.kind)
                    pool, scale = c.pool[name][at, h], c.scale[name]
                    if slot:
                        s = max(s, scale[at, h])
                        pool[:slot] = round8(pool[:slot] * (scale[at, h] / s), c.kind)
                    pool[slot:slot + m] = round8(val / s, c.kind)
                    scale[at, h] = s
                    t += m


def attention(c, q, table, lens, n_q=None, scale=None, causal=True, window=0, softcap=0.0):
    """o, lse, weights [B, H, max len], and what tolerances need: sum of p |v| per output, the largest sum of
    |scale q k| per sequence.  q: torch CPU tensor."""
    q = q.double().numpy()
    B, Hq, n, D = q.shape
    H = c.pool["k"].shape[1]
    G = Hq // H
    scale = float(np.float32(1.0 / math.sqrt(D) if scale is None else scale))
    o, a = np.zeros((B, Hq, n, D)), np.zeros((B, Hq, n, D))
    lse, w = np.full((B, Hq, n), -np.inf), np.zeros((B, H, max(1, max(lens))))
    sabs = np.zeros(B)
    for b in range(B):
        L, rows = lens[b], n if n_q is None else n_q[b]
        pages = np.asarray(table[b][:-(-L // c.page)], int)
        for h in range(Hq):
            if L == 0 or rows == 0:
                continue
            k, v = c.tokens("k", pages, h // G, L), c.tokens("v", pages, h // G, L)
            s = q[b, h, :rows] @ k.T * scale
            sabs[b] = max(sabs[b], (np.abs(q[b, h, :rows]) @ np.abs(k).T * abs(scale)).max())
            if softcap:
                s = softcap * np.tanh(s / softcap)
            i, j = (L - rows + np.arange(rows))[:, None], np.arange(L)[None]
            if causal:
                s = np.where(j <= i, s, -np.inf)
            if window:
                s = np.where(j > i - window, s, -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isfinite(m), m, 0.0))
            l = p.sum(1, keepdims=True)
            some = l[:, 0] > 0
            p = np.where(l > 0, p / np.where(l > 0, l, 1.0), 0.0)
            lse[b, h, :rows][some] = (m[:, 0] + np.log(np.where(l[:, 0] > 0, l[:, 0], 1.0)))[some]
            o[b, h, :rows], a[b, h, :rows] = p @ v, p @ np.abs(v)
            w[b, h // G, :L] += p.sum(0)
    return o, lse, w, a, sabs


def evict(c, table, lens, weights, positions, keep, recent, into=None):
    """Changes c (the blocks of `into`, or in place).  weights [B, H, W] float32 and positions numpy, changed in place
    without `into`; returns (lens, {(b, h): [slot that ends in slot j]})."""
    B, H, W = weights.shape
    old = {n: (c.pool[n].copy(), c.scale[n].copy()) for n in c.pool}
    w0, p0 = weights.copy(), None if positions is None else positions.copy()
    src = {}
    for b in range(B):
        n = lens[b]
        for h in range(H):
            pos = np.arange(W) if p0 is None else p0[b, h]
            latest = max((int(x) for x in pos[:n]), default=0)

            def rank(j):
                x = float(w0[b, h, j])
                x = -math.inf if math.isnan(x) else x
                if recent and int(pos[j]) > latest - recent:
                    x = math.inf
                return (-x, j)

            kept = sorted(sorted(range(n), key=rank)[:keep])
            if into is not None:
                src[b, h] = kept
                to = into
            else:
                stay = [j for j in kept if j < keep]
                movers = [j for j in kept if j >= keep]
                got = {j: j for j in stay}
                holes = [j for j in range(min(n, keep)) if j not in got]
                got.update(zip(holes, movers))
                src[b, h] = [got[j] for j in range(min(n, keep))]
                to = table
            s = src[b, h]
            for name, (pool, scale) in old.items():
                for m in range(0, len(s), c.page):
                    part = s[m:m + c.page]
                    if into is None and part == list(range(m, m + len(part))):
                        continue
                    at = to[b][m // c.page]
                    blocks = [table[b][j // c.page] for j in part]
                    top = max(scale[x, h] for x in blocks)
                    for t, (j, x) in enumerate(zip(part, blocks)):
                        ratio = float(np.float32(scale[x, h] / top)) if top else math.nan
                        val = pool[x, h, j % c.page]
                        if scale[x, h] != top:
                            val = round8((val.astype(np.float32) * np.float32(ratio)).astype(np.float64), c.kind)
                        c.pool[name][at, h, t] = val
                    c.scale[name][at, h] = top
            if into is None:
                for j, x in enumerate(s):
                    weights[b, h, j] = w0[b, h, x]
                    positions[b, h, j] = p0[b, h, x]
    return [min(n, keep) for n in lens], src


# ----------------------------------------------------------------- random caches

def make_pools(g, P, H, page, D, kind, nan_outside=True):
    """Stored values of every size, scales from 2^-9 to 2^-5 (1.5 times that for some: scales need not be powers)."""
    def one():
        x = torch.randn(P, H, page, D, generator=g) * (100.0 if kind == E4M3 else 40.0)
        x = x.clamp(-MAX[kind], MAX[kind])
        return (x.round() if kind == I8 else x).to(kind)

    def scale():
        s = torch.randint(-9, -4, (P, H), generator=g).float().exp2()
        return torch.where(torch.rand(P, H, generator=g) < 0.3, s * 1.5, s)
    return one(), one(), scale(), scale()


def make_table(g, total, page, spare=2, width=None):
    """Pages in random order, -1 where a sequence needs none; returns (rows of ints, number of pages)."""
    need = [-(-t // page) for t in total]
    P = sum(need) + spare
    order = torch.randperm(P, generator=g).tolist()
    width = max(1, max(need)) if width is None else width
    return [[order.pop() for _ in range(k)] + [-1] * (width - k) for k in need], P, order


def spoil(pool, table, lens, page):
    """Bytes behind every sequence's tokens, and blocks that nobody holds, become NaN (e4m3) or -128."""
    bad = torch.full_like(pool.view(torch.uint8), 0x7F if pool.dtype == E4M3 else 0x80)
    raw = pool.view(torch.uint8)
    for row, n in zip(table, lens):
        for m in range(-(-n // page)):
            k = min(page, n - m * page)
            bad[row[m], :, :k] = raw[row[m], :, :k]
    raw.copy_(bad)
