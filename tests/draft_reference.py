"""Decoding with a tree of drafted tokens, from its definition, in 64 bits, sequence by sequence, on the CPU."""
from __future__ import annotations

import math

import numpy as np

import cache_reference as R


def line(tree, i):
    """Node i and the nodes above it, itself first.  An entry that is no earlier row counts as -1."""
    got = [i]
    while 0 <= tree[got[-1]] < got[-1]:
        got.append(tree[got[-1]])
    return got


def visible(tree, L, rows, window=0):
    """[rows, L]: the slots that each node sees."""
    see = np.zeros((rows, L), bool)
    base = L - rows
    for i in range(rows):
        if base + i < 0:
            continue
        up = line(tree, i)
        at = base + len(up) - 1  # its position
        for j in range(max(base, 0)):
            see[i, j] = not window or j > at - window
        for d, a in enumerate(up):
            if base + a >= 0 and (not window or d < window):
                see[i, base + a] = True
    return see


def attention(c, q, table, lens, trees, n_q=None, scale=None, window=0, softcap=0.0, hidden=()):
    """o, lse, weights, and what tolerances need: as cache_reference.attention.  hidden: slots that nobody sees."""
    q = q.double().numpy()
    B, Hq, n, D = q.shape
    H = c.pool["k"].shape[1]
    scale = float(np.float32(1.0 / math.sqrt(D) if scale is None else scale))
    o, a = np.zeros((B, Hq, n, D)), np.zeros((B, Hq, n, D))
    lse, w = np.full((B, Hq, n), -np.inf), np.zeros((B, H, max(1, max(lens))))
    sabs = np.zeros(B)
    for b in range(B):
        L, rows = lens[b], n if n_q is None else n_q[b]
        if L == 0 or rows == 0:
            continue
        pages = np.asarray(table[b][:-(-L // c.page)], int)
        see = visible(trees[b], L, rows, window)
        see[:, list(hidden)] = False
        some = see.any(1)
        for h in range(Hq):
            k, v = c.tokens("k", pages, h // (Hq // H), L), c.tokens("v", pages, h // (Hq // H), L)
            s = q[b, h, :rows] @ k.T * scale
            sabs[b] = max(sabs[b], (np.abs(q[b, h, :rows]) @ np.abs(k).T * abs(scale)).max())
            if softcap:
                s = softcap * np.tanh(s / softcap)
            s = np.where(see, s, -np.inf)
            m = np.where(some, s.max(1), 0.0)[:, None]
            p = np.exp(s - m)
            l = p.sum(1, keepdims=True)
            p = np.where(l > 0, p / np.where(l > 0, l, 1.0), 0.0)
            lse[b, h, :rows][some] = (m[:, 0] + np.log(np.where(l[:, 0] > 0, l[:, 0], 1.0)))[some]
            o[b, h, :rows], a[b, h, :rows] = p @ v, p @ np.abs(v)
            w[b, h // (Hq // H), :L] += p.sum(0)
    return o, lse, w, a, sabs


def prob(x):
    """What is no positive finite number counts as 0."""
    x = np.asarray(x, np.float64)
    return np.where((x > 0) & np.isfinite(x), x, 0.0)


def residuals(p, q, tokens):
    """What is left of p behind each of the children `tokens`, rejected in turn: [(r, Z)], the first before any."""
    r, z = prob(p), 1.0
    got = [(r, z)]
    for t in tokens:
        if q is None:
            there = 0 <= t < len(r)
            z = z - (r[t] if there else 0.0)
            r = r.copy()
            if there:
                r[t] = 0.0
        else:
            r = np.maximum(r - z * prob(q), 0.0)
            z = r.sum()
        got.append((r, z))
    return got


def verify(p, tokens, tree, u, u_next, q=None, nodes=None):
    """One sequence: (path, token).  p, q: [n, V]; lists otherwise."""
    nodes = len(tokens) if nodes is None else nodes
    if nodes == 0:
        return [], -1
    V = p.shape[1]
    path = [0]
    while True:
        c = path[-1]
        children = [i for i in range(c + 1, nodes) if tree[i] == c]
        left = residuals(p[c], None if q is None else q[c], [tokens[i] for i in children])
        for i, (r, z) in zip(children, left):
            t = tokens[i]
            if not 0 <= t < V:
                continue
            if float(u[i]) * (1.0 if q is None else float(prob(q[c][t]))) * z < r[t]:
                path.append(i)
                break
        else:
            r = left[-1][0]
            break
    if not r.sum() > 0:
        r = prob(p[c])
    upto = np.cumsum(r)
    if not upto[-1] > 0:
        return path, 0
    x = float(u_next)
    x = min(x, 1.0) if x > 0 else 0.0
    hit = np.nonzero(upto > x * upto[-1])[0]
    return path, int(hit[0]) if len(hit) else int(np.nonzero(r)[0][-1])


def accept(c, table, lens, path, count, n_q, weights=None):
    """Changes c and weights ([B, H, W] numpy); returns the new lengths."""
    out = []
    for b, L in enumerate(lens):
        base = L - n_q[b]
        line = path[b][:count[b]]
        out.append(base + count[b])
        slots = list(range(base)) + [base + a for a in line]  # whose token ends in slot j
        if weights is not None:
            weights[b, :, base:base + count[b]] = weights[b][:, [base + a for a in line]]
        for name in ("k", "v"):
            pool, scale = c.pool[name].copy(), c.scale[name].copy()
            for m in range(base // c.page, -(-len(slots) // c.page)):
                part = slots[m * c.page:(m + 1) * c.page]
                if part == list(range(m * c.page, m * c.page + len(part))):
                    continue
                at = table[b][m]
                for h in range(pool.shape[1]):
                    blocks = [table[b][j // c.page] for j in part]
                    top = max(scale[x, h] for x in blocks)
                    for t, (j, x) in enumerate(zip(part, blocks)):
                        val = pool[x, h, j % c.page]
                        if scale[x, h] != top:
                            ratio = np.float32(np.float32(scale[x, h]) / np.float32(top))
                            val = R.round8((val.astype(np.float32) * ratio).astype(np.float64), c.kind)
                        c.pool[name][at, h, t] = val
                    c.scale[name][at, h] = top
    return out


def random_tree(rng, n, shape):
    """n parents.  rng: random.Random."""
    if shape == "chain":
        return [i - 1 for i in range(n)]
    if shape == "star":
        return [-1] + [0] * (n - 1)
    if shape == "forest":
        return [-1] + [-1 if rng.random() < 0.3 else rng.randrange(i) for i in range(1, n)]
    return [-1] + [rng.randrange(max(0, i - 6), i) for i in range(1, n)]
