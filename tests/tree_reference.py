"""A tree's verification in plain 64-bit numpy, from include/pld.h: the
reference of its tests. No code is shared with the library, and none with
target_reference.py but the rotation."""

from __future__ import annotations

import math

import numpy as np

import target_reference as R


def branch(parent, t):
    """Nodes from t up to the root, t first; parent[s - 1] is node s's."""
    up = [t]
    while up[-1]:
        up.append(int(parent[up[-1] - 1]))
    return up


def normed(x, weight, eps):
    """x [heads, dim] over its root mean square; also the magnitude that the
    rounding errors of a norm scale with."""
    if weight is None:
        return x.copy()
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * weight


def attend(q, kc, vc, table, lengths, dlen, parent, page, scale, window, ks=None, vs=None):
    """As target_reference.attend, for trees: parent [b, rows - 1]."""
    b, rows, hq, dim = q.shape
    hk = kc.shape[1]
    g = hq // hk
    out, lse = np.full(q.shape, np.nan), np.full((b, rows, hq), np.nan)
    mass, span = np.full(q.shape, np.nan), np.full((b, rows, hq), np.nan)
    for i in range(b):
        n = R.block_rows(lengths[i], dlen[i])
        if n == 0:
            continue
        L = lengths[i]
        ids = table[i, :-(-(L - 1 + n) // page)]
        k = kc[ids].transpose(1, 0, 2, 3).reshape(hk, -1, dim)
        v = vc[ids].transpose(1, 0, 3, 2).reshape(hk, -1, dim)
        for t in range(n):
            up = branch(parent[i], t)
            at = L - 1 + len(up) - 1
            cells = [j for j in range(L - 1) if not window or j > at - window]
            cells += [L - 1 + s for k_, s in reversed(list(enumerate(up)))
                      if not window or k_ < window]
            for h in range(hq):
                kh = k[h // g][cells] * (1.0 if ks is None else ks[h // g])
                vh = v[h // g][cells] * (1.0 if vs is None else vs[h // g])
                s = scale * (kh @ q[i, t, h])
                m = s.max()
                e = np.exp(s - m)
                out[i, t, h] = (e / e.sum()) @ vh
                lse[i, t, h] = m + math.log(e.sum())
                mass[i, t, h] = (e / e.sum()) @ np.abs(vh)
                span[i, t, h] = abs(scale) * (np.abs(kh) @ np.abs(q[i, t, h])).max()
    return out, lse, mass, span


def verify_one(z, x, parent, d, temperature, u, u_draw):
    """One request: logits z [rows, vocab], tokens x and parents of nodes 1..d,
    uniforms u of theirs. Tokens, path, log probabilities."""
    tokens, path, logp, v = [], [0], [], 0
    while True:
        w = z[v] / (temperature if temperature > 0 else 1.0)
        lp = w - w.max()
        lp = lp - math.log(np.exp(lp).sum())
        p, best, on = np.exp(lp), int(np.argmax(z[v])), None
        for c in range(v + 1, d + 1):
            if parent[c - 1] != v:
                continue
            y = int(x[c - 1])
            take = y == best if temperature == 0 else float(u[c - 1]) * p.sum() < p[y]
            if take:
                on = c
                break
            if temperature > 0:
                p[y] = 0.0
        if on is None:
            break
        tokens.append(y)
        logp.append(lp[y])
        path.append(on)
        v = on
    if temperature == 0:
        pick = best
    else:
        c = np.cumsum(p)
        live = np.nonzero(p > 0)[0]
        over = live[c[live] > float(u_draw) * c[-1]]
        pick = int(over[0]) if over.size else int(live[-1])
    return tokens + [pick], path, logp + [lp[pick]]


def keep(kc, vc, table, lengths, path, accepted, page):
    """The caches [layers, pages, heads, ...] after the moves."""
    k, v = kc.copy(), vc.copy()
    for b, (L, a) in enumerate(zip(lengths, accepted)):
        for i in range(1, a + 1):
            src, dst = L - 1 + path[b][i], L - 1 + i
            x, y = table[b, src // page], table[b, dst // page]
            k[:, y, :, dst % page] = kc[:, x, :, src % page]
            v[:, y, :, :, dst % page] = vc[:, x, :, :, src % page]
    return k, v


def random_tree(rng, d, kids=4, on=0.5):
    """Parents of d nodes: a chain that goes on with probability `on`, else a
    branch off any node with fewer than `kids` children."""
    parent, count = [], [0] * (d + 1)
    for t in range(1, d + 1):
        p = t - 1
        if rng.random() >= on:
            p = int(rng.integers(0, t))
            while count[p] >= kids:
                p = int(rng.integers(0, t))
        count[p] += 1
        parent.append(p)
    return parent


def shapes(d):
    """Trees of d nodes that are not like random ones."""
    return {"chain": list(range(d)), "star": [0] * d,
            "comb": [0 if t == 1 else (t - 2 if t % 2 else t - 1) for t in range(1, d + 1)],
            "binary": [(t - 1) // 2 for t in range(1, d + 1)]}
