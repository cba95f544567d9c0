"""The verify step's operators in plain 64-bit numpy, from include/pld.h: the
reference of the GPU tests. No code is shared with the library. Each function
also returns what a tolerance needs (sums of magnitudes)."""

from __future__ import annotations

import math

import numpy as np


def block_rows(length: int, dlen: int) -> int:
    return 0 if length == 0 or dlen == -1 else 1 + dlen


def rope_frequencies(rot_dim, scaling="plain", base=10000.0, factor=1.0, original_len=32768,
                     beta_fast=32.0, beta_slow=1.0):
    """Radians per position of each pair."""
    out = []
    for i in range(rot_dim // 2):
        f = base ** (-2.0 * i / rot_dim)
        if scaling == "linear":
            f = f / factor
        elif scaling == "banded":
            # the (real) pair index that turns beta times in original_len
            def pair(beta):
                return rot_dim * math.log(original_len / (2.0 * math.pi * beta)) / (
                    2.0 * math.log(base))
            lo = max(0, math.floor(pair(beta_fast)))
            hi = min(rot_dim - 1, math.ceil(pair(beta_slow)))
            slow = (i - lo) / max(hi - lo, 0.001)
            slow = min(1.0, max(0.0, slow))
            f = f / factor * slow + f * (1.0 - slow)
        out.append(f)
    return np.array(out)


def rotate(x, p, freq, rot_dim, interleaved, magnitude):
    """x [heads, dim] at position p; also the magnitudes that its rounding
    error scales with."""
    y, size = x.copy(), np.zeros_like(x)
    for i in range(rot_dim // 2):
        j, k = (2 * i, 2 * i + 1) if interleaved else (i, i + rot_dim // 2)
        c, s = math.cos(p * freq[i]), math.sin(p * freq[i])
        y[:, j] = magnitude * (x[:, j] * c - x[:, k] * s)
        y[:, k] = magnitude * (x[:, j] * s + x[:, k] * c)
        size[:, j] = size[:, k] = magnitude * (np.abs(x[:, j]) + np.abs(x[:, k]))
    return y, size


def attend(q, kc, vc, table, lengths, dlen, page, scale, window, ks=None, vs=None):
    """q [b, rows, hq, dim]; caches as pld.h lays them out. Returns out, lse,
    the sum of probability times |v|, and the largest sum of |q k| * scale of
    a row's scores; rows without a block hold NaN."""
    b, rows, hq, dim = q.shape
    hk = kc.shape[1]
    g = hq // hk
    out = np.full(q.shape, np.nan)
    lse = np.full((b, rows, hq), np.nan)
    mass = np.full(q.shape, np.nan)
    span = np.full((b, rows, hq), np.nan)
    for i in range(b):
        n = block_rows(lengths[i], dlen[i])
        if n == 0:
            continue
        end = lengths[i] - 1 + n
        ids = table[i, :-(-end // page)]
        k = kc[ids].transpose(1, 0, 2, 3).reshape(hk, -1, dim)[:, :end]
        v = vc[ids].transpose(1, 0, 3, 2).reshape(hk, -1, dim)[:, :end]
        for h in range(hq):
            kh = k[h // g] * (1.0 if ks is None else ks[h // g])
            vh = v[h // g] * (1.0 if vs is None else vs[h // g])
            for t in range(n):
                p = lengths[i] - 1 + t
                lo = max(0, p - window + 1) if window else 0
                s = scale * (kh[lo:p + 1] @ q[i, t, h])
                m = s.max()
                e = np.exp(s - m)
                out[i, t, h] = (e / e.sum()) @ vh[lo:p + 1]
                lse[i, t, h] = m + math.log(e.sum())
                mass[i, t, h] = (e / e.sum()) @ np.abs(vh[lo:p + 1])
                span[i, t, h] = abs(scale) * (np.abs(kh[lo:p + 1]) @ np.abs(q[i, t, h])).max()
    return out, lse, mass, span


def verify_one(z, x, d, claimed, probs, temperature, u, u_draw):
    """One request: z [rows, vocab], draft x, draft length d, claimed[t] True
    where position t has drafter probabilities probs[t]. Returns the tokens
    (accepted, then drawn) and their log probabilities."""
    tokens, logp = [], []
    for t in range(d + 1):
        w = z[t] / (temperature if temperature > 0 else 1.0)
        lp = w - w.max()
        lp = lp - math.log(np.exp(lp).sum())
        p = np.exp(lp)
        if t < d:
            if temperature == 0:
                take = x[t] == int(np.argmax(z[t]))
            else:
                take = float(u[t]) * (float(probs[t][x[t]]) if claimed[t] else 1.0) < p[x[t]]
            if take:
                tokens.append(int(x[t]))
                logp.append(lp[x[t]])
                continue
        if temperature == 0:
            pick = int(np.argmax(z[t]))
        else:
            r = p.copy()
            if t < d and claimed[t]:
                left = np.maximum(p - probs[t], 0.0)
                r = left if left.sum() > 0 else p
            elif t < d:
                r[x[t]] = 0.0
            c = np.cumsum(r)
            live = np.nonzero(r > 0)[0]
            over = live[c[live] > float(u_draw) * c[-1]]
            pick = int(over[0]) if over.size else int(live[-1])
        tokens.append(pick)
        logp.append(lp[pick])
        break
    return tokens, logp
