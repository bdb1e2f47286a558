"""fp64 oracle of speculative decoding over the bf16 paged cache: append with rotation, tree attention, accept.

Written from the definitions in include/jfa.h, with plain loops over sequences, tokens and
heads; nothing here is shared with the kernels. Caches are float arrays [num_pages, P, Hkv, d].
"""
from __future__ import annotations

import numpy as np


def rotate(x, cos, sin, interleaved=False):
    """One token's heads [H, d] turned by one row of the tables (rot_dim / 2 pairs)."""
    half = len(cos)
    y = np.array(x, dtype=np.float64)
    for j in range(half):
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        y[:, a] = x[:, a] * cos[j] - x[:, b] * sin[j]
        y[:, b] = x[:, b] * cos[j] + x[:, a] * sin[j]
    return y


def cell(table_row, P, t):
    return int(table_row[t // P]), t % P


def append_rope(q, k, v, kc, vc, table, seqlens, offsets, cos, sin, positions=None, interleaved=False):
    """jfa_cache_append_rope, in place on kc and vc. Returns the rotated q (None without q)."""
    P = kc.shape[1]
    out = None if q is None else np.full(q.shape, np.nan)
    for b in range(len(seqlens)):
        n = int(offsets[b + 1] - offsets[b])
        for i in range(n):
            row, t = int(offsets[b]) + i, int(seqlens[b]) - n + i
            p = t if positions is None else int(positions[row])
            c, s = ([], []) if cos is None else (cos[p], sin[p])
            at = cell(table[b], P, t)
            kc[at] = rotate(k[row], c, s, interleaved)
            vc[at] = v[row]
            if q is not None:
                out[row] = rotate(q[row], c, s, interleaved)
    return out


def gather(c, table_row, L):
    """Rows of positions 0..L-1 of one sequence: [L, Hkv, d]."""
    P = c.shape[1]
    return np.stack([c[cell(table_row, P, t)] for t in range(L)]) if L else np.zeros((0,) + c.shape[2:])


def visible(L, n, mask=None):
    """[n, L] truth values: what each of the last n tokens sees; mask: their words, None for a chain."""
    see = np.ones((n, L), dtype=bool)
    for i in range(n):
        for j in range(n):
            see[i, L - n + j] = j <= i if mask is None else bool((int(mask[i]) >> j) & 1)
    return see


def decode_tree(q, kc, vc, table, seqlens, offsets, scale, mask=None):
    """jfa_decode_tree. Returns O, LSE and, per row, sum_j P_j |v_j| and max_j sum_d |q_d k_jd| * scale
    over what it sees, from which errors are bounded. Rows of no sequence are NaN."""
    total, Hq, d = q.shape
    G = Hq // kc.shape[2]
    O, absO = np.full(q.shape, np.nan), np.zeros(q.shape)
    LSE, size = np.full((total, Hq), np.nan), np.zeros((total, Hq))
    for b in range(len(seqlens)):
        o0, n, L = int(offsets[b]), int(offsets[b + 1] - offsets[b]), int(seqlens[b])
        if n == 0:
            continue
        K, V = gather(kc, table[b], L), gather(vc, table[b], L)
        see = visible(L, n, None if mask is None else mask[o0:o0 + n])
        for i in range(n):
            O[o0 + i], LSE[o0 + i] = 0.0, -np.inf
            if not see[i].any():
                continue
            for h in range(Hq):
                Kh, Vh = K[see[i], h // G], V[see[i], h // G]
                s = scale * (Kh @ q[o0 + i, h])
                m = np.max(s)
                p = np.exp(s - m)
                z = p.sum()
                p /= z
                O[o0 + i, h] = p @ Vh
                absO[o0 + i, h] = p @ np.abs(Vh)
                size[o0 + i, h] = scale * np.max(np.abs(Kh) @ np.abs(q[o0 + i, h]))
                LSE[o0 + i, h] = m + np.log(z)
    return O, LSE, absO, size


def accept(kc, vc, table, seqlens, offsets, accepted, counts):
    """jfa_cache_accept, in place. Returns the new lengths."""
    P = kc.shape[1]
    lens = np.zeros(len(seqlens), dtype=np.int32)
    for b in range(len(seqlens)):
        C = int(seqlens[b]) - int(offsets[b + 1] - offsets[b])
        n = int(counts[b])
        for c in (kc, vc):
            rows = [c[cell(table[b], P, C + int(accepted[b][k]))].copy() for k in range(n)]
            for k in range(n):
                c[cell(table[b], P, C + k)] = rows[k]
        lens[b] = C + n
    return lens
