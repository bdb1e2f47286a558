"""fp64 oracle of the 8-bit paged KV cache: append, decode with attention weights, evict.

Written from the definitions in include/jfa.h, with plain loops over sequences,
heads and blocks; nothing here is shared with the kernels. Caches are numpy
arrays: codes uint8 [num_pages, P, Hkv, d], scales float [num_pages, P / block, Hkv].
"""
from __future__ import annotations

import numpy as np

from oracle.attention import e4m3_decode

E4M3 = e4m3_decode(np.arange(127, dtype=np.uint8))  # the 127 non-negative finite values, ascending


def e4m3_encode(x):
    """Nearest e4m3 codes (ties to the even code) of float64 values up to 448 in magnitude; NaN -> 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(E4M3, a), 1, 126)
    lo = hi - 1
    up = (a - E4M3[lo] > E4M3[hi] - a) | ((a - E4M3[lo] == E4M3[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo) | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def block_scale(amax):
    """The smallest power of two >= 2^-126 with amax / scale <= 448."""
    s = 2.0 ** -126
    while amax > 448.0 * s:
        s *= 2.0
    return s


def append(k, v, kc, vc, ks, vs, table, seqlens, offsets, weights=None):
    """jfa_cache_append_fp8, in place on the numpy arrays."""
    P, block = kc.shape[1], kc.shape[1] // ks.shape[1]
    for x, c, sc in ((k, kc, ks), (v, vc, vs)):
        x = np.where(np.isfinite(x), x, np.nan)
        for b in range(len(seqlens)):
            L, n = int(seqlens[b]), int(offsets[b + 1] - offsets[b])
            f = L - n
            for start in range(f // block * block, L, block):
                pos = np.arange(max(start, f), min(start + block, L))
                if not len(pos):
                    continue
                old = np.arange(start, max(start, f))
                page, cell = int(table[b][start // P]), start % P // block
                for h in range(x.shape[1]):
                    new = x[offsets[b] + pos - f, h]
                    s = block_scale(np.max(np.abs(new), initial=0.0, where=~np.isnan(new)))
                    if len(old):
                        was = float(sc[page, cell, h])
                        s = max(s, was)
                        if s > was:
                            c[page, old % P, h] = e4m3_encode(e4m3_decode(c[page, old % P, h]) * was / s)
                    sc[page, cell, h] = s
                    c[page, pos % P, h] = e4m3_encode(new / s)
    if weights is not None:
        for b in range(len(seqlens)):
            n = int(offsets[b + 1] - offsets[b])
            weights[b, :, int(seqlens[b]) - n:int(seqlens[b])] = 0


def gather(c, sc, row, L):
    """Values of positions 0..L-1 of one sequence: float64 [L, Hkv, d]."""
    P, block = c.shape[1], c.shape[1] // sc.shape[1]
    t = np.arange(L)
    page = np.asarray(row)[t // P].astype(np.int64)
    return e4m3_decode(c[page, t % P]) * sc[page, t % P // block].astype(np.float64)[..., None]


def decode(q, kc, vc, ks, vs, table, seqlens, scale, weights=None, decay=1.0):
    """jfa_decode_fp8. Returns O, LSE, the new weights (a list of [Hkv, L] per sequence) and, per
    output row, sum_j P_j |v_j|, max_j sum_d |q_d k_jd| * scale and keys * max_j P_j * (scale of
    v_j's block), from which errors are bounded."""
    B, ql, Hq, d = q.shape
    Hkv = kc.shape[2]
    G = Hq // Hkv
    O = np.zeros((B, ql, Hq, d))
    absO = np.zeros((B, ql, Hq, d))
    size = np.zeros((B, ql, Hq))
    top = np.zeros((B, ql, Hq))
    P, block = vc.shape[1], vc.shape[1] // vs.shape[1]
    LSE = np.full((B, ql, Hq), -np.inf)
    W = []
    for b in range(B):
        L = int(seqlens[b])
        K, V = gather(kc, ks, table[b], L), gather(vc, vs, table[b], L)
        w = np.zeros((Hkv, L))
        t = np.arange(L)
        vscale = vs[np.asarray(table[b])[t // P].astype(np.int64), t % P // block].astype(np.float64)
        for i in range(ql):
            see = max(0, L - ql + i + 1)
            if not see:
                continue
            for h in range(Hq):
                Kh, Vh = K[:see, h // G], V[:see, h // G]
                s = scale * (Kh @ q[b, i, h])
                m = np.max(s)
                p = np.exp(s - m)
                z = p.sum()
                p /= z
                O[b, i, h] = p @ Vh
                absO[b, i, h] = p @ np.abs(Vh)
                size[b, i, h] = scale * np.max(np.abs(Kh) @ np.abs(q[b, i, h]))
                top[b, i, h] = see * np.max(p * vscale[:see, h // G])
                LSE[b, i, h] = m + np.log(z)
                w[h // G, :see] += p
        if weights is not None:
            w = w + decay * weights[b, :, :L].astype(np.float64)
        W.append(w)
    return O, LSE, W, absO, size, top


def evict(kc, vc, ks, vs, table, seqlens, weights, keep, new_table, first=0, recent=0):
    """jfa_cache_evict_fp8, in place on the numpy arrays. Returns kept, new_seqlens, new_weights."""
    B, Hkv, _ = weights.shape
    P, block = kc.shape[1], kc.shape[1] // ks.shape[1]
    kept = np.full((B, Hkv, keep), -1, dtype=np.int32)
    lens = np.minimum(np.asarray(seqlens), keep).astype(np.int32)
    new_w = np.zeros((B, Hkv, np.asarray(new_table).shape[1] * P), dtype=np.float32)
    for b in range(B):
        L, n = int(seqlens[b]), int(lens[b])
        values = [gather(c, sc, table[b], L) for c, sc in ((kc, ks), (vc, vs))]
        for h in range(Hkv):
            w = weights[b, h, :L].astype(np.float64)
            rank = sorted(range(L), key=lambda t: (not (t < first or t >= L - recent),
                                                   np.inf if np.isnan(w[t]) else -w[t], t))
            mine = sorted(rank[:n])
            kept[b, h, :n] = mine
            new_w[b, h, :n] = weights[b, h, mine]
            for x, c, sc in zip(values, (kc, vc), (ks, vs)):
                for j0 in range(0, n, block):
                    j = np.arange(j0, min(j0 + block, n))
                    y = x[np.array(mine)[j], h]
                    s = block_scale(np.max(np.abs(y), initial=0.0, where=~np.isnan(y)))
                    page = int(new_table[b][j0 // P])
                    sc[page, j0 % P // block, h] = s
                    c[page, j % P, h] = e4m3_encode(y / s)
    return kept, lens, new_w
