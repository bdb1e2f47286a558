"""The operators of the 8-bit paged KV cache: their cases, inputs, plain forms and 64-bit values.

A cache holds e4m3 codes [num_pages, page_size, kv_heads, d] for K and V and fp32 scales
[num_pages, page_size / block, kv_heads]; the value of a code is e4m3(code) * scale of its block.
Token t of sequence b lives in page page_table[b][t / page_size], slot t % page_size.

  append   bf16 K and V of new tokens are quantized into the cache (block scales are powers of two)
  decode   attention of the last q_len tokens of each sequence over its cache, optionally adding
           each cached token's attention weight to a running sum
  evict    the tokens of the largest weights (with the first and the most recent ones) are kept,
           in order, in new pages

`run` computes them with torch operations in 32 bits, or, with `own` set, by the library's calls.
"""
import math

import numpy as np
import torch

own = False

F8 = torch.float8_e4m3fn
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _decode(name, batch, q_len, hq, hkv, d, page, block, lo, hi, weights):
    c = dict(op="decode", batch=batch, q_len=q_len, hq=hq, hkv=hkv, d=d, page=page, block=block, lo=lo, hi=hi,
             weights=weights)
    return dict(name=name, **c) if name else c


def _append(name, batch, hkv, d, page, block, lo, hi, new_lo, new_hi, weights):
    c = dict(op="append", batch=batch, hkv=hkv, d=d, page=page, block=block, lo=lo, hi=hi, new_lo=new_lo,
             new_hi=new_hi, weights=weights)
    return dict(name=name, **c) if name else c


def _evict(name, batch, hkv, d, page, block, lo, hi, keep, first, recent):
    c = dict(op="evict", batch=batch, hkv=hkv, d=d, page=page, block=block, lo=lo, hi=hi, keep=keep, first=first,
             recent=recent)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one user's short conversation, one token: only latency counts
        _decode("decode_one_short", 1, 1, 32, 8, 128, 16, 16, 1, 1013, False),
        # the library's decode workload: 32 sequences of 1k to 32k tokens, 32 query heads on 8 KV heads
        _decode("decode_ragged", 32, 1, 32, 8, 128, 16, 16, 1024, 32768, False),
        # the same server keeping the weights that eviction goes by
        _decode("decode_ragged_weights", 32, 1, 32, 8, 128, 16, 16, 1024, 32768, True),
        # one very long document: few rows, the whole card has to share its keys
        _decode("decode_one_long", 1, 1, 32, 8, 128, 128, 64, 1, 131071, False),
        # four draft tokens checked at once, 16 rows a KV head
        _decode("decode_draft_tokens", 16, 4, 32, 8, 128, 16, 16, 500, 8192, True),
        # a smaller model: head_dim 64, seven query heads a KV head, pages that end inside a tile
        _decode("decode_d64_odd", 24, 1, 28, 4, 64, 24, 8, 37, 4099, True),
        # a decode step's new tokens, one a sequence
        _append("append_step", 32, 8, 128, 16, 16, 1024, 32767, 1, 1, True),
        # prompts of mixed lengths entering the cache, into empty sequences
        _append("append_prompts", 16, 8, 128, 16, 16, 0, 0, 61, 8192, False),
        # a long prompt's next piece behind what is there, off the blocks' borders
        _append("append_chunk_d64", 5, 4, 64, 48, 8, 333, 5001, 301, 2048, True),
        # one conversation cut back
        _evict("evict_one_short", 1, 8, 128, 16, 16, 1, 1999, 512, 4, 64),
        # the decode workload's caches cut to 2k tokens
        _evict("evict_ragged", 32, 8, 128, 16, 16, 1024, 32768, 2048, 16, 256),
        # one very long document cut to an eighth
        _evict("evict_one_long", 1, 8, 128, 128, 64, 1, 131071, 16384, 64, 1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "append", "evict"])
    d = rng.choice([64, 128, 128])
    page, block = rng.choice([(16, 16), (16, 16), (128, 64), (64, 32), (24, 8), (1, 1), (48, 16), (128, 128), (7, 1)])
    hkv = rng.choice([1, 2, 4, 5, 8])
    batch = _log(rng, 1, 40)
    most = 500_000  # cached tokens of all sequences; the largest listed case has 540 thousand of 8 heads
    hi = max(2, min(_log(rng, 20, 130_000), most // batch))
    lo = max(1, int(hi * rng.uniform(0.02, 1.0)))
    if op == "decode":
        group = rng.choice([1, 2, 3, 4, 4, 6, 8, 16])
        q_len = rng.randint(1, min(8, 16 // group)) if rng.random() < 0.4 else 1
        return _decode("", batch, q_len, group * hkv, hkv, d, page, block, lo, hi, rng.random() < 0.5)
    if op == "append":
        new_hi = _log(rng, 1, max(1, min(8192, 130_000 // batch)))
        return _append("", batch, hkv, d, page, block, min(lo, 20_000), min(hi, 30_000), rng.randint(0, new_hi), new_hi,
                       rng.random() < 0.5)
    keep = max(1, int(hi * rng.uniform(0.05, 0.6)))
    first = rng.randint(0, min(64, keep // 3))
    return _evict("", batch, hkv, d, page, block, lo, hi, keep, first, rng.randint(0, min(1024, keep // 2)))


def _spread(n, lo, hi):
    """n lengths from lo to hi in even steps."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(c):
    return _spread(c["batch"], c["lo"], c["hi"])


def work(case):
    c, B, H, d = case, case["batch"], case["hkv"], case["d"]
    row = 2 * (d + 4.0 / c["block"])  # a cached token's K and V of one head, with its share of the scales
    L = sum(_lengths(c))
    if c["op"] == "decode":
        rows = B * c["q_len"] * c["hq"]
        nbytes = L * H * row + rows * (4 * d + 4) + 4 * B + 4 * sum(-(-n // c["page"]) for n in _lengths(c))
        if c["weights"]:
            nbytes += 8 * L * H
        return {"bytes": nbytes, "flops": 4.0 * L * c["q_len"] * c["hq"] * d}
    if c["op"] == "append":
        n = sum(_spread(B, c["new_lo"], c["new_hi"]))
        return {"bytes": n * H * (4 * d + row + (4 if c["weights"] else 0)) + 12 * B, "flops": 4.0 * n * H * d}
    kept = sum(min(n, c["keep"]) for n in _lengths(c))
    return {"bytes": 4 * L * H + kept * H * (2 * row + 8) + 8 * B, "flops": 4.0 * kept * H * d}


# ------------------------------------------------------------------ inputs

def _pow2_scale(amax):
    """The smallest power of two s with amax / s <= 448, and at least 2^-126."""
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [0.5, 1)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)
    e = torch.where(amax > 0, e, torch.full_like(e, -126))
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _pool(g, pages, page, block, H, d):
    """A filled cache: keys (or values) of uneven size, quantized block by block."""
    x = torch.randn(pages, page, H, d, generator=g, device="cuda")
    x *= torch.exp(0.7 * torch.randn(pages, page, H, 1, generator=g, device="cuda"))
    s = _pow2_scale(x.view(pages, page // block, block, H, d).abs().amax((2, 4)))
    x /= s.repeat_interleave(block, 1)[..., None]
    return x.to(F8).view(torch.uint8), s


def _tables(g, lengths, page, pages, spare, width):
    """Pages handed out in a random order: page_table [B, width], unused entries -1."""
    need = torch.tensor([-(-n // page) for n in lengths], device="cuda")
    ids = torch.randperm(pages - spare, generator=g, device="cuda", dtype=torch.int64)
    slot = torch.arange(width, device="cuda")[None, :]
    at = (need.cumsum(0) - need)[:, None] + slot
    return torch.where(slot < need[:, None], ids[at.clamp(max=len(ids) - 1)], -1).to(torch.int32)


def prepare(case, seed):
    c, B, H, d, P, blk = case, case["batch"], case["hkv"], case["d"], case["page"], case["block"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    perm = torch.randperm(B, generator=g, device="cuda").tolist()
    L = [_lengths(c)[i] for i in perm]
    s = dict(c)
    new = [0] * B
    if c["op"] == "append":
        perm = torch.randperm(B, generator=g, device="cuda").tolist()
        new = [_spread(B, c["new_lo"], c["new_hi"])[i] for i in perm]
        L = [a + b for a, b in zip(L, new)]
    spare = 0
    if c["op"] == "evict":
        spare = sum(-(-min(n, c["keep"]) // P) for n in L)
    pages = sum(-(-n // P) for n in _lengths(c)) + sum(-(-n // P) for n in new) + spare
    s["kc"], s["ks"] = _pool(g, pages, P, blk, H, d)
    s["vc"], s["vs"] = _pool(g, pages, P, blk, H, d)
    s["table"] = _tables(g, L, P, pages, spare, -(-(c["hi"] + max(new)) // P))
    s["lens"] = torch.tensor(L, dtype=torch.int32, device="cuda")
    cap = s["table"].shape[1] * P
    if c["op"] == "decode":
        s["q"] = torch.randn(B, c["q_len"], c["hq"], d, generator=g, device="cuda").to(torch.bfloat16)
        if c["weights"]:
            s["w"] = torch.rand(B, H, cap, generator=g, device="cuda")
            s["w_out"] = torch.zeros_like(s["w"])
    elif c["op"] == "append":
        n = sum(new)
        s["max_new"] = max(new)
        s["offs"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
        for x in ("k", "v"):
            t = torch.randn(n, H, d, generator=g, device="cuda")
            s[x] = (t * torch.exp(0.9 * torch.randn(n, H, 1, generator=g, device="cuda"))).to(torch.bfloat16)
        s["w"] = torch.rand(B, H, cap, generator=g, device="cuda") if c["weights"] else None
    else:
        # summed attention weights: heavy-tailed, and none at all for one token in ten
        w = torch.exp(2.0 * torch.randn(B, H, cap, generator=g, device="cuda") - 6.0)
        s["w"] = w * (torch.rand(B, H, cap, generator=g, device="cuda") > 0.1)
        fit = [min(n, c["keep"]) for n in L]
        t = _tables(g, fit, P, spare, 0, -(-c["keep"] // P))  # room for `keep` tokens each
        s["new_table"] = torch.where(t >= 0, t + (pages - spare), t)
        s["spare"] = spare
    return s


# ------------------------------------------------------------------ the plain forms

def _dense(codes, scales, table, block):
    """The values that the pages of a table hold: fp32 [B, tokens, H, d]."""
    at = table.clamp(min=0).long()
    x = codes[at].view(F8).float() * scales[at].repeat_interleave(block, 2)[..., None]
    return x.flatten(1, 2)


def _plain_decode(s):
    B, ql, Hq, d = s["q"].shape
    H = s["hkv"]
    G = Hq // H
    q = s["q"].float().view(B, ql, H, G, d).transpose(1, 2).reshape(B, H, ql * G, d)
    k = _dense(s["kc"], s["ks"], s["table"], s["block"])
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)) / math.sqrt(d)
    T = k.shape[1]
    del k
    t = torch.arange(T, device="cuda")
    L = s["lens"].long()
    limit = L[:, None] - ql + torch.arange(ql, device="cuda").repeat_interleave(G)[None, :]
    sc = torch.where(t <= limit[:, None, :, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = torch.exp(sc - m)
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    p = p / torch.where(l > 0, l, torch.ones_like(l))
    v = _dense(s["vc"], s["vs"], s["table"], s["block"])
    o = torch.matmul(p, v.transpose(1, 2))
    o = o.view(B, H, ql, G, d).transpose(1, 2).reshape(B, ql, Hq, d).to(torch.bfloat16)
    lse = lse.view(B, H, ql, G).transpose(1, 2).reshape(B, ql, Hq)
    if not s["weights"]:
        return {"o": o, "lse": lse}
    w = torch.where(t < L[:, None, None], 0.97 * s["w"] + p.sum(2), s["w_out"])
    return {"o": o, "lse": lse, "weights": w}


def _plain_store(x, codes, scales, block, page, slot, first_page, first_slot, old_in_first):
    """Quantizes x [n, H, d] into (page, slot) of each token; the block of a sequence's first new
    token may hold older tokens (slots first_slot - old_in_first ... first_slot - 1)."""
    per = scales.shape[1]
    H, d = x.shape[1:]
    s = scales.view(-1, H)
    cell = page * per + slot // block
    x = x.float()
    amax = x.abs().amax(-1)
    need = torch.zeros_like(s).scatter_reduce(0, cell[:, None].expand(-1, H), amax, "amax")
    new = _pow2_scale(need)
    mixed = first_page[old_in_first > 0] * per + first_slot[old_in_first > 0] // block
    old = s[mixed].clone()
    grown = torch.maximum(old, new[mixed])
    new[mixed] = grown
    s[cell] = new[cell]
    # the older tokens of those blocks, at the grown scale
    n_old = old_in_first[old_in_first > 0]
    which = torch.arange(len(n_old), device="cuda").repeat_interleave(n_old)
    back = torch.arange(len(which), device="cuda") - (n_old.cumsum(0) - n_old)[which] + 1
    po, so = first_page[old_in_first > 0][which], first_slot[old_in_first > 0][which] - back
    was = codes[po, so].view(F8).float()
    codes[po, so] = (was * old[which][..., None] / grown[which][..., None]).to(F8).view(torch.uint8)
    codes[page, slot] = (x / new[cell][..., None]).to(F8).view(torch.uint8)


def _plain_append(s):
    P, blk = s["page"], s["block"]
    L, offs = s["lens"].long(), s["offs"].long()
    n = offs[1:] - offs[:-1]
    seq = torch.arange(len(n), device="cuda").repeat_interleave(n)
    pos = (L - n)[seq] + torch.arange(len(seq), device="cuda") - offs[seq]
    page, slot = s["table"][seq, pos // P].long(), pos % P
    some = n > 0
    f = (L - n)[some]
    fp, fs = s["table"][some, f // P].long(), f % P
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        _plain_store(x, codes, scales, blk, page, slot, fp, fs, fs % blk)
    out = _cache_values(s)
    if s["weights"]:
        s["w"][seq, :, pos] = 0.0
        out["weights"] = s["w"]
    return out


def _cache_values(s, start=0):
    return {"k": s["kc"][start:].view(F8), "v": s["vc"][start:].view(F8), "k_scale": s["ks"][start:],
            "v_scale": s["vs"][start:]}


def _plain_evict(s):
    B, H, T = s["w"].shape
    P, blk, keep, d = s["page"], s["block"], s["keep"], s["d"]
    L = s["lens"].long()[:, None, None]
    t = torch.arange(T, device="cuda")
    w = torch.where(torch.isnan(s["w"]), -math.inf, s["w"])
    by_weight = torch.sort(w, dim=-1, descending=True, stable=True).indices
    rank = torch.where((t < s["first"]) | (t >= L - s["recent"]), 1, 0) + torch.where(t < L, 0, -2)
    by_rank = torch.sort(rank.expand(B, H, T).gather(-1, by_weight), dim=-1, descending=True, stable=True).indices
    kept = by_weight.gather(-1, by_rank)[..., :keep]
    if keep > T:
        kept = torch.cat([kept, torch.zeros(B, H, keep - T, dtype=kept.dtype, device="cuda")], -1)
    j = torch.arange(keep, device="cuda")
    n = L.clamp(max=keep)
    kept = torch.sort(torch.where(j < n, kept, T), -1).values
    valid = kept < T
    src = torch.where(valid, kept, torch.zeros_like(kept))
    page = s["table"].clamp(min=0).long()[torch.arange(B, device="cuda")[:, None, None], src // P]
    h = torch.arange(H, device="cuda")[None, :, None]
    width = s["new_table"].shape[1] * P
    new_w = torch.zeros(B, H, width, device="cuda")
    new_w[..., :keep] = torch.where(valid, s["w"].gather(-1, src), 0.0)
    b, hh, jj = torch.nonzero(valid, as_tuple=True)
    to = s["new_table"][b, jj // P].long()
    pad = -keep % blk
    for codes, scales in ((s["kc"], s["ks"]), (s["vc"], s["vs"])):
        x = codes[page, src % P, h].view(F8).float() * scales[page, src % P // blk, h][..., None]
        x = torch.where(valid[..., None], x, 0.0)
        amax = torch.nn.functional.pad(x.abs().amax(-1), (0, pad)).view(B, H, -1, blk).amax(-1)
        sn = _pow2_scale(amax).repeat_interleave(blk, -1)[..., :keep]
        y = (x / sn[..., None]).to(F8).view(torch.uint8)
        codes[to, jj % P, hh] = y[b, hh, jj]
        scales[to, jj % P // blk, hh] = sn[b, hh, jj]
    kept = torch.where(valid, kept, -1).to(torch.int32)
    return {"kept": kept, "lens": n.flatten().to(torch.int32), "weights": new_w,
            **_cache_values(s, len(s["kc"]) - s["spare"])}


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import varlen_flashattention_gb300 as jfa
        cache = (s["kc"], s["vc"], s["ks"], s["vs"])
        if s["op"] == "decode":
            if not s["weights"]:
                o, lse = jfa.jfa_decode_fp8(s["q"], *cache, s["table"], s["lens"])
                return {"o": o, "lse": lse}
            o, lse = jfa.jfa_decode_fp8(s["q"], *cache, s["table"], s["lens"], weights=s["w"], decay=0.97,
                                        weights_out=s["w_out"])
            return {"o": o, "lse": lse, "weights": s["w_out"]}
        if s["op"] == "append":
            jfa.jfa_cache_append_fp8(s["k"], s["v"], *cache, s["table"], s["lens"], s["offs"], s["max_new"],
                                     weights=s["w"])
            return {**_cache_values(s), "weights": s["w"]} if s["weights"] else _cache_values(s)
        kept, lens, w = jfa.jfa_cache_evict_fp8(*cache, s["table"], s["lens"], s["w"], s["keep"], s["new_table"],
                                                first=s["first"], recent=s["recent"])
        return {"kept": kept, "lens": lens, "weights": w, **_cache_values(s, len(s["kc"]) - s["spare"])}
    if s["op"] == "decode":
        return _plain_decode(s)
    return _plain_append(s) if s["op"] == "append" else _plain_evict(s)


# ------------------------------------------------------------------ the values in 64 bits

def _e4m3_table():
    code = np.arange(256)
    e, m = (code >> 3) & 15, code & 7
    x = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    x[(code & 127) == 127] = np.nan
    return torch.tensor(np.where(code > 127, -x, x), device="cuda")


def _powers(lo, hi):
    return torch.tensor([2.0 ** e for e in range(lo, hi)], dtype=torch.float64, device="cuda")


def _round_e4m3(x):
    """The nearest e4m3 value (ties to even) of 64-bit numbers of at most 448."""
    p = _powers(-6, 9)  # the values from p[i] up to p[i + 1] are p[i] / 8 apart, those below p[0] as above it
    step = p[(torch.searchsorted(p, x.abs(), right=True) - 1).clamp(min=0)] / 8
    return torch.round(x / step) * step


def _exact_scale(amax):
    p = _powers(-126, 128)
    return p[torch.searchsorted(p * E4M3_MAX, amax.contiguous())]  # the first whose 448-fold is not below amax


def _exact_decode(s):
    tab = _e4m3_table()
    B, ql, Hq, d = s["q"].shape
    H, P, blk = s["hkv"], s["page"], s["block"]
    G = Hq // H
    o = torch.zeros(B, ql, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, ql, Hq), -math.inf, dtype=torch.float64, device="cuda")
    w = s["w_out"].double() if s["weights"] else None
    for b, L in enumerate(s["lens"].tolist()):
        t = torch.arange(L, device="cuda")
        pg, slot = s["table"][b].long()[t // P], t % P
        k, v = (tab[c[pg, slot].int()] * sc[pg, slot // blk].double()[..., None]
                for c, sc in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        total = torch.zeros(H, L, dtype=torch.float64, device="cuda")
        for i in range(ql):
            see = max(0, L - ql + i + 1)
            if see:
                q = s["q"][b, i].double().view(H, G, d)
                x = torch.einsum("hgd,thd->hgt", q, k[:see]) * d ** -0.5
                z = torch.logsumexp(x, -1)
                p = torch.exp(x - z[..., None])
                o[b, i] = torch.einsum("hgt,thd->hgd", p, v[:see]).reshape(Hq, d)
                lse[b, i] = z.reshape(Hq)
                total[:, :see] += p.sum(1)
        if w is not None:
            w[b, :, :L] = 0.97 * s["w"][b, :, :L].double() + total
    return {"o": o, "lse": lse, "weights": w} if s["weights"] else {"o": o, "lse": lse}


def _exact_append(s):
    """Block by block of the new tokens; whole caches come back, as held values and scales."""
    tab = _e4m3_table()
    P, blk = s["page"], s["block"]
    offs, L = s["offs"].tolist(), s["lens"].tolist()
    out = {}
    for n, x, c, sc in (("k", s["k"], s["kc"], s["ks"]), ("v", s["v"], s["vc"], s["vs"])):
        val, scale = tab[c.int()], sc.double()
        for b in range(len(L)):
            f, e = L[b] - (offs[b + 1] - offs[b]), L[b]
            if f == e:
                continue
            pos = torch.arange(f // blk * blk, -(-e // blk) * blk, device="cuda")  # whole blocks
            real = pos < e
            pg = s["table"][b].long()[pos // P]
            y = torch.zeros(len(pos), *x.shape[1:], dtype=torch.float64, device="cuda")
            y[(pos >= f) & real] = x[offs[b]:offs[b + 1]].double()
            before = scale[pg[0], int(pos[0]) % P // blk].clone()
            S = _exact_scale(y.view(-1, blk, *x.shape[1:]).abs().amax((1, 3)))
            if f % blk:
                S[0] = torch.maximum(S[0], before)
            keep = pos < f
            y[keep] = val[pg[keep], pos[keep] % P] * before[None, :, None]
            held = _round_e4m3(y / S.repeat_interleave(blk, 0)[..., None])
            val[pg[real], pos[real] % P] = held[real]
            scale[pg[::blk], pos[::blk] % P // blk] = S
        out[n], out[n + "_scale"] = val, scale
    if s["weights"]:
        w = s["w"].double()
        for b in range(len(L)):
            w[b, :, L[b] - (offs[b + 1] - offs[b]):L[b]] = 0
        out["weights"] = w
    return out


def _exact_evict(s):
    tab = _e4m3_table()
    B, H, _ = s["w"].shape
    P, blk, keep, first, recent = s["page"], s["block"], s["keep"], s["first"], s["recent"]
    w = s["w"].double().cpu().numpy()
    L, table, fresh = s["lens"].tolist(), s["table"].long(), s["new_table"].long()
    base = len(s["kc"]) - s["spare"]
    kept = np.full((B, H, keep), -1)
    new_w = np.zeros((B, H, fresh.shape[1] * P))
    val = {n: tab[s[n][base:].int()] for n in ("kc", "vc")}
    scale = {n: s[n][base:].double() for n in ("ks", "vs")}
    for b in range(B):
        n = min(L[b], keep)
        for h in range(H):
            at = np.arange(L[b])
            safe = (at < first) | (at >= L[b] - recent)
            order = np.lexsort((at, -w[b, h, :L[b]], ~safe))
            kept[b, h, :n] = np.sort(order[:n])
            new_w[b, h, :n] = w[b, h, kept[b, h, :n]]
        src = torch.tensor(kept[b, :, :n], device="cuda")
        j = torch.arange(n, device="cuda")
        to = fresh[b][j // P] - base
        hh = torch.arange(H, device="cuda")[:, None]
        for c, sc in (("kc", "ks"), ("vc", "vs")):
            x = tab[s[c][table[b][src // P], src % P, hh].int()]
            x = x * s[sc][table[b][src // P], src % P // blk, hh].double()[..., None]
            y = torch.zeros(H, -(-n // blk) * blk, x.shape[-1], dtype=torch.float64, device="cuda")
            y[:, :n] = x
            S = _exact_scale(y.view(H, -1, blk, x.shape[-1]).abs().amax((2, 3))).repeat_interleave(blk, 1)
            val[c][to, j % P] = _round_e4m3(y / S[..., None])[:, :n].transpose(0, 1)
            scale[sc][to, j % P // blk] = S[:, :n].t().contiguous()
    return {"kept": kept, "lens": np.minimum(L, keep), "weights": new_w, "k": val["kc"], "v": val["vc"],
            "k_scale": scale["ks"], "v_scale": scale["vs"]}


def exact(case, seed):
    s = prepare(case, seed)
    return {"decode": _exact_decode, "append": _exact_append, "evict": _exact_evict}[s["op"]](s)
