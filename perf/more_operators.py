"""The operators of speculative decoding over the bf16 paged cache: cases, inputs, plain forms, 64-bit values.

Token t of sequence b lives in page page_table[b][t / page_size], slot t % page_size of caches
[num_pages, page_size, kv_heads, d]. The last n_b tokens of a sequence are its new ones.

  append   q and k of new tokens are rotated by their positions, k and v written to their pages
  tree     attention of n_b drafted tokens over their sequence's cache: a node sees every token
           before the drafts and those drafts whose bit is set in its mask (its ancestors)
  accept   the drafts that were accepted move to the places right behind the earlier tokens

`run` computes them with torch operations in 32 bits, or, with `own` set, by the library's calls.
"""
import math

import numpy as np
import torch

own = False


# ------------------------------------------------------------------ cases

def _append(name, batch, hq, hkv, d, rot, interleaved, page, lo, hi, new_lo, new_hi, tree):
    c = dict(op="append", batch=batch, hq=hq, hkv=hkv, d=d, rot=rot, interleaved=interleaved, page=page, lo=lo, hi=hi,
             new_lo=new_lo, new_hi=new_hi, tree=tree)
    return dict(name=name, **c) if name else c


def _tree(name, batch, hq, hkv, d, page, lo, hi, new_lo, new_hi, chain):
    c = dict(op="tree", batch=batch, hq=hq, hkv=hkv, d=d, page=page, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi,
             chain=chain)
    return dict(name=name, **c) if name else c


def _accept(name, batch, hkv, d, page, lo, hi, new_lo, new_hi, most):
    c = dict(op="accept", batch=batch, hkv=hkv, d=d, page=page, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, most=most)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # a decode step's new tokens, one a sequence, into the library's decode workload
        _append("append_step", 32, 32, 8, 128, 128, False, 16, 1024, 32767, 1, 1, False),
        # prompts of mixed lengths entering the cache, into empty sequences
        _append("append_prompts", 16, 32, 8, 128, 128, False, 16, 0, 0, 61, 8192, False),
        # drafts of a smaller model: half of head_dim 64 rotated in neighbouring pairs, positions by depth in the tree
        _append("append_drafts_d64", 24, 28, 4, 64, 32, True, 24, 37, 4099, 1, 13, True),
        # one user's short conversation, a tree of 16 drafts: only latency counts
        _tree("tree_one_short", 1, 32, 8, 128, 16, 1, 1013, 16, 16, False),
        # the library's decode workload, one token a sequence
        _tree("tree_one_token", 32, 32, 8, 128, 16, 1024, 32767, 1, 1, True),
        # the same with 16 drafts a sequence, 64 rows a KV head
        _tree("tree_ragged", 32, 32, 8, 128, 16, 1024, 32768, 16, 16, False),
        # one very long document, a tree of 60 drafts: the whole card has to share its keys
        _tree("tree_one_long", 1, 32, 8, 128, 128, 1, 131011, 60, 60, False),
        # wide trees on wide groups, 512 rows a KV head: arithmetic counts
        _tree("tree_wide", 16, 32, 4, 128, 16, 500, 8192, 64, 64, False),
        # a smaller model: head_dim 64, seven query heads a KV head, trees of uneven size, pages that end inside a tile
        _tree("tree_d64_odd", 24, 28, 4, 64, 24, 37, 4099, 1, 13, False),
        # a step's accepted drafts kept
        _accept("accept_step", 32, 8, 128, 16, 1024, 8192, 16, 16, 6),
        # a large server's step: many sequences, wide trees, long accepted paths
        _accept("accept_many", 512, 8, 128, 16, 64, 500, 1, 64, 17),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "tree", "tree", "accept"])
    d = rng.choice([64, 128, 128])
    page = rng.choice([16, 16, 128, 64, 24, 1, 48, 7, 4])
    hkv = rng.choice([1, 2, 4, 5, 8])
    batch = _log(rng, 1, 40)
    if op == "append":
        hq = hkv * rng.choice([1, 2, 3, 4, 4, 6, 7, 8])
        rot = rng.choice([d, d, d // 2, d // 4])
        tree = rng.random() < 0.4
        new_hi = _log(rng, 1, 64) if tree else _log(rng, 1, max(1, min(8192, 60_000 // batch)))
        hi = _log(rng, 1, 20_000)
        lo = rng.randint(0, hi)
        return _append("", batch, hq, hkv, d, rot, rng.random() < 0.4, page, lo, hi, rng.randint(0, new_hi), new_hi, tree)
    new_hi = _log(rng, 1, 64)
    new_lo = rng.randint(0, new_hi) if batch > 1 else new_hi
    if op == "accept":
        batch = _log(rng, 1, 512)
        hi = min(_log(rng, 1, 8192), 200_000 // batch)
        return _accept("", batch, hkv, d, page, rng.randint(0, hi), hi, new_lo, new_hi, rng.randint(1, new_hi))
    group = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    # scores of a sequence's longest: within those of the largest listed case
    most = min(500_000, 250_000_000 // (group * hkv * new_hi))
    hi = max(2, min(_log(rng, 20, 130_000), most // batch))
    lo = int(hi * rng.uniform(0.0, 1.0))
    return _tree("", batch, group * hkv, hkv, d, page, lo, hi, new_lo, new_hi, rng.random() < 0.3)


def _spread(n, lo, hi):
    """n lengths from lo to hi in even steps."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _sizes(c, rng):
    """Tokens before the new ones, and new tokens, of each sequence: lengths spread evenly, in a random order."""
    before = [_spread(c["batch"], c["lo"], c["hi"])[i] for i in rng.permutation(c["batch"])]
    new = [_spread(c["batch"], c["new_lo"], c["new_hi"])[i] for i in rng.permutation(c["batch"])]
    return before, new


def work(case):
    c, B, d = case, case["batch"], case["d"]
    new = _spread(B, c["new_lo"], c["new_hi"])
    if c["op"] == "append":
        n, heads = sum(new), c["hq"] + 2 * c["hkv"]
        table = min(n, c["hi"] + c["new_hi"]) * c["rot"] * 4
        return {"bytes": n * (heads * d * 4 + 4) + table + 8 * B, "flops": 3.0 * n * (c["hq"] + c["hkv"]) * c["rot"]}
    if c["op"] == "accept":
        rows = sum(min(n, c["most"]) for n in new)  # the longest path that `prepare` accepts, on average half of it
        return {"bytes": 0.5 * rows * (c["hkv"] * d * 8 + 4) + 12 * B, "flops": 0.0}
    # which length meets which number of drafts is left to the seed: their mean
    L = [a + sum(new) / B for a in _spread(B, c["lo"], c["hi"])]
    rows = sum(new) * c["hq"]
    pages = sum(math.ceil(x / c["page"]) for x in L)
    return {"bytes": sum(L) * c["hkv"] * d * 4 + rows * (4 * d + 4) + sum(new) * 8 + 4 * pages + 8 * B,
            "flops": 4.0 * sum(L) * (sum(new) / B) * c["hq"] * d}


# ------------------------------------------------------------------ inputs

def _tables(rng, lengths, page, pages, width):
    """Pages handed out in a random order: page_table [B, width], unused entries -1."""
    ids = rng.permutation(pages)
    table = np.full((len(lengths), width), -1)
    at = 0
    for b, n in enumerate(lengths):
        need = -(-n // page)
        table[b, :need] = ids[at:at + need]
        at += need
    return torch.tensor(table, dtype=torch.int32, device="cuda")


def _trees(rng, new):
    """Random trees of at most 64 nodes, parents before children: depth of each node and the bits of what
    it sees (its ancestors and itself), both [sum(new)]."""
    B, most = len(new), max(new)
    depth = np.zeros((B, most), dtype=np.int64)
    seen = np.zeros((B, most), dtype=np.uint64)
    for i in range(most):
        parent = np.where(rng.random(B) < 0.1, -1, rng.integers(max(0, i - 6), max(1, i), B)) if i else np.full(B, -1)
        up = np.maximum(parent, 0)
        root = parent < 0
        depth[:, i] = np.where(root, 0, depth[np.arange(B), up] + 1)
        seen[:, i] = np.where(root, np.uint64(0), seen[np.arange(B), up]) | np.uint64(1 << i)
    used = np.arange(most)[None, :] < np.asarray(new)[:, None]
    return depth, seen, used


def prepare(case, seed):
    c, B, P, H, d = case, case["batch"], case["page"], case["hkv"], case["d"]
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    before, new = _sizes(c, rng)
    L = [a + n for a, n in zip(before, new)]
    n = sum(new)
    pages = max(1, sum(-(-x // P) for x in L))
    s = dict(c)
    s["lens"] = torch.tensor(L, dtype=torch.int32, device="cuda")
    s["offs"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    s["table"] = _tables(rng, L, P, pages, max(1, -(-max(L) // P)))
    for x in ("kc", "vc"):  # keys and values of uneven size
        t = torch.randn(pages, P, H, d, generator=g, device="cuda")
        s[x] = t.mul_(torch.exp(0.3 * torch.randn(pages, P, H, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    if c["op"] == "append":
        Hq, rot = c["hq"], c["rot"]
        # what a projection leaves behind: q, k and v of a token side by side in one row
        qkv = torch.randn(n, (Hq + 2 * H) * d, generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, H * d, H * d], dim=1))
        angle = torch.arange(max(L) + 1, dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["positions"] = None
        if c["tree"] and n:
            depth, _, used = _trees(rng, new)
            s["positions"] = torch.tensor((np.asarray(before)[:, None] + depth)[used], dtype=torch.int32, device="cuda")
    elif c["op"] == "tree":
        s["q"] = torch.randn(n, c["hq"], d, generator=g, device="cuda").to(torch.bfloat16)
        s["mask"], s["most"] = None, max(new)
        if not c["chain"] and n:
            _, seen, used = _trees(rng, new)
            s["mask"] = torch.tensor(seen[used].view(np.int64), device="cuda")
    else:
        # accepted paths: in order, of uneven length (none at all for some)
        width = min(c["most"], max(1, max(new)))
        path, count = np.zeros((B, width), dtype=np.int32), np.zeros(B, dtype=np.int32)
        for b in range(B):
            count[b] = rng.integers(0, min(new[b], width) + 1)
            path[b, :count[b]] = np.sort(rng.choice(new[b], count[b], replace=False)) if count[b] else 0
        s["path"], s["count"] = torch.tensor(path, device="cuda"), torch.tensor(count, device="cuda")
    return s


# ------------------------------------------------------------------ the plain forms

def _new_tokens(s):
    """Sequence, index within it and position of every new token."""
    L, offs = s["lens"].long(), s["offs"].long()
    n = offs[1:] - offs[:-1]
    seq = torch.arange(len(n), device="cuda").repeat_interleave(n)
    i = torch.arange(len(seq), device="cuda") - offs[seq]
    return seq, i, (L - n)[seq] + i


def _plain_rotate(x, cos, sin, interleaved):
    x = x.float()
    half = cos.shape[1]
    cos, sin = cos[:, None, :], sin[:, None, :]
    y = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :half], x[..., half:2 * half]
        y[..., :half], y[..., half:2 * half] = a * cos - b * sin, b * cos + a * sin
    return y.to(torch.bfloat16)


def _plain_append(s):
    seq, _, slot = _new_tokens(s)
    at = slot if s["positions"] is None else s["positions"].long()
    cos, sin = s["cos"][at], s["sin"][at]
    page = s["table"][seq, slot // s["page"]].long()
    s["kc"][page, slot % s["page"]] = _plain_rotate(s["k"], cos, sin, s["interleaved"])
    s["vc"][page, slot % s["page"]] = s["v"]
    return {"q": _plain_rotate(s["q"], cos, sin, s["interleaved"]), "k_cache": s["kc"], "v_cache": s["vc"]}


def _dense(cache, table):
    """The tokens that the pages of a table hold: fp32 [B, tokens, H, d]."""
    return cache[table.clamp(min=0).long()].flatten(1, 2).float()


def _plain_tree(s):
    n, Hq, d = s["q"].shape
    B, H, most = s["batch"], s["hkv"], s["most"]
    if n == 0:
        return {"o": torch.empty_like(s["q"]), "lse": torch.empty(0, Hq, device="cuda")}
    G = Hq // H
    seq, i, _ = _new_tokens(s)
    q = torch.zeros(B, most, Hq, d, device="cuda")
    q[seq, i] = s["q"].float()
    bits = torch.zeros(B, most, dtype=torch.int64, device="cuda")
    bits[seq, i] = s["mask"] if s["mask"] is not None else \
        torch.where(i < 63, (2 << i.clamp(max=62)) - 1, torch.full_like(i, -1))
    k = _dense(s["kc"], s["table"])
    T = k.shape[1]
    sc = torch.matmul(q.view(B, most, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, most * G, d),
                      k.permute(0, 2, 3, 1)) / math.sqrt(d)
    del k
    L = s["lens"].long()
    first = L - (s["offs"][1:] - s["offs"][:-1])  # the first draft's position
    t = torch.arange(T, device="cuda")
    j = t - first[:, None]
    draft = (bits[:, :, None] >> j.clamp(0, 63)[:, None, :]) & 1
    sees = (j < 0)[:, None, :] | ((t < L[:, None])[:, None, :] & (draft == 1))
    sc = sc.view(B, H, most, G, T).masked_fill_(~sees[:, None, :, None, :], -math.inf)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)
    p = p.div_(torch.where(l > 0, l, torch.ones_like(l))).view(B, H, most * G, T)
    v = torch.where((t < L[:, None])[:, :, None, None], _dense(s["vc"], s["table"]), 0.0)
    o = torch.matmul(p, v.transpose(1, 2))
    o = o.view(B, H, most, G, d).permute(0, 2, 1, 3, 4).reshape(B, most, Hq, d)[seq, i].to(torch.bfloat16)
    return {"o": o, "lse": lse.view(B, H, most, G).permute(0, 2, 1, 3).reshape(B, most, Hq)[seq, i]}


def _plain_accept(s):
    P, L, table = s["page"], s["lens"].long(), s["table"]
    first = L - (s["offs"][1:] - s["offs"][:-1])
    k = torch.arange(s["path"].shape[1], device="cuda")
    b, k = torch.nonzero(k < s["count"][:, None], as_tuple=True)
    src, dst = first[b] + s["path"][b, k], first[b] + k
    sp, dp = table[b, src // P].long(), table[b, dst // P].long()
    for c in (s["kc"], s["vc"]):
        c[dp, dst % P] = c[sp, src % P]
    return {"lens": (first + s["count"]).to(torch.int32), "k_cache": s["kc"], "v_cache": s["vc"]}


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        import varlen_flashattention_gb300 as jfa
        cache = (s["kc"], s["vc"], s["table"], s["lens"])
        if s["op"] == "append":
            q = jfa.jfa_cache_append_rope(s["q"], s["k"], s["v"], *cache, s["offs"], s["cos"], s["sin"],
                                          positions=s["positions"], interleaved=s["interleaved"])
            return {"q": q, "k_cache": s["kc"], "v_cache": s["vc"]}
        if s["op"] == "tree":
            o, lse = jfa.jfa_decode_tree(s["q"], *cache, s["offs"], s["mask"], max_q=s["most"])
            return {"o": o, "lse": lse}
        lens = jfa.jfa_cache_accept(*cache, s["offs"], s["path"], s["count"])
        return {"lens": lens, "k_cache": s["kc"], "v_cache": s["vc"]}
    return {"append": _plain_append, "tree": _plain_tree, "accept": _plain_accept}[s["op"]](s)


# ------------------------------------------------------------------ the values in 64 bits

def _exact_append(s):
    L, offs, P, half = s["lens"].tolist(), s["offs"].tolist(), s["page"], s["rot"] // 2
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else (slice(0, half), slice(half, 2 * half))
    out = {"q": s["q"].double(), "k_cache": s["kc"].double(), "v_cache": s["vc"].double()}
    for b in range(len(L)):
        rows = slice(offs[b], offs[b + 1])
        n = offs[b + 1] - offs[b]
        at = torch.arange(L[b] - n, L[b], device="cuda")
        turn = at if s["positions"] is None else s["positions"][rows].long()
        page, slot = s["table"][b].long()[at // P], at % P
        z = torch.complex(s["cos"].double()[turn], s["sin"].double()[turn])[:, None, :]
        for name in ("q", "k"):
            x = s[name][rows].double()
            w = torch.complex(x[..., lo], x[..., hi]) * z
            x[..., lo], x[..., hi] = w.real, w.imag
            if name == "q":
                out["q"][rows] = x
            else:
                out["k_cache"][page, slot] = x
        out["v_cache"][page, slot] = s["v"][rows].double()
    return out


def _exact_tree(s):
    n, Hq, d = s["q"].shape
    H, P = s["hkv"], s["page"]
    o = torch.zeros(n, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((n, Hq), -math.inf, dtype=torch.float64, device="cuda")
    offs = s["offs"].tolist()
    masks = None if s["mask"] is None else s["mask"].tolist()
    for b, L in enumerate(s["lens"].tolist()):
        first = L - (offs[b + 1] - offs[b])
        t = torch.arange(L, device="cuda")
        pg, slot = s["table"][b].long()[t // P], t % P
        k, v = s["kc"][pg, slot].double(), s["vc"][pg, slot].double()
        for i in range(offs[b], offs[b + 1]):
            if masks is None:
                see = t <= first + i - offs[b]
            else:
                see = torch.tensor([j < 0 or bool(masks[i] >> j & 1) for j in range(-1, L - first)], device="cuda")
                see = torch.cat([see[:1].expand(first), see[1:]])
            x = torch.einsum("hgd,thd->hgt", s["q"][i].double().view(H, -1, d), k) / math.sqrt(d)
            x = x.masked_fill(~see, -math.inf)
            z = torch.logsumexp(x, -1)
            p = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
            o[i] = torch.einsum("hgt,thd->hgd", p, v).reshape(Hq, d)
            lse[i] = z.reshape(Hq)
    return {"o": o, "lse": lse}


def _exact_accept(s):
    P, table = s["page"], s["table"].tolist()
    L, offs, count, path = s["lens"].tolist(), s["offs"].tolist(), s["count"].tolist(), s["path"].tolist()
    at, src = [], []
    for b in range(len(L)):
        first = L[b] - (offs[b + 1] - offs[b])
        for k in range(count[b]):
            for lst, t in ((at, first + k), (src, first + path[b][k])):
                lst.append(table[b][t // P] * P + t % P)
    out = {"lens": np.array([L[b] - (offs[b + 1] - offs[b]) + count[b] for b in range(len(L))])}
    for name, c in (("k_cache", s["kc"]), ("v_cache", s["vc"])):
        rows = c.double().flatten(0, 1)
        rows[at] = rows[src]
        out[name] = rows.view(c.shape)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "tree": _exact_tree, "accept": _exact_accept}[s["op"]](s)
