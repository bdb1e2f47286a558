"""GPU parity of the 8-bit paged cache where masks, single roundings and largest sizes decide.

Codes, scales and positions are compared with the fp64 oracle bit for bit; the weights by the
bounds that tests/test_gpu_fp8_cache.py derives.
"""
import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import kv_cache as kvo
from tests.parity import np64
from tests.test_gpu_fp8_cache import _bf16, _cache, _case, _gpu, _same_codes, check_decode

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ accumulated weights

# beside the join (short rows of the table) and behind it (more than 32 parts a sequence), with 4, 8 and 16 rows
@pytest.mark.parametrize("lens", [[40, 5, 70, 300], [1200], [1203]])
@pytest.mark.parametrize("G,ql", [(1, 4), (2, 4), (4, 2), (4, 4), (3, 5)])
@pytest.mark.parametrize("what", ["nan", "inf", "key"])
def test_weights_of_tokens_that_a_nan_row_does_not_see(lens, G, ql, what):
    """A query row that is NaN makes NaN of the weights of the tokens it sees, and of no others."""
    c = _case(40, lens, 2, 64, 16, 16)
    rng = c["rng"]
    q = _bf16(rng, len(lens), ql, 2 * G, 64)
    for b in range(len(lens)):
        if what == "key":  # seen by the last query token alone: all of head 0's weights, none of head 1's
            t = lens[b] - 1
            c["kc"][c["table"][b, t // 16], t % 16, 0, 3] = 0x7F
        elif what == "nan" or lens[b] > 30:  # (of few keys all may be below 0: a row of -infinities)
            q[b, 0, G - 1, 5] = float(what)
            q[b, ql // 2, 2 * G - 1, 9] = -float(what)
    w = rng.random((len(lens), 2, c["cap"])).astype(np.float32)
    was = np.full_like(w, -7.0)
    out = torch.from_numpy(was).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(_gpu(c)), weights=torch.from_numpy(w).cuda(), decay=0.97,
                                weights_out=out, check=True)
    with np.errstate(invalid="ignore"):
        O, LSE, W, _, A, _ = kvo.decode(np64(q), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"], 0.125, w, 0.97)
    assert (np.isnan(np64(o)) == np.isnan(O)).all() and (np.isnan(np64(lse)) == np.isnan(LSE)).all()
    worst = (64 + 8) * 2.0 ** -23 * np.nanmax(np.where(np.isfinite(A), A, 0)) + 2.0 ** -20
    got = out.cpu().numpy()
    for b, L in enumerate(lens):
        assert (np.isnan(got[b, :, :L]) == np.isnan(W[b])).all(), f"sequence {b}"
        some = ~np.isnan(W[b])
        tol = (2 * worst + 2.0 ** -20) * np.abs(W[b]) + 2.0 ** -40
        assert (np.abs(got[b, :, :L] - W[b])[some] <= tol[some]).all(), f"sequence {b}"
        assert (got[b, :, L:] == -7.0).all()
    if what != "key":  # the newest token is seen by the last query token alone
        assert not np.isnan(got[0, 0, lens[0] - 1]) and np.isnan(got[0, 0, :lens[0] - ql + 1]).all()


# ------------------------------------------------------------------ one rounding

def _tie_scales(values):
    """Pairs of one of `values` and a scale whose product is next to the middle of two e4m3 values, nearer
    than fp32 can tell: rounded to fp32 it is the middle."""
    mid = (kvo.E4M3[8:126] + kvo.E4M3[9:127]) / 2
    mid = mid[(mid > 1) & (mid < 4)]
    x, t = (a.ravel() for a in np.meshgrid(np.asarray(values, dtype=np.float64), mid))
    s = (t / x).astype(np.float32)
    p = x * s.astype(np.float64)
    good = (p != t) & (p.astype(np.float32) == t.astype(np.float32)) & (s < 2)
    assert good.sum() > 20
    return x[good], s[good]


def _tie_cache(c, rng, block):
    """Codes and scales of the cache replaced by ones whose values lie next to e4m3's middles."""
    x, s = _tie_scales(kvo.E4M3[56:64])
    code = {float(v): i for i, v in enumerate(kvo.E4M3)}
    codes = np.array([code[float(v)] for v in x], dtype=np.uint8)
    for n, sc in (("kc", "ks"), ("vc", "vs")):
        pick = rng.integers(0, len(s), c[sc].shape)
        c[sc][:] = s[pick]
        hit = np.repeat(codes[pick], block, 1)[..., None] | (rng.integers(0, 2, c[n].shape).astype(np.uint8) << 7)
        low = rng.integers(0, 80, c[n].shape).astype(np.uint8)
        c[n][:] = np.where(rng.random(c[n].shape) < 0.5, hit, low)


def _evict_equals(c, keep, first=0, recent=0, what=""):
    lens, P = c["lens"], c["P"]
    B, width = len(lens), -(-keep // P)
    w = c["rng"].random((B, c["H"], c["cap"])).astype(np.float32)
    new = np.full((B, width), -1, dtype=np.int32)
    at = 0
    for b, L in enumerate(lens):
        n = -(-min(int(L), keep) // P)
        new[b, :n] = c["free"][at:at + n]
        at += n
    g = _gpu(c)
    kept, nl, nw = jfa.jfa_cache_evict_fp8(*_cache(g), torch.from_numpy(w).cuda(), keep, torch.from_numpy(new).cuda(),
                                           first=first, recent=recent, check=True)
    k2, l2, w2 = kvo.evict(c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, w, keep, new, first, recent)
    assert (kept.cpu().numpy() == k2).all() and (nl.cpu().numpy() == l2).all() and (nw.cpu().numpy() == w2).all()
    for x in ("ks", "vs"):
        assert (g[x].cpu().numpy() == c[x]).all(), f"{what}: {x}"
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), f"{what}: {x}"


LAYOUTS = [(128, 16, 16), (64, 16, 8), (128, 1, 1), (64, 24, 8), (128, 128, 64)]


@pytest.mark.parametrize("d,P,block", LAYOUTS)
def test_evict_scales_that_are_no_powers_of_two(d, P, block):
    c = _case(41, [300, 40, 7, 129], 2, d, P, block, spare=300)
    for x in ("ks", "vs"):
        c[x] *= c["rng"].uniform(0.5, 1.5, c[x].shape).astype(np.float32)
    _evict_equals(c, 90, 2, 5)


@pytest.mark.parametrize("d,P,block", LAYOUTS)
def test_evict_rounds_once(d, P, block):
    """Values a hair from the middle of two e4m3 values at the new scale go to the nearer one."""
    c = _case(42, [300, 40, 7, 129], 2, d, P, block, spare=300)
    _tie_cache(c, c["rng"], block)
    _evict_equals(c, 90, 2, 5)


@pytest.mark.parametrize("powers", [15, 16, 17, 20])
@pytest.mark.parametrize("odd", [False, True])
def test_evict_tiny_codes_under_large_scales(powers, odd):
    """Blocks of which only the smallest codes are in use, or none, get a scale up to 2^17 times smaller."""
    c = _case(43, [300, 77], 2, 64, 16, 8, spare=300)
    rng = c["rng"]
    top = 8 >> max(0, powers - 14)  # codes 1 .. 7: e4m3's subnormals
    for n, sc in (("kc", "ks"), ("vc", "vs")):
        c[n][:] = rng.integers(0, top + 1, c[n].shape) | (rng.integers(0, 2, c[n].shape) << 7)
        c[sc][:] = 2.0 ** rng.integers(-3, 4, c[sc].shape)
        if odd:
            c[sc] *= rng.uniform(0.5, 1.5, c[sc].shape).astype(np.float32)
    _evict_equals(c, 61, 1, 3)


@pytest.mark.parametrize("e", [118, 119, 120, 121, 127])
@pytest.mark.parametrize("odd", [False, True])
def test_evict_largest_scales(e, odd):
    """Values past fp32's largest number, which a code and its scale can hold, keep their size."""
    c = _case(44, [100, 33], 2, 64, 16, 8, spare=30)
    rng = c["rng"]
    for sc in ("ks", "vs"):
        c[sc][:] = 2.0 ** rng.integers(e - 3, e + 1, c[sc].shape)
        if odd:
            c[sc] *= rng.uniform(0.5, 1.0, c[sc].shape).astype(np.float32)
    _evict_equals(c, 40, 2, 5)


def _append_equals(c, old, new, k, v):
    lens = [a + b for a, b in zip(old, new)]
    assert list(c["lens"]) == lens
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), max(new), check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs)
    for x in ("ks", "vs"):
        assert (g[x].cpu().numpy() == c[x]).all(), x
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x


# a warp a scale block with 16 or 32 rows, and chunks
GROWN = [(128, 16, 16, [5, 1, 15, 8, 20], [1, 2, 1, 3, 5]), (64, 32, 32, [5, 1, 31, 8, 40], [20, 21, 1, 30, 22]),
         (128, 128, 128, [5, 100, 127, 64, 200], [60, 1, 1, 300, 40]), (64, 24, 8, [3, 1, 7, 12, 20], [40, 1, 1, 2, 30])]


@pytest.mark.parametrize("d,P,block,old,new", GROWN)
@pytest.mark.parametrize("growth", [2.0, 4.0])
def test_append_rewrites_older_codes_with_one_rounding(d, P, block, old, new, growth):
    """Older codes under a scale that is no power of two and grows two- to eightfold."""
    c = _case(45, [a + b for a, b in zip(old, new)], 3, d, P, block)
    _tie_cache(c, c["rng"], block)
    n = sum(new)
    k, v = (_bf16(c["rng"], n, 3, d) for _ in range(2))
    at = 0
    for m in new:  # every sequence's first new token sets the scale
        k[at, :, 0] = v[at, :, d - 1] = 448 * growth
        at += m
    _append_equals(c, old, new, k, v)


@pytest.mark.parametrize("d,P,block,old,new", GROWN)
@pytest.mark.parametrize("odd", [1.0, 1.5])
def test_append_rewrites_the_largest_older_codes(d, P, block, old, new, odd):
    """Older values at the end of bf16's range, under scales of 2^118 to 1.5 * 2^119 that grow to 2^120."""
    c = _case(46, [a + b for a, b in zip(old, new)], 2, d, P, block)
    for x in ("ks", "vs"):
        c[x][:] = np.float32(odd) * np.exp2(c["rng"].integers(118, 120, c[x].shape)).astype(np.float32)
    n = sum(new)
    k, v = (_bf16(c["rng"], n, 2, d) for _ in range(2))
    k[:, :, 1] = v[:, :, 2] = 3.38e38
    _append_equals(c, old, new, k, v)


@pytest.mark.parametrize("d,P,block,old,new", GROWN)
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -125, 2.0 ** 126, 2.0 ** 127, 1.5 * 2.0 ** -126, 1.5 * 2.0 ** 126])
def test_append_behind_the_smallest_and_largest_scales(d, P, block, old, new, scale):
    """New values of the scale's own size, which keep it, and much smaller ones."""
    c = _case(50, [a + b for a, b in zip(old, new)], 2, d, P, block)
    c["ks"][:] = c["vs"][:] = scale
    n = sum(new)
    size = 2.0 ** c["rng"].integers(-12, 1, (n, 2, 1)) * min(scale * 100, 2.0 ** 125)
    k, v = ((_bf16(c["rng"], n, 2, d).double() * torch.from_numpy(size)).to(torch.bfloat16) for _ in range(2))
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    _append_equals(c, old, new, k, v)


@pytest.mark.parametrize("d,P,block,old,new", GROWN)
def test_append_new_codes_with_one_rounding(d, P, block, old, new):
    """New values whose quotient by an older scale, no power of two, is a hair from the middle of two codes."""
    c = _case(47, [a + b for a, b in zip(old, new)], 3, d, P, block)
    rng = c["rng"]
    values = (1 + np.arange(128) / 128.0)[3::7]  # bf16
    mid = (kvo.E4M3[8:126] + kvo.E4M3[9:127]) / 2
    mid = mid[(mid > 1) & (mid < 4)]
    x, t = (a.ravel() for a in np.meshgrid(values, mid))
    s = (x / t).astype(np.float32)
    y = x / s.astype(np.float64)
    good = (y != t) & ((x.astype(np.float32) / s) == t.astype(np.float32))
    x, s = x[good], s[good]
    assert len(x) > 100
    n, H = sum(new), 3
    k, v = (torch.zeros(n, H, d) for _ in range(2))
    for y, sc in ((k, "ks"), (v, "vs")):
        at = 0
        for b, m in enumerate(new):
            f = old[b]
            page, cell = c["table"][b, f // P], f % P // block
            for h in range(H):
                i = rng.integers(0, len(x))
                c[sc][page, cell, h] = s[i]
                y[at:at + m, h] = torch.from_numpy(x[i] * rng.choice([1.0, -1.0, 0.5, 2.0, 64.0], (m, d))).float()
            at += m
    _append_equals(c, old, new, k.to(torch.bfloat16), v.to(torch.bfloat16))


# ------------------------------------------------------------------ scales at both ends

@pytest.mark.parametrize("ks,q_size", [(126, -122), (127, -120), (-126, 120), (100, -98)])
@pytest.mark.parametrize("vs", [126, 120, -126])
@pytest.mark.parametrize("lens,ql", [([33, 4000], 1), ([1203], 4)])
def test_decode_largest_and_smallest_scales(ks, q_size, vs, lens, ql):
    """Keys and queries whose product is of usual size, values near fp32's ends: small codes, so that O is a bf16."""
    c = _case(51, lens, 1, 128, 16, 16)
    for n in ("kc", "vc"):
        c[n][:] = c["rng"].integers(0, 49, c[n].shape) | (c["rng"].integers(0, 2, c[n].shape) << 7)
    c["ks"][:], c["vs"][:] = 2.0 ** ks, 2.0 ** vs
    q = (_bf16(c["rng"], len(lens), ql, 4, 128).double() * 2.0 ** q_size).to(torch.bfloat16)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(_gpu(c)), scale=0.25, check=True)
    check_decode(c, q, o, lse, 0.25, what="ends")


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("B,H,block", [(40, 2, 16), (40, 2, 8), (3, 40, 128)])
def test_append_with_a_loose_bound_on_new_tokens(B, H, block):
    """max_new is a bound: one that is far above every sequence's count changes nothing."""
    rng = np.random.default_rng(48)
    old, new = rng.integers(0, 40, B), rng.integers(0, 30, B)
    lens = [int(a + b) for a, b in zip(old, new)]
    c = _case(48, lens, H, 64, 128, block)
    n = int(new.sum())
    k, v = _bf16(rng, n, H, 64), _bf16(rng, n, H, 64)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), 2 ** 31 - 1, check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs)
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x
    assert (g["ks"].cpu().numpy() == c["ks"]).all() and (g["vs"].cpu().numpy() == c["vs"]).all()


# ------------------------------------------------------------------ the same again

@pytest.mark.parametrize("lens,Hkv,G,ql,d", [([3000, 1, 0, 700], 2, 4, 1, 128), ([5000], 1, 4, 4, 64),
                                             ([40000] + [300] * 70, 1, 8, 1, 128)])
def test_decode_repeats_itself(lens, Hkv, G, ql, d):
    """The same inputs give the same bits, whatever the workspace held before."""
    c = _case(49, lens, Hkv, d, 16, 16)
    g, q = _gpu(c), _bf16(c["rng"], len(lens), ql, Hkv * G, d).cuda()
    w = torch.from_numpy(c["rng"].random((len(lens), Hkv, c["cap"])).astype(np.float32)).cuda()
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    runs = []
    for fill in (0, 0xA5, 0xFF):
        ws.fill_(fill)
        out = torch.zeros_like(w)
        runs.append((*jfa.jfa_decode_fp8(q, *_cache(g), weights=w, weights_out=out, workspace=ws, check=True), out))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
