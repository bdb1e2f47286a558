"""GPU parity of the 8-bit paged cache: append, decode with attention weights, evict.

Append and evict are compared with the fp64 oracle bit for bit (codes, scales,
positions, weights and every byte they must leave alone). The decode's tolerances
are derived per output row from the arithmetic, with u = 2^-24:
  * a score is a sum of d products, exact in fp16 x fp16 -> fp32, added in fp32
    (an addition may truncate: 2^-23 of the running magnitude), then scaled by a
    few rounded factors: |ds| <= (d + 8) 2^-23 A + 2^-20, A = max_j scale sum_d
    |q_d k_jd|; the constant covers the approximate exponential and logarithm
    (2^-21 each, absolute in the exponent);
  * LSE moves by at most the scores' error, plus its own few roundings;
  * O: weights carry the scores' error twice (numerator, denominator) and one
    rounding to fp16, half a step 2^-11; the sum and the joins of the parts add
    far less than 2^-13 together; the bf16 result rounds by half a step 2^-8:
    |dO| <= (2^-11 + 2^-13 + 2 |ds|) sum_j P_j |v_j| + 2^-8 |O|. That half step is
    relative down to fp16's smallest normal number; below it is 2^-25 absolute. A
    weight is held as w_j = P_j vs_j / r with r at most 2^-7 of the largest P_j vs_j
    (vs: the scale of the value's block), so a key adds at most 2^-25 * 448 * r <=
    2^-32 * 448 * max_j P_j vs_j more, and all L keys L times that. bf16's own half
    step is likewise 2^-134 absolute below its smallest normal number 2^-126;
  * a token's weight, in fp32: (2 |ds| + 2^-20) of itself.
"""
import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import kv_cache as kvo
from tests.parity import np64

pytestmark = pytest.mark.gpu


def _case(seed, lens, H, d, P, block, cap_pages=None, spread=3, spare=3):
    """A filled cache and a batch over it, on the host. Slots past the lengths and
    pages of nobody hold NaN codes, table entries of no use are out of range."""
    rng = np.random.default_rng(seed)
    need = [-(-L // P) for L in lens]
    pages = sum(need) + spare
    mp = max(max(need, default=0), 1) if cap_pages is None else cap_pages
    perm = rng.permutation(pages)
    table = np.full((len(lens), mp), 2 ** 30, dtype=np.int32)
    live = np.zeros((pages, P), dtype=bool)
    at = 0
    for b, L in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        t = np.arange(L)
        live[table[b][t // P], t % P] = True

    def fill():
        x = rng.standard_normal((pages, P, H, d)) * np.exp(spread * rng.standard_normal((pages, P, H, 1)) / 3)
        sc = np.empty((pages, P // block, H), dtype=np.float32)
        a = np.abs(x).reshape(pages, P // block, block, H, d).max((2, 4))
        sc[:] = 2.0 ** np.ceil(np.log2(a / 448.0))
        codes = kvo.e4m3_encode(np.clip(x / np.repeat(sc, block, 1)[..., None], -448, 448))
        codes[~live] = 0x7F
        return codes, sc
    kc, ks = fill()
    vc, vs = fill()
    return dict(kc=kc, vc=vc, ks=ks, vs=vs, table=table, lens=np.array(lens, dtype=np.int32), rng=rng, P=P, H=H, d=d,
                free=perm[at:], cap=mp * P)


def _gpu(c):
    return {n: torch.from_numpy(c[n].copy()).cuda() for n in ("kc", "vc", "ks", "vs", "table", "lens")}


def _cache(g):
    return g["kc"], g["vc"], g["ks"], g["vs"], g["table"], g["lens"]


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def _same_codes(a, b):
    """Equal codes; any NaN equals any NaN."""
    return bool(((a == b) | ((a & 0x7F == 0x7F) & (b & 0x7F == 0x7F))).all())


def check_decode(c, q, o, lse, scale, w_in=None, w_out=None, w_was=None, decay=1.0, what=""):
    O, LSE, W, absO, A, top = kvo.decode(np64(q), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"], scale,
                                    w_in, decay)
    ds = (c["d"] + 8) * 2.0 ** -23 * A + 2.0 ** -20
    o, lse = np64(o), np64(lse)
    bound = (2.0 ** -11 + 2.0 ** -13 + 2 * ds)[..., None] * absO + 2.0 ** -8 * np.abs(O) + \
        (448 * 2.0 ** -32 * top)[..., None] + 2.0 ** -134
    assert (np.isnan(o) == np.isnan(O)).all(), what
    bad = ~(np.abs(o - O) <= bound) & ~np.isnan(O)
    assert not bad.any(), f"{what}: O off by {np.nanmax(np.abs(o - O) - bound):.3e} over its bound at {np.argwhere(bad)[:3]}"
    none = np.isneginf(LSE)
    assert (np.isneginf(lse) == none).all() and (o[none] == 0).all(), what
    with np.errstate(invalid="ignore"):
        e = np.abs(lse - LSE)
    ok = none | np.isnan(LSE) | (e <= ds + (np.abs(LSE) + 1) * 2.0 ** -21)
    assert ok.all(), f"{what}: LSE {e[~ok].max():.3e}"
    if w_out is not None:
        got = w_out.cpu().numpy()
        worst = ds.max(initial=0.0)
        for b, w in enumerate(W):
            L = w.shape[1]
            tol = (2 * worst + 2.0 ** -20) * np.abs(w) + 2.0 ** -40
            assert (np.abs(got[b, :, :L] - w) <= tol).all(), f"{what}: weights of sequence {b}"
            assert (got[b, :, L:] == w_was[b, :, L:]).all(), f"{what}: weights past the end of sequence {b}"


LENS = [0, 1, 2, 15, 16, 17, 33, 100, 777, 1500]


@pytest.mark.parametrize("Hq,Hkv,q_len", [(8, 2, 1), (8, 2, 2), (7, 1, 1), (3, 3, 1), (3, 3, 5), (16, 1, 1), (6, 2, 4)])
@pytest.mark.parametrize("d,P,block", [(128, 16, 16), (64, 16, 8), (128, 1, 1), (64, 24, 8), (128, 128, 128)])
def test_decode_ragged(Hq, Hkv, q_len, d, P, block):
    c = _case(1, LENS, Hkv, d, P, block)
    g = _gpu(c)
    q = _bf16(c["rng"], len(LENS), q_len, Hq, d)
    w = c["rng"].random((len(LENS), Hkv, c["cap"])).astype(np.float32)
    was = np.full_like(w, -7.0)
    w_out = torch.from_numpy(was).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.3, weights=torch.from_numpy(w).cuda(), decay=0.75,
                                weights_out=w_out, check=True)
    check_decode(c, q, o, lse, 0.3, w, w_out, was, 0.75, "weights")
    # without the weights: the same O and LSE, bit for bit
    o2, lse2 = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.3, check=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    # in place, and as plain sums
    w1 = torch.from_numpy(w).cuda()
    jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.3, weights=w1, decay=0.75, check=True)
    w2 = torch.zeros_like(w1)
    jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.3, weights_out=w2, check=True)
    for b, L in enumerate(LENS):
        assert torch.equal(w1[b, :, :L], w_out[b, :, :L])
        assert torch.allclose(w2[b, :, :L], w_out[b, :, :L] - 0.75 * torch.from_numpy(w[b, :, :L]).cuda(), atol=3e-7)
        assert (w2[b, :, L:] == 0).all()


@pytest.mark.parametrize("lens", [[40000], [1], [0], [0, 0, 9000, 0, 3, 20000], [7] * 300])
def test_decode_cut_and_joined(lens):
    """One long sequence over all the SMs, parts that end inside segments, many short ones."""
    c = _case(2, lens, 2, 128, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], len(lens), 1, 8, 128)
    w = torch.zeros(len(lens), 2, c["cap"]).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights_out=w, check=True)
    check_decode(c, q, o, lse, 128 ** -0.5, None, w, np.zeros(w.shape, dtype=np.float32), what=str(lens)[:30])
    for b, L in enumerate(lens):  # every head's weights sum to the four query heads of its group
        if L:
            assert torch.allclose(w[b].double().sum(-1), torch.full((2,), 4.0, device="cuda").double(), atol=1e-4)


@pytest.mark.parametrize("B", [31, 513, 700])
def test_decode_many_sequences(B):
    """Past 512 sequences one kernel numbers the tiles for all blocks of the next."""
    lens = [int(x) for x in np.random.default_rng(20).integers(0, 60, B)]
    c = _case(20, lens, 1, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], B, 2, 4, 64)
    w = torch.zeros(B, 1, c["cap"]).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights_out=w, check=True)
    check_decode(c, q, o, lse, 64 ** -0.5, None, w, np.zeros(w.shape, dtype=np.float32), what=f"B={B}")
    g["lens"][B - 1] = -1
    with pytest.raises(jfa.JfaError, match="inconsistent device input"):
        jfa.jfa_decode_fp8(q.cuda(), *_cache(g), check=True)


@pytest.mark.parametrize("B", [90, 512, 2100])
def test_decode_padded_batch(B):
    """Few sequences in use among many empty ones, at the ends and far apart: parts cross long runs of nothing."""
    lens = [0] * B
    for b, L in ((0, 700), (1, 33), (B // 3, 1900), (B // 3 + 40, 16), (B - 2, 5000), (B - 1, 1)):
        lens[b] = L
    c = _case(31, lens, 2, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], B, 1, 6, 64)
    w = torch.zeros(B, 2, c["cap"]).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights_out=w, check=True)
    check_decode(c, q, o, lse, 64 ** -0.5, None, w, np.zeros(w.shape, dtype=np.float32), what=f"B={B}")


@pytest.mark.parametrize("H,lens", [(40, [700, 3]), (2700, [20, 0, 35])])
def test_decode_many_heads(H, lens):
    """More heads than a part's warps, and than all warps."""
    c = _case(21, lens, H, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], len(lens), 1, H, 64)
    w = torch.zeros(len(lens), H, c["cap"]).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights_out=w, check=True)
    check_decode(c, q, o, lse, 0.125, None, w, np.zeros(w.shape, dtype=np.float32), what=f"H={H}")


def test_decode_one_long_among_short():
    """One sequence cut into more than 64 parts in a batch whose rows a warp each joins."""
    lens = [30000] + [20] * 19
    c = _case(22, lens, 1, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], len(lens), 1, 5, 64)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), check=True)
    check_decode(c, q, o, lse, 0.125, what="one long")


@pytest.mark.parametrize("lens,Hq,Hkv,q_len,d", [
    ([30] * 50 + [20000] + [20] * 39, 4, 1, 4, 128),     # thousands of parts: the weights behind the join
    ([9, 16000] + [20] * 12, 16, 4, 3, 64),              # hundreds: beside it
    ([12000, 0, 15, 14000] + [0, 33] * 10, 16, 8, 2, 128),
    ([9000] + [0] * 598 + [7000], 6, 2, 1, 64),          # numbered by a kernel of its own
])
def test_decode_weights_of_long_sequences_among_short(lens, Hq, Hkv, q_len, d):
    c = _case(35, lens, Hkv, d, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], len(lens), q_len, Hq, d)
    w = c["rng"].random((len(lens), Hkv, c["cap"])).astype(np.float32)
    out = torch.from_numpy(w).cuda()
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights=out, decay=0.5, check=True)
    check_decode(c, q, o, lse, d ** -0.5, w, out, w, 0.5, what="long among short")
    o2, lse2 = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), check=True)
    again = torch.from_numpy(w).cuda()
    o3, lse3 = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), weights=again, decay=0.5, check=True)
    assert torch.equal(o, o3) and torch.equal(lse, lse3) and torch.equal(out, again)  # the same, whatever ran first
    check_decode(c, q, o2, lse2, d ** -0.5, what="without weights")


def test_decode_shared_pages():
    """Sequences that share a prefix's pages, and a sequence that holds a page twice."""
    c = _case(23, [64, 64, 100], 2, 64, 16, 8)
    c["table"][1, :3] = c["table"][0, :3]
    c["table"][2, 4] = c["table"][2, 1]
    g = _gpu(c)
    q = _bf16(c["rng"], 3, 2, 6, 64)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), check=True)
    check_decode(c, q, o, lse, 0.125, what="shared")


def test_decode_scales_of_every_size():
    """Blocks of very different magnitude, blocks of zeros, and scales that are no powers of two."""
    c = _case(3, [500, 64, 1000], 2, 128, 16, 16)
    rng = c["rng"]
    c["vs"] *= (2.0 ** rng.integers(-30, 30, c["vs"].shape)).astype(np.float32)
    c["ks"] *= rng.uniform(0.5, 1.5, c["ks"].shape).astype(np.float32)
    c["vs"] *= rng.uniform(0.5, 1.5, c["vs"].shape).astype(np.float32)
    zero = c["table"][0, 3]
    c["vc"][zero], c["vs"][zero] = 0, 2.0 ** -126
    c["kc"][c["table"][2, 5]], c["ks"][c["table"][2, 5]] = 0, 2.0 ** -126
    q = _bf16(rng, 3, 2, 8, 128)
    q[1] *= 2.0 ** 40   # row scaling of Q: the scores of tiny keys
    c["ks"][c["table"][1, :4]] *= np.float32(2.0 ** -40)
    q[2] *= 2.0 ** -30
    g = _gpu(c)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.2, check=True)
    check_decode(c, q, o, lse, 0.2, what="scales")


def test_decode_of_the_smallest_values():
    """Values near fp32's smallest normal number keep their size (fp32 outputs of the parts, bf16 O)."""
    c = _case(26, [33, 4000], 1, 128, 16, 16)
    c["vs"][:] = 2.0 ** -126
    c["vs"][c["table"][1, 100]] = 2.0 ** -120
    g = _gpu(c)
    q = _bf16(c["rng"], 2, 1, 4, 128)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), check=True)
    check_decode(c, q, o, lse, 128 ** -0.5, what="small")
    assert (o != 0).float().mean() > 0.99


def test_decode_records_events_around_its_main_kernel():
    c = _case(27, [3000], 2, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], 1, 1, 8, 64).cuda()
    ev = (torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True))
    o, lse = jfa.jfa_decode_fp8(q, *_cache(g), events=ev, check=True)
    assert 0 < ev[0].elapsed_time(ev[1]) < 1000
    o2, lse2 = jfa.jfa_decode_fp8(q, *_cache(g), check=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_few_keys_dominate():
    """Sharp rows: the reference maximum moves far and often, most weights vanish."""
    c = _case(4, [3000, 700], 1, 64, 16, 4)
    q = (_bf16(c["rng"], 2, 1, 8, 64).float() * 20).to(torch.bfloat16)
    g = _gpu(c)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.5, check=True)
    check_decode(c, q, o, lse, 0.5, what="sharp")


def test_decode_nan_reaches_only_the_rows_that_see_it():
    lens, ql = [40, 5, 70], 4
    c = _case(5, lens, 2, 64, 16, 16)
    t = lens[0] - 2  # seen by the last two query tokens of sequence 0 only
    c["vc"][c["table"][0, t // 16], t % 16, 1, 7] = 0xFF
    t = lens[2] - 1
    c["kc"][c["table"][2, t // 16], t % 16, 0, 3] = 0x7F
    c["vc"][c["table"][1, 0], 0, 0, 63] = 0x7F  # seen by every query token of sequence 1 that sees anything
    g = _gpu(c)
    q = _bf16(c["rng"], 3, ql, 8, 64)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(g), scale=0.125, check=True)
    check_decode(c, q, o, lse, 0.125, what="NaN")
    n = torch.isnan(o.float()).cpu()
    assert n[0, :2].sum() == 0 and n[0, 2:, 4:, 7].all() and n[0, :, :4].sum() == 0
    assert n[2, 3, :4].all() and n[2, :3].sum() == 0 and n[1, :, :4, 63].all()


def test_decode_past_32_bit_offsets():
    """A cache of more than 2^32 bytes a tensor, its last pages in use."""
    P, H, d = 128, 8, 128
    pages = (1 << 32) // (P * H * d) + 40
    kc = torch.full((pages, P, H, d), 0x7F, dtype=torch.uint8, device="cuda")
    vc = torch.full_like(kc, 0x7F)
    ks = torch.full((pages, 2, H), 2.0 ** -8, device="cuda")
    vs = torch.full_like(ks, 2.0 ** -7)
    rng = np.random.default_rng(6)
    use = [pages - 1, 0, pages - 17]
    L = 300
    small = rng.integers(0, 120, (2, 3, P, H, d)).astype(np.uint8)
    for i, pg in enumerate(use):
        kc[pg], vc[pg] = torch.from_numpy(small[0, i]).cuda(), torch.from_numpy(small[1, i]).cuda()
    table = torch.tensor([use], dtype=torch.int32, device="cuda")
    lens = torch.tensor([L], dtype=torch.int32, device="cuda")
    q = _bf16(rng, 1, 1, 16, d)
    o, lse = jfa.jfa_decode_fp8(q.cuda(), kc, vc, ks, vs, table, lens, check=True)
    c = dict(kc=small[0], vc=small[1], ks=np.full((3, 2, H), 2.0 ** -8, dtype=np.float32),
             vs=np.full((3, 2, H), 2.0 ** -7, dtype=np.float32), table=np.array([[0, 1, 2]]), lens=[L], d=d)
    check_decode(c, q, o, lse, d ** -0.5, what="far pages")
    # append there, and evict into the last page of all
    k, v = _bf16(rng, 70, H, d), _bf16(rng, 70, H, d)
    lens += 70
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), kc, vc, ks, vs, table, lens, torch.tensor([0, 70], dtype=torch.int32,
                             device="cuda"), 70, check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [L + 70], [0, 70])
    for i, pg in enumerate(use):
        assert _same_codes(kc[pg].cpu().numpy(), c["kc"][i]) and (vs[pg].cpu().numpy() == c["vs"][i]).all()
    w = rng.random((1, H, 3 * P)).astype(np.float32)
    fresh = pages - 2
    jfa.jfa_cache_evict_fp8(kc, vc, ks, vs, table, lens, torch.from_numpy(w).cuda(), 100,
                            torch.tensor([[fresh]], dtype=torch.int32, device="cuda"), check=True)
    for n in ("kc", "vc", "ks", "vs"):
        c[n] = np.concatenate([c[n], c[n][:1]])
    kvo.evict(c["kc"], c["vc"], c["ks"], c["vs"], c["table"], [L + 70], w, 100, np.array([[3]]))
    assert _same_codes(vc[fresh, :100].cpu().numpy(), c["vc"][3, :100])
    assert (ks[fresh].cpu().numpy() == c["ks"][3]).all()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("d,P,block", [(128, 16, 16), (64, 16, 8), (128, 1, 1), (64, 7, 1), (64, 24, 8),
                                       (128, 128, 128), (64, 128, 64)])
@pytest.mark.parametrize("old,new", [([0, 5, 16, 130, 300, 9], [1, 1, 1, 1, 1, 0]),
                                     ([0, 0, 3, 127, 128, 250], [0, 300, 125, 1, 129, 40])])
def test_append(d, P, block, old, new):
    lens = [a + b for a, b in zip(old, new)]
    c = _case(7, lens, 3, d, P, block)
    rng = c["rng"]
    n = sum(new)
    k, v = (_bf16(rng, n, 3, d) * (2.0 ** torch.from_numpy(rng.integers(-12, 12, (n, 3, 1)))) for _ in range(2))
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    k[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0])
    v[n // 2] = 0
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    w = rng.random((len(lens), 3, c["cap"])).astype(np.float32)
    g, gw = _gpu(c), torch.from_numpy(w.copy()).cuda()
    got = jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), max(new), weights=gw,
                                   check=True)
    assert got[0] is g["kc"] and got[3] is g["vs"]
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs, w)
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x
    for x in ("ks", "vs"):
        assert (g[x].cpu().numpy() == c[x]).all(), x
    assert (gw.cpu().numpy() == w).all()


@pytest.mark.parametrize("B,new_hi", [(200, 3), (150, 400), (40, 700)])
def test_append_many_sequences(B, new_hi):
    """Scale blocks with a fixed number each, and runs found in the offsets."""
    rng = np.random.default_rng(24)
    old, new = rng.integers(0, 40, B), rng.integers(0, new_hi + 1, B)
    new[3] = new_hi
    lens = [int(a + b) for a, b in zip(old, new)]
    c = _case(24, lens, 1, 64, 16, 8)
    n = int(new.sum())
    k, v = _bf16(rng, n, 1, 64), _bf16(rng, n, 1, 64)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), new_hi, check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs)
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x
    assert (g["ks"].cpu().numpy() == c["ks"]).all() and (g["vs"].cpu().numpy() == c["vs"]).all()


@pytest.mark.parametrize("d,P,block,old,new", [
    (128, 32, 32, [0, 5, 31, 32, 300, 9], [65, 1, 300, 32, 33, 0]),
    (64, 96, 32, [0, 5, 31, 32, 300, 9], [65, 1, 300, 32, 33, 0]),
    (128, 128, 128, [0, 120, 127, 128, 300, 9], [32, 17, 2, 31, 0, 25]),
    (64, 128, 64, [0, 60, 63, 64, 300, 9], [17, 17, 17, 17, 1, 16]),
    (128, 16, 16, [0, 15, 16, 1, 300, 9], [16, 2, 15, 17, 0, 400]),
    (64, 8, 2, [0, 1, 2, 3, 300, 9], [16, 2, 15, 1, 0, 3]),
    (128, 64, 64, [0, 60, 63, 64, 300, 9], [200, 1, 129, 64, 0, 65]),
])
def test_append_behind_scales_of_every_kind(d, P, block, old, new):
    """Every number of rows a warp holds, and chunks, behind blocks whose scale is larger or smaller."""
    lens = [a + b for a, b in zip(old, new)]
    c = _case(32, lens, 2, d, P, block)
    rng = c["rng"]
    for x in ("ks", "vs"):
        c[x][:] = rng.choice(np.float32([2.0 ** -20, 2.0 ** -9, 2.0 ** -6, 0.25, 4.0]), c[x].shape)
    n = sum(new)
    k, v = (_bf16(rng, n, 2, d) for _ in range(2))
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), max(new), check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs)
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x
    assert (g["ks"].cpu().numpy() == c["ks"]).all() and (g["vs"].cpu().numpy() == c["vs"]).all()


@pytest.mark.parametrize("d,P,block,new", [(128, 32, 32, 20), (64, 64, 64, 50), (128, 128, 128, 9)])
def test_append_at_a_scale_that_is_no_power_of_two(d, P, block, new):
    """A caller's scale of 0.3 has room for the new values (below 0.3 * 448) and stays. A code is then off by half
    a step, 2^-4 of the value or 2^-10 of the scale, and the quotient's own rounding to fp32, 2^-24 of it."""
    old = block - 3
    c = _case(34, [old + new], 2, d, P, block)
    c["ks"][:] = c["vs"][:] = 0.3
    k, v = _bf16(c["rng"], new, 2, d), _bf16(c["rng"], new, 2, d)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.tensor([0, new], dtype=torch.int32).cuda(), new,
                             check=True)
    first = c["table"][0, old // P]
    for x, sc, y in (("kc", "ks", k), ("vc", "vs", v)):
        s = np.float64(np.float32(0.3))
        assert (g[sc][first].cpu().numpy()[-1] == np.float32(0.3)).all()
        got = kvo.e4m3_decode(g[x][first, P - 3:].cpu().numpy()) * s
        want = np64(y)[:3]
        assert (np.abs(got - want) <= 2.0 ** -4 * (1 + 2.0 ** -20) * np.abs(want) + 2.0 ** -10 * s).all()


@pytest.mark.parametrize("B,long,block", [(1100, 500, 16), (1100, 500, 8), (33, 129, 64), (600, 32, 128)])
def test_append_one_prompt_among_steps(B, long, block):
    """One long run of new tokens among sequences that get one or none: its place is found in the offsets."""
    rng = np.random.default_rng(33)
    old, new = rng.integers(0, 40, B), rng.integers(0, 2, B)
    new[B // 2], new[B - 1] = long, min(long, 33)
    lens = [int(a + b) for a, b in zip(old, new)]
    c = _case(33, lens, 1, 64, 128, block)
    n = int(new.sum())
    k, v = _bf16(rng, n, 1, 64), _bf16(rng, n, 1, 64)
    offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), long, check=True)
    kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs)
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x
    assert (g["ks"].cpu().numpy() == c["ks"]).all() and (g["vs"].cpu().numpy() == c["vs"]).all()


def test_append_extreme_values():
    """Subnormal and largest bf16 values, and a caller's scale that is no power of two."""
    x = torch.tensor([2.0 ** -133, -2.0 ** -126, 3.3895e38, 448.0, 449.0, 1.0, -0.0, 2.0 ** -140]).to(torch.bfloat16)
    k = torch.stack([x.roll(i).repeat(8) * s for i, s in ((0, 1.0), (1, 0.0), (2, 1.0), (3, 2.0 ** -60))])
    k = k.to(torch.bfloat16)[:, None].repeat(1, 2, 1)
    v = torch.zeros_like(k)
    v[:, :, :7] = 2.0 ** -131
    c = _case(8, [4, 9], 2, 64, 8, 4)
    c["ks"][:], c["vs"][:] = 0.3, 0.7
    kk, vv = torch.cat([k, k[:3]]), torch.cat([v, k[:3]])
    offs = np.array([0, 4, 7], dtype=np.int32)  # sequence 1 appends behind six tokens at the scale 0.3
    g = _gpu(c)
    jfa.jfa_cache_append_fp8(kk.cuda(), vv.cuda(), *_cache(g), torch.from_numpy(offs).cuda(), 4, check=True)
    # the quotient by a scale that is no power of two is rounded to fp32 first
    ks, vs = c["ks"].copy(), c["vs"].copy()
    kvo.append(np64(kk), np64(vv), c["kc"], c["vc"], ks, vs, c["table"], [4, 9], offs)
    assert (g["ks"].cpu().numpy() == ks).all() and (g["vs"].cpu().numpy() == vs).all()
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x


# ------------------------------------------------------------------ evict

@pytest.mark.parametrize("d,P,block", [(128, 16, 16), (64, 16, 8), (128, 1, 1), (64, 24, 8), (128, 128, 128)])
@pytest.mark.parametrize("keep,first,recent", [(40, 4, 8), (1, 0, 0), (130, 0, 130), (257, 100, 0), (2000, 3, 3)])
def test_evict(d, P, block, keep, first, recent):
    _evict_case([0, 1, 40, 41, 500, 1300], 2, d, P, block, keep, first, recent)


@pytest.mark.parametrize("lens,H,d,P,block,keep", [
    ([0, 1, 40, 41, 500, 1300] + [90] * 34, 8, 128, 16, 16, 100),
    ([0, 30, 60, 61, 700, 9000] + [200] * 20, 8, 64, 24, 8, 61),
])
def test_evict_fills_the_card(lens, H, d, P, block, keep):
    """More (sequence, head) pairs than the card's SMs hold blocks for."""
    _evict_case(lens, H, d, P, block, keep, 2, 5)


@pytest.mark.parametrize("lens,H,d,P,block,keep,cap_pages", [
    ([0, 3, 200, 41, 500, 20000, 1300], 24, 64, 128, 32, 100, 1100),
    ([0, 3, 90, 41, 500, 1300] + [0] * 290 + [77, 0, 1, 300], 4, 64, 16, 16, 61, 700),
    ([700, 3, 90, 41, 500, 1300, 9000], 2, 128, 8, 8, 300, 4100),
])
def test_evict_of_short_sequences_in_wide_tables(lens, H, d, P, block, keep, cap_pages):
    """Rows of the page table far longer than most sequences, and batches mostly of empty ones."""
    _evict_case(lens, H, d, P, block, keep, 2, 5, cap_pages)


def _evict_case(lens, H, d, P, block, keep, first, recent, cap_pages=None):
    width = -(-keep // P)
    c = _case(9, lens, H, d, P, block, cap_pages, spare=width * len(lens) + 1)
    rng = c["rng"]
    w = np.exp(2 * rng.standard_normal((len(lens), H, c["cap"]))).astype(np.float32)
    w[rng.random(w.shape) < 0.3] = 0
    w[4, 0] = 1.0            # all equal: the lowest positions stay
    w[5, 1, 7:900:3] = np.nan
    w[5, 0, 20:40] = -1.0
    w[3, 0, :20] = np.inf
    w[3, 1, :41] = -0.0
    new = np.full((len(lens), width), -1, dtype=np.int32)
    used = [-(-min(L, keep) // P) for L in lens]
    at = 0
    for b, n in enumerate(used):
        new[b, :n] = c["free"][at:at + n]
        at += n
    g, gw = _gpu(c), torch.from_numpy(w).cuda()
    kept, nl, nw = jfa.jfa_cache_evict_fp8(*_cache(g), gw, keep, torch.from_numpy(new).cuda(), first=first,
                                           recent=recent, check=True)
    k2, l2, w2 = kvo.evict(c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, w, keep, new, first, recent)
    assert (kept.cpu().numpy() == k2).all() and (nl.cpu().numpy() == l2).all()
    assert np.array_equal(nw.cpu().numpy(), w2, equal_nan=True)
    for x in ("ks", "vs"):
        assert (g[x].cpu().numpy() == c[x]).all(), x
    for x in ("kc", "vc"):
        assert _same_codes(g[x].cpu().numpy(), c[x]), x


@pytest.mark.parametrize("L,keep", [(70001, 5000), (33333, 33000), (131072, 1), (5000, 77), (9001, 4000),
                                    (20000, 3), (200003, 40001), (140000, 139999)])
@pytest.mark.parametrize("ties", [2, 9])
def test_evict_long(L, keep, ties):
    """Selection over a long sequence (positions and weights; the rows move as above): every number of
    blocks and keys a thread, with ties at the border and without."""
    rng = np.random.default_rng(10)
    pages, P = -(-L // 128), 128
    fresh = -(-keep // P)
    kc = torch.zeros(pages + fresh, P, 1, 64, dtype=torch.uint8, device="cuda")
    ks = torch.ones(pages + fresh, 1, 1, device="cuda")
    w = np.round(np.abs(rng.standard_cauchy((1, 1, pages * P))), ties).astype(np.float32)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    new = torch.arange(pages, pages + fresh, dtype=torch.int32, device="cuda")[None]
    kept, nl, nw = jfa.jfa_cache_evict_fp8(kc, kc.clone(), ks, ks.clone(), table, torch.tensor([L], dtype=torch.int32,
                                           device="cuda"), torch.from_numpy(w).cuda(), keep, new, check=True)
    expect = np.sort(np.lexsort((np.arange(L), -w[0, 0, :L]))[:keep])
    assert (kept[0, 0].cpu().numpy() == expect).all() and int(nl[0]) == keep
    assert (nw[0, 0, :keep].cpu().numpy() == w[0, 0, expect]).all()


def test_evict_long_with_many_heads():
    """40 heads of one long sequence, eight blocks each, and the rows they keep."""
    L, keep, H = 70000, 1000, 40
    rng = np.random.default_rng(28)
    pages, fresh = -(-L // 128), -(-keep // 128)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc = torch.randint(0, 127, (pages + fresh, 128, H, 64), generator=g, device="cuda", dtype=torch.uint8)
    vc = torch.randint(0, 127, (pages + fresh, 128, H, 64), generator=g, device="cuda", dtype=torch.uint8)
    ks, vs = torch.ones(pages + fresh, 2, H, device="cuda"), torch.ones(pages + fresh, 2, H, device="cuda")
    w = rng.random((1, H, pages * 128)).astype(np.float32)
    table = torch.arange(pages + fresh, dtype=torch.int32, device="cuda")[None]
    kept, _, nw = jfa.jfa_cache_evict_fp8(kc, vc, ks, vs, table[:, :pages].contiguous(),
                                          torch.tensor([L], dtype=torch.int32, device="cuda"),
                                          torch.from_numpy(w).cuda(), keep, table[:, pages:].contiguous(), check=True)
    for h in range(H):
        expect = np.sort(np.lexsort((np.arange(L), -w[0, h, :L]))[:keep])
        assert (kept[0, h].cpu().numpy() == expect).all()
        assert (nw[0, h, :keep].cpu().numpy() == w[0, h, expect]).all()
        at = torch.from_numpy(expect).cuda()
        for c, sc in ((kc, ks), (vc, vs)):
            old = c.flatten(0, 1)[at, h].view(torch.float8_e4m3fn).float()
            new = c[pages:].flatten(0, 1)[:keep, h].view(torch.float8_e4m3fn).float()
            scale = sc[pages:].flatten(0, 1)[:, h].repeat_interleave(64)[:keep, None]
            assert torch.equal(old, new * scale)  # the new scale is at most 1: nothing is rounded


def test_evict_many_sequences_and_pages():
    """A warp checks a sequence past 15 of them; more pages than a bitmap holds are looked at in runs."""
    rng = np.random.default_rng(25)
    B, L, keep, pages = 20, 300, 50, 600_000
    table = rng.permutation(pages).astype(np.int32)[:B * (L + keep)].reshape(B, L + keep)
    src, new = np.ascontiguousarray(table[:, :L]), np.ascontiguousarray(table[:, L:])
    kc = torch.zeros(pages, 1, 1, 64, dtype=torch.uint8, device="cuda")
    ks = torch.ones(pages, 1, 1, device="cuda")
    codes = rng.integers(0, 127, (B, L, 64)).astype(np.uint8)
    kc[torch.from_numpy(src.ravel()).cuda().long(), 0, 0] = torch.from_numpy(codes.reshape(-1, 64)).cuda()
    w = rng.random((B, 1, L)).astype(np.float32)
    lens = torch.full((B,), L, dtype=torch.int32, device="cuda")

    def call(table, fresh):
        return jfa.jfa_cache_evict_fp8(kc, kc, ks, ks, torch.from_numpy(table).cuda(), lens, torch.from_numpy(w).cuda(),
                                       keep, torch.from_numpy(fresh).cuda(), check=True)
    kept = call(src, new)[0].cpu().numpy()[:, 0]
    got = kc[torch.from_numpy(new.ravel()).cuda().long(), 0, 0].cpu().numpy().reshape(B, keep, 64)
    scale = ks[torch.from_numpy(new.ravel()).cuda().long(), 0, 0].cpu().numpy().reshape(B, keep, 1)
    for b in range(B):
        expect = np.sort(np.lexsort((np.arange(L), -w[b, 0]))[:keep])
        assert (kept[b] == expect).all()
        assert (kvo.e4m3_decode(got[b]) * scale[b] == kvo.e4m3_decode(codes[b, expect])).all()
    for bad in (int(src[19, 299]), int(new[0, 0]), pages, -1):  # still held, given out twice, no page
        wrong = new.copy()
        wrong[17, 49] = bad
        with pytest.raises(jfa.JfaError, match="inconsistent device input"):
            call(src, wrong)


# ------------------------------------------------------------------ wrong device data

def test_wrong_pages_and_lengths_are_reported():
    c = _case(11, [40, 50], 2, 64, 16, 16, spare=8)
    q = _bf16(c["rng"], 2, 1, 4, 64).cuda()
    k = _bf16(c["rng"], 2, 2, 64).cuda()
    offs = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    w = torch.zeros(2, 2, c["cap"], device="cuda")
    new = torch.from_numpy(np.array(c["free"][:4], dtype=np.int32).reshape(2, 2)).cuda()
    for bad in ((1 << 30), -1, c["kc"].shape[0]):
        g = _gpu(c)
        g["table"][1, 3] = bad  # the page of the newest tokens
        for call in (lambda: jfa.jfa_decode_fp8(q, *_cache(g), check=True),
                     lambda: jfa.jfa_cache_append_fp8(k, k, *_cache(g), offs, 1, check=True),
                     lambda: jfa.jfa_cache_evict_fp8(*_cache(g), w, 20, new, recent=10, check=True)):
            with pytest.raises(jfa.JfaError, match="inconsistent device input"):
                call()
    for L in (-1, c["cap"] + 1):
        g = _gpu(c)
        g["lens"][0] = L
        for call in (lambda: jfa.jfa_decode_fp8(q, *_cache(g), check=True),
                     lambda: jfa.jfa_cache_append_fp8(k, k, *_cache(g), offs, 1, check=True),
                     lambda: jfa.jfa_cache_evict_fp8(*_cache(g), w, 20, new, check=True)):
            with pytest.raises(jfa.JfaError, match="inconsistent device input"):
                call()
    g = _gpu(c)
    before = {n: g[n].clone() for n in ("kc", "vc", "ks", "vs")}
    for offsets, most in (([0, 2, 1], 2), ([0, 1, 3], 2), ([1, 1, 2], 2), ([0, 0, 2], 1), ([-1, 1, 2], 2)):
        o = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        with pytest.raises(jfa.JfaError, match="inconsistent device input"):
            jfa.jfa_cache_append_fp8(k, k, *_cache(g), o, most, check=True)
    # pages in use, or given out twice, are not written by an eviction
    g = _gpu(c)
    for table in ([[int(c["table"][1, 0]), int(c["free"][0])], [int(c["free"][1]), int(c["free"][2])]],
                  [[int(c["free"][0]), int(c["free"][1])], [int(c["free"][1]), int(c["free"][2])]]):
        g = _gpu(c)
        with pytest.raises(jfa.JfaError, match="inconsistent device input"):
            jfa.jfa_cache_evict_fp8(*_cache(g), w, 20, torch.tensor(table, dtype=torch.int32, device="cuda"),
                                    check=True)
        for page in (int(c["table"][1, 0]), int(c["free"][1]) if table[0][0] == int(c["free"][0]) else
                     int(c["table"][0, 0])):
            assert torch.equal(g["kc"][page], before["kc"][page]) and torch.equal(g["vs"][page], before["vs"][page])


# ------------------------------------------------------------------ together

class _Server:
    """A cache that is filled, read and cut back step by step, beside the oracle's copy."""

    def __init__(self, seed, B, H, G, d, P, block, pages, mp):
        self.rng = np.random.default_rng(seed)
        self.c = dict(kc=np.full((pages, P, H, d), 0x7F, dtype=np.uint8), d=d)
        self.c["vc"] = self.c["kc"].copy()
        self.c["ks"] = np.full((pages, P // block, H), np.nan, dtype=np.float32)
        self.c["vs"] = self.c["ks"].copy()
        self.c["table"] = np.full((B, mp), -1, dtype=np.int32)
        self.c["lens"] = np.zeros(B, dtype=np.int32)
        self.w = np.zeros((B, H, mp * P), dtype=np.float32)
        self.free = list(self.rng.permutation(pages))
        self.B, self.H, self.G, self.d, self.P = B, H, G, d, P
        self.g = {n: torch.from_numpy(self.c[n].copy()).cuda() for n in ("kc", "vc", "ks", "vs", "table", "lens")}
        self.gw = torch.from_numpy(self.w.copy()).cuda()

    def append(self, new):
        lens = self.c["lens"] + np.array(new, dtype=np.int32)
        for b, L in enumerate(lens):
            for i in range(-(-int(self.c["lens"][b]) // self.P), -(-int(L) // self.P)):
                self.c["table"][b, i] = self.free.pop()
        self.c["lens"] = lens
        self.g["table"].copy_(torch.from_numpy(self.c["table"]))
        self.g["lens"].copy_(torch.from_numpy(lens))
        n = sum(new)
        k, v = _bf16(self.rng, n, self.H, self.d), _bf16(self.rng, n, self.H, self.d)
        offs = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        jfa.jfa_cache_append_fp8(k.cuda(), v.cuda(), *_cache(self.g), torch.from_numpy(offs).cuda(), max(new),
                                 weights=self.gw, check=True)
        c = self.c
        kvo.append(np64(k), np64(v), c["kc"], c["vc"], c["ks"], c["vs"], c["table"], lens, offs, self.w)

    def decode(self, ql):
        q = _bf16(self.rng, self.B, ql, self.H * self.G, self.d)
        was = self.gw.cpu().numpy()
        o, lse = jfa.jfa_decode_fp8(q.cuda(), *_cache(self.g), weights=self.gw, decay=0.9, check=True)
        check_decode(self.c, q, o, lse, self.d ** -0.5, was, self.gw, was, 0.9, "server")
        self.w = self.gw.cpu().numpy()

    def evict(self, keep, first, recent):
        new = np.full((self.B, self.c["table"].shape[1]), -1, dtype=np.int32)
        for b, L in enumerate(self.c["lens"]):
            for i in range(-(-min(int(L), keep) // self.P)):
                new[b, i] = self.free.pop()
        gn = torch.from_numpy(new).cuda()
        kept, nl, nw = jfa.jfa_cache_evict_fp8(*_cache(self.g), self.gw, keep, gn, first=first, recent=recent,
                                               check=True)
        c = self.c
        k2, l2, w2 = kvo.evict(c["kc"], c["vc"], c["ks"], c["vs"], c["table"], c["lens"], self.w, keep, new, first,
                               recent)
        assert (kept.cpu().numpy() == k2).all() and (nw.cpu().numpy() == w2).all()
        self.free += [int(p) for b in range(self.B) for p in c["table"][b, :-(-int(c["lens"][b]) // self.P)]]
        c["table"], c["lens"], self.w = new, l2, w2
        self.g["table"], self.g["lens"], self.gw = gn, nl, nw

    def same(self):
        for b, L in enumerate(self.c["lens"]):
            t = np.arange(int(L))
            page = self.c["table"][b][t // self.P]
            for x in ("kc", "vc"):
                assert _same_codes(self.g[x].cpu().numpy()[page, t % self.P], self.c[x][page, t % self.P]), x


@pytest.mark.parametrize("d,P,block", [(64, 16, 8), (128, 16, 16)])
def test_append_decode_evict_in_turn(d, P, block):
    s = _Server(12, 3, 2, 4, d, P, block, 80, 12)
    s.append([37, 0, 90])
    for step in range(4):
        s.append([1, 1, 1])
        s.decode(1)
    s.append([2, 2, 2])
    s.decode(2)
    s.same()
    s.evict(32, 4, 8)
    s.same()
    for step in range(3):
        s.append([1, 1, 1])
        s.decode(1)
    s.evict(20, 2, 4)
    s.append([60, 1, 0])
    s.decode(1)
    s.same()


def test_cache_replayed_from_a_cuda_graph():
    """A decode step (append, attention with weights) and an eviction, captured with one workspace
    and replayed on new values; each replay equals the same calls made one by one."""
    lens = [40, 513, 16]
    c = _case(13, lens, 2, 128, 16, 16, spare=20)
    new = torch.from_numpy(np.array(c["free"][:9], dtype=np.int32).reshape(3, 3)).cuda()
    offs = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    state = {**_gpu(c), "w": torch.rand(3, 2, c["cap"], device="cuda"), "q": _bf16(c["rng"], 3, 1, 16, 128).cuda(),
             "k": _bf16(c["rng"], 3, 2, 128).cuda(), "v": _bf16(c["rng"], 3, 2, 128).cuda()}
    out = dict(o=torch.empty_like(state["q"]), lse=torch.empty(3, 1, 16, device="cuda"),
               kept=torch.empty(3, 2, 48, dtype=torch.int32, device="cuda"),
               new_seqlens=torch.empty(3, dtype=torch.int32, device="cuda"),
               new_weights=torch.empty(3, 2, 48, device="cuda"))

    def step(s, r, workspace):
        jfa.jfa_cache_append_fp8(s["k"], s["v"], *_cache(s), offs, 1, weights=s["w"], workspace=workspace)
        jfa.jfa_decode_fp8(s["q"], *_cache(s), weights=s["w"], decay=0.5, o=r["o"], lse=r["lse"], workspace=workspace)
        jfa.jfa_cache_evict_fp8(*_cache(s), s["w"], 48, new, first=2, recent=3, kept=r["kept"],
                                new_seqlens=r["new_seqlens"], new_weights=r["new_weights"], workspace=workspace)

    first = {n: t.clone() for n, t in state.items()}
    step(state, out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(state, out, ws)
    for seed in range(3):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        fresh = {n: t.clone() for n, t in first.items()}
        for n in ("q", "k", "v"):
            fresh[n] = torch.randn(fresh[n].shape, generator=gen, device="cuda").to(torch.bfloat16)
        for n in state:
            state[n].copy_(fresh[n])
        ws.fill_(0xA5)
        graph.replay()
        torch.cuda.synchronize()
        assert jfa.jfa_read_device_status(ws) == (0, 0)
        alone = {n: torch.empty_like(t) for n, t in out.items()}
        step(fresh, alone, None)
        torch.cuda.synchronize()
        for n in out:
            assert torch.equal(out[n], alone[n]), n
        for n in fresh:
            same = _same_codes(state[n].cpu().numpy(), fresh[n].cpu().numpy()) if n in ("kc", "vc") else \
                torch.equal(state[n], fresh[n])
            assert same, n


def test_cache_on_side_streams():
    """Two batches at once on two streams, each with its own cache and workspace."""
    runs = []
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i, s in enumerate(streams):
        c = _case(14 + i, [2000, 1, 300 + i], 2, 128, 16, 16)
        g = _gpu(c)
        q = _bf16(c["rng"], 3, 1, 8, 128)
        runs.append((c, g, q, q.cuda(), torch.empty(16 << 20, dtype=torch.uint8, device="cuda")))
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        got = [jfa.jfa_decode_fp8(r[3], *_cache(r[1]), workspace=r[4], stream=s) for r, s in zip(runs, streams)]
        torch.cuda.synchronize()
    for (c, _, q, _, _), (o, lse) in zip(runs, got):
        check_decode(c, q, o, lse, 128 ** -0.5, what="streams")
    # results and workspace of the binding's own, on a stream that is not the current one
    c, g, q, qg, _ = runs[0]
    streams[1].wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        o, lse = jfa.jfa_decode_fp8(qg, *_cache(g), stream=streams[1], check=True)
    check_decode(c, q, o, lse, 128 ** -0.5, what="own results")


def test_float8_tensors_and_empty_batches():
    c = _case(16, [33], 2, 64, 16, 16)
    g = _gpu(c)
    q = _bf16(c["rng"], 1, 1, 4, 64).cuda()
    o, lse = jfa.jfa_decode_fp8(q, *_cache(g), check=True)
    f8 = (g["kc"].view(torch.float8_e4m3fn), g["vc"].view(torch.float8_e4m3fn), *_cache(g)[2:])
    o2, lse2 = jfa.jfa_decode_fp8(q, *f8, check=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    none = (*_cache(g)[:4], g["table"][:0].contiguous(), g["lens"][:0].contiguous())
    o, lse = jfa.jfa_decode_fp8(q[:0].contiguous(), *none, check=True)
    assert o.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    jfa.jfa_cache_append_fp8(k, k, *none, z, 0, check=True)
    jfa.jfa_cache_evict_fp8(*none, torch.zeros(0, 2, c["cap"], device="cuda"), 16,
                            torch.zeros(0, 1, dtype=torch.int32, device="cuda"), check=True)
    # a batch that gets no new token, and one whose table has no pages at all
    before = g["kc"].clone()
    jfa.jfa_cache_append_fp8(k, k, *_cache(g), torch.zeros(2, dtype=torch.int32, device="cuda"), 0, check=True)
    assert torch.equal(before, g["kc"])
    no_pages = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    o, lse = jfa.jfa_decode_fp8(q, *_cache(g)[:4], no_pages, torch.zeros(1, dtype=torch.int32, device="cuda"),
                                check=True)
    assert (o == 0).all() and torch.isneginf(lse).all()
