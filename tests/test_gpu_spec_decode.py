"""GPU parity of speculative decoding over the bf16 paged cache: append with rotation, tree attention, accept.

What is copied, moved or left alone is compared bit for bit. The tolerances, with u = 2^-24:
  * a rotated value: two products and a sum in fp32 (at most two roundings on each product's
    way), then half a bf16 step: |dx| <= 2^-8 |x'| + 4 u (|x cos| + |y sin|) + 2^-134;
  * a score is a sum of d products, exact in fp32, added in fp32 (an addition may truncate:
    2^-23 of the running magnitude), then scaled by a few rounded factors:
    |ds| <= (d + 8) 2^-23 A + 2^-20, A = max_j scale sum_d |q_d k_jd|; the constant covers the
    approximate exponential and logarithm (2^-21 each, absolute in the exponent);
  * LSE moves by at most the scores' error, plus its own few roundings;
  * O: weights carry the scores' error twice (numerator, denominator) and one rounding to bf16,
    half a step 2^-8; a column's L products are added 16 at a time in fp32, and the joins of the
    parts round a few times more (2^-13 together with the sum of the weights); the bf16 result
    rounds by half a step 2^-8:
    |dO| <= (2^-8 + (L / 16) 2^-23 + 2^-13 + 2 |ds|) sum_j P_j |v_j| + 2^-8 |O| + 2^-134.
    The running maximum of a row is at most 2^8 above its reference, so a weight below 2^-118 of
    the largest may become 0; L of them are far below the 2^-13.
"""
import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import spec_decode as sd
from tests.parity import np64

pytestmark = pytest.mark.gpu
bf16, i32 = torch.bfloat16, torch.int32


def _bf16(rng, *shape, spread=0.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[:-1] + (1,)))
    return torch.from_numpy(x.astype(np.float32)).to(bf16)


def make(seed, before, new, H, d, P, spare=2, wide=0):
    """A batch over a filled cache, on the host: slots of nobody hold NaN, table entries of no use are out of range."""
    rng = np.random.default_rng(seed)
    lens = [a + n for a, n in zip(before, new)]
    need = [-(-x // P) for x in lens]
    pages = sum(need) + spare
    table = np.full((len(lens), max(max(need, default=0), 1) + wide), 2 ** 30, dtype=np.int32)
    perm = rng.permutation(pages)
    live = np.zeros((pages, P), dtype=bool)
    at = 0
    for b, x in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        t = np.arange(x)
        live[table[b][t // P], t % P] = True
    kc, vc = (_bf16(rng, pages, P, H, d, spread=0.5) for _ in range(2))
    for c in (kc, vc):
        c[torch.from_numpy(~live)] = float("nan")
    return dict(rng=rng, kc=kc, vc=vc, table=table, lens=np.array(lens, dtype=np.int32), H=H, d=d, P=P, new=list(new),
                offs=np.concatenate([[0], np.cumsum(new)]).astype(np.int32), before=list(before))


def dev(c):
    t = {n: torch.from_numpy(c[n]).cuda() for n in ("table", "lens", "offs")}
    return dict(kc=c["kc"].cuda(), vc=c["vc"].cuda(), **t)


def cache(g):
    return g["kc"], g["vc"], g["table"], g["lens"]


def words(rng, new, kind):
    """Masks of a batch: random trees (parents before children), or any bits at all, rows without one among them."""
    out = []
    for n in new:
        seen = []
        for i in range(n):
            if kind == "bits":
                w = int(rng.integers(0, 2 ** 64, dtype=np.uint64)) & int(rng.integers(0, 2 ** 64, dtype=np.uint64))
                seen.append(0 if rng.random() < 0.2 else w)
            else:
                parent = int(rng.integers(-1, i)) if i else -1
                seen.append((seen[parent] if parent >= 0 else 0) | 1 << i)
        out += seen
    return np.array(out, dtype=np.uint64)


def check_tree(c, q, o, lse, scale, mask=None, what=""):
    O, LSE, absO, A = sd.decode_tree(np64(q), np64(c["kc"]), np64(c["vc"]), c["table"], c["lens"], c["offs"], scale, mask)
    used = int(c["offs"][-1])
    O, LSE, absO, A, o, lse = (x[:used] for x in (O, LSE, absO, A, np64(o), np64(lse)))
    ds = (c["d"] + 8) * 2.0 ** -23 * A + 2.0 ** -20
    coef = 2.0 ** -8 + c["lens"].max(initial=0) / 16 * 2.0 ** -23 + 2.0 ** -13
    bound = (coef + 2 * ds)[..., None] * absO + 2.0 ** -8 * np.abs(O) + 2.0 ** -134
    fin = np.isfinite(O)
    assert (np.isfinite(o) == fin).all(), what
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(o - O) <= bound) & fin
    assert not bad.any(), f"{what}: O {np.abs(o - O)[bad].max():.3e} at {np.argwhere(bad)[:3]}"
    none = np.isneginf(LSE)
    assert (np.isneginf(lse) == none).all() and (o[none] == 0).all(), what
    with np.errstate(invalid="ignore"):
        ok = none | ~np.isfinite(LSE) | (np.abs(lse - LSE) <= ds + (np.abs(LSE) + 1) * 2.0 ** -21)
    assert ok.all(), f"{what}: LSE {np.abs(lse - LSE)[~ok].max():.3e}"


BEFORE = [0, 0, 5, 127, 128, 100, 700, 129, 1500, 64]
NEW = [1, 9, 0, 1, 3, 64, 33, 17, 40, 64]


def as_i64(mask):
    return torch.from_numpy(mask.view(np.int64)).cuda()


# ------------------------------------------------------------------ tree attention

@pytest.mark.parametrize("d,P", [(128, 16), (64, 16), (128, 1), (64, 24), (128, 128), (128, 7), (64, 4), (128, 256)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1), (3, 3), (16, 1)])
def test_tree_ragged(Hq, Hkv, d, P):
    c = make(1, BEFORE, NEW, Hkv, d, P)
    g = dev(c)
    q = _bf16(c["rng"], sum(NEW), Hq, d)
    for kind in ("tree", "bits", None):
        mask = None if kind is None else words(c["rng"], NEW, kind)
        o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], None if mask is None else as_i64(mask), scale=0.2,
                                     check=True)
        check_tree(c, q, o, lse, 0.2, mask, f"{kind} Hq {Hq} Hkv {Hkv} d {d} P {P}")


@pytest.mark.parametrize("group", [1, 5, 6, 12, 32, 64, 100, 128])
def test_tree_groups(group):
    new = [64, 3, 1, 30]
    c = make(2, [40, 300, 129, 0], new, 1, 64, 16)
    g = dev(c)
    q = _bf16(c["rng"], sum(new), group, 64)
    mask = words(c["rng"], new, "tree")
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask), check=True)
    check_tree(c, q, o, lse, 64 ** -0.5, mask, f"group {group}")


@pytest.mark.parametrize("max_q", [1, 2, 5, 32, 33])
def test_tree_bounds_of_max_q(max_q):
    new = [max_q, max_q - 1, max_q]
    c = make(3, [200, 77, 1000], new, 2, 128, 16)
    g = dev(c)
    q = _bf16(c["rng"], sum(new), 8, 128)
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], max_q=max_q, check=True)
    check_tree(c, q, o, lse, 128 ** -0.5, None, f"max_q {max_q}")


def test_tree_one_long():
    """One sequence cut into as many parts as there are CTAs, and the same bits every time."""
    c = make(4, [9000], [6], 1, 128, 16)
    g = dev(c)
    q = _bf16(c["rng"], 6, 4, 128)
    mask = words(c["rng"], [6], "tree")
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask), check=True)
    check_tree(c, q, o, lse, 128 ** -0.5, mask)
    for _ in range(3):
        o2, lse2 = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask))
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_tree_many_sequences():
    """More sequences than threads of a block, most of them empty; more lines than CTAs."""
    rng = np.random.default_rng(5)
    new = [int(n) if rng.random() < 0.3 else 0 for n in rng.integers(1, 9, 1000)]
    before = [int(x) for x in rng.integers(0, 40, 1000)]
    c = make(5, before, new, 2, 64, 8)
    g = dev(c)
    q = _bf16(c["rng"], sum(new), 4, 64)
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], check=True)
    check_tree(c, q, o, lse, 0.125)


def test_tree_is_the_small_query_decode():
    """A chain of equal lengths gives what jfa_decode_smallq gives, to bf16's rounding."""
    B, n, Hq, Hkv = 3, 4, 8, 2
    c = make(6, [700, 33, 128], [n] * B, Hkv, 128, 16)
    g = dev(c)
    q = _bf16(c["rng"], B * n, Hq, 128)
    g["kc"].nan_to_num_(0)
    g["vc"].nan_to_num_(0)
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"])
    o2, lse2 = jfa.jfa_decode_smallq(q.view(B, n, Hq, 128).cuda(), *cache(g), 4, check=True)
    assert (lse.view_as(lse2) - lse2).abs().max() < 1e-4
    assert (o.float().view_as(o2) - o2.float()).abs().max() < 3e-2


@pytest.mark.parametrize("Hq", [2, 32])
def test_tree_not_finite(Hq):
    """Infinities and NaN in K or V of a draft reach the rows that see it and no others; those of earlier
    tokens reach every row of their sequence."""
    new, before = [20, 40, 33, 5], [115, 640, 0, 300]
    c = make(7, before, new, 2, 128, 16)
    mask = words(c["rng"], new, "bits")
    at = lambda b, t: sd.cell(c["table"][b], 16, t)
    inf, nan = float("inf"), float("nan")
    c["vc"][at(0, 116)][0, 3] = inf
    c["vc"][at(0, 134)][1, 100] = nan
    c["vc"][at(1, 640 + 7)][0] = nan
    c["vc"][at(1, 640 + 39)][1, 5] = -inf
    c["vc"][at(1, 640 + 38)][1, 5] = inf
    c["kc"][at(2, 4)][0, 7] = nan
    c["kc"][at(2, 20)][1, 7] = nan
    c["vc"][at(3, 17)][1, 64] = nan
    g = dev(c)
    q = _bf16(c["rng"], sum(new), Hq, 128)
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask), check=True)
    check_tree(c, q, o, lse, 128 ** -0.5, mask)
    assert np.isfinite(np64(o)).any() and not np.isfinite(np64(o)).all()


def test_tree_scores_far_apart():
    """Maxima that grow late, and rows whose scores differ by thousands."""
    new = [16, 64]
    c = make(8, [500, 1000], new, 1, 128, 16)
    for b, x in enumerate(c["lens"]):
        for t in range(int(x)):
            c["kc"][sd.cell(c["table"][b], 16, t)] *= 0.05 * (1 + 40 * t / int(x))
    g = dev(c)
    q = _bf16(c["rng"], sum(new), 4, 128, spread=1.5)
    mask = words(c["rng"], new, "tree")
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask), scale=1.0, check=True)
    check_tree(c, q, o, lse, 1.0, mask)


def test_tree_leaves_rows_behind_the_last_sequence():
    new = [3, 5]
    c = make(9, [30, 200], new, 2, 64, 16)
    g = dev(c)
    q = _bf16(c["rng"], 12, 4, 64)
    o, lse = torch.full_like(q, 7).cuda(), torch.full((12, 4), 7.0, device="cuda")
    jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], o=o, lse=lse, check=True)
    check_tree(c, q, o, lse, 0.125)
    assert (o[8:] == 7).all() and (lse[8:] == 7).all()


def test_tree_bad_input():
    """Lengths, offsets and page entries out of range: reported, and only their sequences are touched by it."""
    new = [3, 5, 2]
    c = make(10, [30, 200, 60], new, 2, 64, 16)
    q = _bf16(c["rng"], 10, 4, 64)
    cap = c["table"].shape[1] * 16
    for what, b, x in (("lens", 1, cap + 1), ("lens", 1, 4), ("lens", 1, -1), ("offs", 1, 9), ("table", 1, None), ("max_q", 1, 4)):
        g = dev(c)
        max_q = 64
        if what == "table":
            g["table"][1, 3] = 10 ** 6
        elif what == "max_q":
            max_q = x
        else:
            g[what][b] = x
        o, lse = torch.full_like(q, 7).cuda(), torch.full((10, 4), 7.0, device="cuda")
        with pytest.raises(jfa.JfaError, match="501"):
            jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], max_q=max_q, o=o, lse=lse, check=True)
        if what in ("lens", "max_q"):
            assert (o[3:8] == 0).all() and torch.isneginf(lse[3:8]).all()
        if what != "offs":
            good = dict(c, lens=c["lens"][[0, 2]], table=c["table"][[0, 2]], offs=np.array([0, 3, 5], dtype=np.int32))
            rows = [0, 1, 2, 8, 9]
            check_tree(good, q[rows], o[rows], lse[rows], 0.125)


def test_tree_without_work():
    c = make(11, [30, 20], [0, 0], 2, 64, 16)
    g = dev(c)
    o, lse = jfa.jfa_decode_tree(torch.zeros(0, 4, 64, dtype=bf16).cuda(), *cache(g), g["offs"], check=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    o = torch.full((2, 4, 64), 7, dtype=bf16).cuda()
    jfa.jfa_decode_tree(torch.zeros(2, 4, 64, dtype=bf16).cuda(), *cache(g), g["offs"], o=o, check=True)
    assert (o == 7).all()
    e = torch.zeros(0, dtype=i32).cuda()
    jfa.jfa_decode_tree(torch.zeros(0, 4, 64, dtype=bf16).cuda(), g["kc"], g["vc"], e.view(0, 3), e,
                        torch.zeros(1, dtype=i32).cuda(), check=True)


# ------------------------------------------------------------------ append

def tables(rows, rot):
    angle = np.arange(rows)[:, None] * 10000.0 ** (-np.arange(rot // 2) / max(rot // 2, 1))
    return np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)


def check_append(c, g, q, k, v, q_out, cos, sin, positions=None, interleaved=False, what=""):
    kc, vc = np64(c["kc"]), np64(c["vc"])
    was = kc.copy()
    want = sd.append_rope(None if q is None else np64(q), np64(k), np64(v), kc, vc, c["table"], c["lens"], c["offs"], cos,
                          sin, positions, interleaved)
    got_k, got_v = np64(g["kc"]), np64(g["vc"])
    assert np.array_equal(got_v, vc, equal_nan=True), what
    used = int(c["offs"][-1])

    def close(x, y, src, what):
        # |x cos| + |y sin| of a pair is at most the pair's length times sqrt(2), and at most 1.5 of its head's largest times 2
        top = np.abs(src).max(-1, keepdims=True, initial=0.0)
        with np.errstate(invalid="ignore"):
            ok = (np.abs(x - y) <= 2.0 ** -8 * np.abs(y) + 4 * 2.0 ** -24 * 2 * top + 2.0 ** -134) | (np.isnan(x) & np.isnan(y))
        assert ok.all(), f"{what}: {np.nanmax(np.abs(x - y)[~ok])}"

    rows = [sd.cell(c["table"][b], c["P"], int(c["lens"][b]) - n + i) for b, n in enumerate(c["new"]) for i in range(n)]
    touched = np.zeros(kc.shape[:2], dtype=bool)
    for i, at in enumerate(rows):
        touched[at] = True
        close(got_k[at], kc[at], np64(k)[i], f"{what}: K")
    assert np.array_equal(got_k[~touched], was[~touched], equal_nan=True), what
    if q is not None:
        close(np64(q_out)[:used], want[:used], np64(q)[:used], f"{what}: Q")
        rot = 0 if cos is None else 2 * cos.shape[1]
        assert torch.equal(q_out[:used, :, rot:].cpu(), q[:used, :, rot:])


@pytest.mark.parametrize("d,P,rot", [(128, 16, 128), (64, 16, 64), (128, 1, 32), (64, 24, 16), (128, 7, 96), (64, 128, 48),
                                     (128, 16, 0)])
@pytest.mark.parametrize("Hq,Hkv", [(8, 2), (7, 1), (3, 3), (40, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(Hq, Hkv, d, P, rot, interleaved):
    c = make(20, BEFORE, NEW, Hkv, d, P)
    g = dev(c)
    n = sum(NEW)
    qkv = _bf16(c["rng"], n, (Hq + 2 * Hkv) * d)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=1))
    cos, sin = tables(2000, rot) if rot else (None, None)
    gt = qkv.cuda()
    gq, gk, gv = (x.unflatten(1, (-1, d)) for x in gt.split([Hq * d, Hkv * d, Hkv * d], dim=1))
    tab = [None if x is None else torch.from_numpy(x).cuda() for x in (cos, sin)]
    out = jfa.jfa_cache_append_rope(gq, gk, gv, *cache(g), g["offs"], *tab, interleaved=interleaved, check=True)
    check_append(c, g, q, k, v, out, cos, sin, None, interleaved)
    assert torch.equal(gt.cpu(), qkv)  # what is read stays


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_positions_and_in_place(interleaved):
    new = [5, 0, 16, 1]
    c = make(21, [3, 50, 100, 999], new, 2, 64, 16)
    g = dev(c)
    n = sum(new)
    q, k, v = (_bf16(c["rng"], n + 3, h, 64) for h in (6, 2, 2))  # three rows behind the last sequence
    pos = c["rng"].integers(0, 77, n + 3).astype(np.int32)
    pos[n:] = -5
    cos, sin = tables(77, 64)
    gq = q.cuda()
    out = jfa.jfa_cache_append_rope(gq, k.cuda(), v.cuda(), *cache(g), g["offs"], torch.from_numpy(cos).cuda(),
                                    torch.from_numpy(sin).cuda(), positions=torch.from_numpy(pos).cuda(),
                                    interleaved=interleaved, q_out=gq, check=True)
    assert out is gq and torch.equal(gq[n:].cpu(), q[n:])
    check_append(c, g, q, k, v, gq, cos, sin, pos, interleaved)
    g2 = dev(c)
    assert jfa.jfa_cache_append_rope(None, k.cuda(), v.cuda(), *cache(g2), g["offs"], torch.from_numpy(cos).cuda(),
                                     torch.from_numpy(sin).cuda(), positions=torch.from_numpy(pos).cuda(),
                                     interleaved=interleaved, check=True) is None
    for x in ("kc", "vc"):
        assert np.array_equal(np64(g[x]), np64(g2[x]), equal_nan=True)


def test_append_not_finite_stays_in_its_pair():
    c = make(22, [10], [4], 1, 64, 16)
    g = dev(c)
    q, k, v = (_bf16(c["rng"], 4, 1, 64) for _ in range(3))
    k[1, 0, 3], k[2, 0, 40], v[0, 0, 5] = float("nan"), float("inf"), float("nan")
    cos, sin = tables(20, 32)
    jfa.jfa_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), *cache(g), g["offs"], torch.from_numpy(cos).cuda(),
                              torch.from_numpy(sin).cuda(), check=True)
    new = np64(g["kc"])[c["table"][0][0], 10:14, 0]
    bad = np.argwhere(~np.isfinite(new)).tolist()
    assert bad == [[1, 3], [1, 19], [2, 40]]


def test_append_bad_input():
    new = [3, 5, 2]
    c = make(23, [30, 200, 60], new, 2, 64, 16)
    q, k, v = (_bf16(c["rng"], 10, h, 64) for h in (4, 2, 2))
    cos, sin = (torch.from_numpy(x).cuda() for x in tables(300, 64))
    cap = c["table"].shape[1] * 16
    good = dict(c, lens=c["lens"][[0, 2]], table=c["table"][[0, 2]], offs=np.array([0, 3, 5], dtype=np.int32), new=[3, 2])
    rows = [0, 1, 2, 8, 9]
    for what in ("long", "short", "negative", "table", "position", "offsets"):
        g = dev(c)
        positions = None
        if what == "table":
            g["table"][1, 200 // 16] = -1
            g["table"][1, 204 // 16] = -1
        elif what == "position":
            positions = torch.cat([torch.arange(30, 33), torch.full((5,), 300), torch.arange(60, 62)]).to(i32).cuda()
        elif what == "offsets":
            g["offs"][3] = 11
        else:
            g["lens"][1] = {"long": cap + 1, "short": 4, "negative": -3}[what]
        out = torch.full_like(q, 7).cuda()
        with pytest.raises(jfa.JfaError, match="551"):
            jfa.jfa_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), *cache(g), g["offs"], cos, sin, positions=positions,
                                      q_out=out, check=True)
        if what != "offsets":
            assert (out[3:8] == 7).all(), what
            check_append(good, g, q[rows], k[rows], v[rows], out[rows], cos.cpu().numpy(), sin.cpu().numpy(), what=what)
    # a table that ends before a sequence does
    g = dev(c)
    with pytest.raises(jfa.JfaError, match="551"):
        jfa.jfa_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), *cache(g), g["offs"], cos[:204], sin[:204], check=True)
    jfa.jfa_cache_append_rope(q.cuda(), k.cuda(), v.cuda(), *cache(g), g["offs"], cos[:205], sin[:205], check=True)


def test_append_without_work():
    c = make(24, [30, 20], [0, 0], 2, 64, 16)
    g = dev(c)
    was = g["kc"].clone()
    none = torch.zeros(0, 2, 64, dtype=bf16).cuda()
    out = jfa.jfa_cache_append_rope(none, none, none, *cache(g), g["offs"], None, None, check=True)
    assert out.shape == (0, 2, 64) and torch.equal(was.nan_to_num(9), g["kc"].nan_to_num(9))


# ------------------------------------------------------------------ accept

@pytest.mark.parametrize("d,P,H", [(128, 16, 8), (64, 16, 3), (128, 1, 2), (64, 24, 5), (128, 7, 1), (64, 128, 2)])
@pytest.mark.parametrize("order", ["rising", "any"])
def test_accept(d, P, H, order):
    new = [64, 1, 0, 9, 33, 64, 16, 7]
    c = make(30, [5, 0, 20, 127, 500, 61, 100, 16], new, H, d, P)
    g = dev(c)
    rng = c["rng"]
    counts = [64, 1, 0, 0, 20, 17, 16, 3]
    path = np.full((len(new), 64), -9, dtype=np.int32)
    for b, n in enumerate(counts):
        pick = rng.permutation(new[b])[:n] if order == "rising" else rng.integers(0, max(new[b], 1), n)
        path[b, :n] = np.sort(pick) if order == "rising" else pick
    lens = jfa.jfa_cache_accept(*cache(g), g["offs"], torch.from_numpy(path).cuda(),
                                torch.tensor(counts, dtype=i32).cuda(), check=True)
    kc, vc = np64(c["kc"]), np64(c["vc"])
    want = sd.accept(kc, vc, c["table"], c["lens"], c["offs"], path, counts)
    assert np.array_equal(lens.cpu().numpy(), want)
    assert np.array_equal(np64(g["kc"]), kc, equal_nan=True) and np.array_equal(np64(g["vc"]), vc, equal_nan=True)


def test_accept_many_and_narrow():
    rng = np.random.default_rng(31)
    new = [int(n) for n in rng.integers(0, 6, 700)]
    c = make(31, [int(x) for x in rng.integers(0, 30, 700)], new, 1, 64, 4)
    counts = np.array([int(rng.integers(0, min(n, 2) + 1)) for n in new], dtype=np.int32)
    path = np.stack([np.resize(rng.permutation(max(n, 1)), 2) for n in new]).astype(np.int32)
    g = dev(c)
    lens = jfa.jfa_cache_accept(*cache(g), g["offs"], torch.from_numpy(path).cuda(), torch.from_numpy(counts).cuda(),
                                check=True)
    kc, vc = np64(c["kc"]), np64(c["vc"])
    assert np.array_equal(lens.cpu().numpy(), sd.accept(kc, vc, c["table"], c["lens"], c["offs"], path, counts))
    assert np.array_equal(np64(g["kc"]), kc, equal_nan=True) and np.array_equal(np64(g["vc"]), vc, equal_nan=True)


def test_accept_bad_input():
    new = [6, 6, 6]
    c = make(32, [10, 20, 30], new, 2, 64, 16)
    path = torch.tensor([[1, 3, 5], [2, 4, 5], [0, 2, 4]], dtype=i32)
    cap = c["table"].shape[1] * 16
    for what in ("count", "negative", "index", "below", "table", "length", "long"):
        g = dev(c)
        p, n = path.clone(), torch.tensor([3, 3, 3], dtype=i32)
        if what in ("count", "negative"):
            n[1] = 4 if what == "count" else -1
        elif what in ("index", "below"):
            p[1, 2] = 6 if what == "index" else -1
        elif what == "table":
            g["table"][1, 1] = -1
        else:
            g["lens"][1] = 5 if what == "length" else cap + 1
        with pytest.raises(jfa.JfaError, match="561"):
            ws = torch.empty(256, dtype=torch.uint8, device="cuda")
            lens = torch.zeros(3, dtype=i32, device="cuda")
            jfa.jfa_cache_accept(*cache(g), g["offs"], p.cuda(), n.cuda(), new_seqlens=lens, workspace=ws, check=True)
        keep = int(g["lens"][1]) if what in ("length", "long") else 20
        assert lens.tolist() == [13, keep, 33], what
        kc, vc = np64(c["kc"]), np64(c["vc"])
        sd.accept(kc, vc, c["table"], c["lens"], c["offs"], path.numpy(), [3, 0, 3])
        assert np.array_equal(np64(g["kc"]), kc, equal_nan=True) and np.array_equal(np64(g["vc"]), vc, equal_nan=True), what


def test_accept_without_work():
    c = make(33, [10, 20], [2, 3], 2, 64, 16)
    g = dev(c)
    lens = jfa.jfa_cache_accept(*cache(g), g["offs"], torch.zeros(2, 0, dtype=i32).cuda(),
                                torch.zeros(2, dtype=i32).cuda(), check=True)
    assert lens.tolist() == [10, 20]


# ------------------------------------------------------------------ together

def test_a_turn_of_speculative_decoding():
    """Prompts enter, trees of drafts enter and attend, paths are accepted, the next token attends: the
    cache then holds what a plain run over the accepted tokens would have put there, bit for bit."""
    rng = np.random.default_rng(40)
    B, H, Hq, d, P, most = 4, 2, 8, 128, 16, 12
    prompt = [37, 128, 5, 250]
    cos, sin = (torch.from_numpy(x).cuda() for x in tables(300, d))
    pages = 80
    table = torch.from_numpy(rng.permutation(pages).reshape(B, 20).astype(np.int32)).cuda()
    nan = float("nan")
    kc, vc = (torch.full((pages, P, H, d), nan, dtype=bf16, device="cuda") for _ in range(2))
    ka, va = kc.clone(), vc.clone()

    def tokens(n):
        return _bf16(rng, n, Hq, d).cuda(), _bf16(rng, n, H, d).cuda(), _bf16(rng, n, H, d).cuda()

    def offsets(n):
        return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).cuda()

    lens = torch.tensor(prompt, dtype=i32).cuda()
    q, k, v = tokens(sum(prompt))
    for c in ((kc, vc), (ka, va)):
        jfa.jfa_cache_append_rope(q, k, v, *c, table, lens, offsets(prompt), cos, sin, check=True)
    for _ in range(2):
        new = [most, 1, 7, most]
        mask = words(rng, new, "tree")
        depth = np.array([int(m).bit_count() - 1 for m in mask])
        offs = offsets(new)
        o = offs.tolist()
        before = lens.tolist()
        pos = np.concatenate([before[b] + depth[o[b]:o[b + 1]] for b in range(B)]).astype(np.int32)
        q, k, v = tokens(sum(new))
        full = lens + torch.tensor(new, dtype=i32).cuda()
        qr = jfa.jfa_cache_append_rope(q, k, v, kc, vc, table, full, offs, cos, sin,
                                       positions=torch.from_numpy(pos).cuda(), check=True)
        out, lse = jfa.jfa_decode_tree(qr, kc, vc, table, full, offs, as_i64(mask), max_q=most, check=True)
        # one accepted path a sequence: the ancestors of a node
        leaf = [int(rng.integers(0, n)) for n in new]
        path = [[j for j in range(new[b]) if int(mask[o[b] + leaf[b]]) >> j & 1] for b in range(B)]
        counts = torch.tensor([len(p) for p in path], dtype=i32).cuda()
        padded = torch.tensor([p + [-1] * (most - len(p)) for p in path], dtype=i32).cuda()
        lens = jfa.jfa_cache_accept(kc, vc, table, full, offs, padded, counts, check=True)
        # the plain run: only the accepted tokens, one after the other
        rows = torch.tensor([o[b] + j for b in range(B) for j in path[b]]).cuda()
        acc = [len(p) for p in path]
        qa = jfa.jfa_cache_append_rope(q[rows], k[rows], v[rows], ka, va, table, lens, offsets(acc), cos, sin, check=True)
        assert torch.equal(qa, qr[rows])
        for b in range(B):
            n = int(lens[b])
            t = torch.arange(n).cuda()
            at = (table[b][t // P].long(), t % P)
            assert torch.equal(kc[at], ka[at]) and torch.equal(vc[at], va[at])
        # the leaf of each path saw the same tokens, in tiles and parts of other sizes
        oa, la = jfa.jfa_decode_tree(qa, ka, va, table, lens, offsets(acc), max_q=most, check=True)
        last = torch.from_numpy(np.cumsum(acc) - 1).cuda()
        leaves = torch.tensor([o[b] + leaf[b] for b in range(B)]).cuda()
        assert (la[last] - lse[leaves]).abs().max() < 1e-4
        assert (oa[last].float() - out[leaves].float()).abs().max() < 2e-2
