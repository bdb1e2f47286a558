"""Values that are not finite in the bf16 paged cache of the tree attention, against the definition in 64 bits:
they reach every row that sees their token, however small its weight and wherever the work is cut, and no other.

The scores here are whole numbers of some hundreds, so that weights lie far below what fp32 holds
(e^-300 = 2^-433) and are still positive in 64 bits. There 0 * infinity is NaN, so such an infinity may arrive as a
NaN; a NaN stays one. What is finite has the bounds of tests/test_gpu_spec_decode.py.
"""
import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import spec_decode as sd
from tests.parity import np64
from tests.test_gpu_spec_decode import _bf16, as_i64, cache, check_tree, dev, make, words

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
LOW = -300.0


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def scored(c, rows, heads, low):
    """Q, and the cache's keys changed so that tokens `low` of each sequence score 300 below the others (scale 1)."""
    q = _bf16(c["rng"], rows, heads, c["d"]) * 0.25
    q[..., 0] = 1.0
    for b, L in enumerate(c["lens"]):
        for t in range(int(L)):
            c["kc"][sd.cell(c["table"][b], c["P"], t)][..., 0] = LOW if low(int(L), t) else 0.0
    return q


def run(c, q, mask, what):
    g = dev(c)
    with np.errstate(invalid="ignore"):
        o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], as_i64(mask), scale=1.0, check=True)
        check_tree(c, q, o, lse, 1.0, mask, what)
        O, LSE, *_ = sd.decode_tree(np64(q), np64(c["kc"]), np64(c["vc"]), c["table"], c["lens"], c["offs"], 1.0, mask)
    assert (np.isnan(np64(o)) >= np.isnan(O)).all(), what
    return np64(o), np64(lse), O, LSE


# A line that no border cuts: one sequence a CTA, all alike, three tiles each. A line that is cut: two sequences of
# some hundred tiles, two to four tiles a CTA. The tokens of low scores are a tile of the former; of the latter nine
# tiles with the value in the middle one, so that some whole part of the line scores low.
@pytest.mark.parametrize("d,P", [(128, 16), (64, 7)])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("n", [16, 40])  # one row tile and two, with four heads a KV head
@pytest.mark.parametrize("cut", [False, True])
def test_weights_that_underflow(cut, n, where, d, P):
    if cut:
        before = [sms() * 128 - 100, sms() * 128 - 163]
    else:
        before = [300] * sms()
    tiles = [-(-(x + n) // 128) for x in before]
    span = 9 if cut else 1
    first = {"first": [0] * len(tiles), "middle": [(x - span) // 2 for x in tiles], "last": [x - span for x in tiles]}[where]
    c = make(100, before, [n] * len(before), 1, d, P)
    at = {int(x): f for x, f in zip(c["lens"], first)}
    q = scored(c, n * len(before), 4, lambda L, t: at[L] <= t // 128 < at[L] + span)
    mask = words(c["rng"], [n] * len(before), "tree")
    for b, x in zip((0, 1), (NAN, INF)):
        L, f = int(c["lens"][b]), first[b]
        t = L - n + 5 if where == "last" else (f + span // 2) * 128 + 77  # a draft, or an earlier token
        c["vc"][sd.cell(c["table"][b], P, t)][0, 3] = x
    c["vc"][sd.cell(c["table"][1], P, int(c["lens"][1]) - n + 2)][0, 9] = -INF  # a draft, of any score
    o, _, O, _ = run(c, q, mask, f"cut {cut} n {n} {where}")
    bad = ~np.isfinite(O)
    seen = [n, n] if where != "last" else [sum(int(w) >> 5 & 1 for w in mask[b * n:b * n + n]) for b in (0, 1)]
    assert [int(bad[b * n:b * n + n, 0, 3].sum()) for b in (0, 1)] == seen and min(seen) > 0  # the values are met
    assert not bad[2 * n:].any()


@pytest.mark.parametrize("cut", [False, True])
@pytest.mark.parametrize("n", [16, 40])
def test_kinds_are_kept(cut, n):
    """With weights that fp32 holds an infinity keeps its sign, and only two of unlike signs make a NaN."""
    before = [sms() * 128 - 100, 700, 90] if cut else [300] * sms()
    c = make(101, before, [n] * len(before), 1, 128, 16)
    L, at = c["lens"], lambda b, t: sd.cell(c["table"][b], 16, int(t))
    c["vc"][at(0, 10)][0, 0] = INF
    c["vc"][at(0, 150)][0, 1] = -INF
    c["vc"][at(0, 20)][0, 2] = INF
    c["vc"][at(0, L[0] - n + 1)][0, 2] = -INF  # a draft, against the earlier token's
    c["vc"][at(0, L[0] - n + 1)][0, 3] = INF
    c["vc"][at(0, L[0] - n + 2)][0, 3] = -INF
    c["vc"][at(0, L[0] - n + 3)][0, 4] = -INF
    c["vc"][at(0, L[0] - 140)][0, 5] = NAN
    c["kc"][at(1, 33)][0, 7] = NAN
    c["kc"][at(2, L[2] - 1)][0, 7] = NAN  # the last draft's key
    q = _bf16(c["rng"], n * len(before), 4, 128)
    mask = words(c["rng"], [n] * len(before), "tree")
    o, lse, O, LSE = run(c, q * 0.1, mask, f"cut {cut} n {n}")
    for x, y in ((o, O), (lse, LSE)):
        assert (np.isnan(x) == np.isnan(y)).all()
        assert (np.isposinf(x) == np.isposinf(y)).all() and (np.isneginf(x) == np.isneginf(y)).all()
    assert np.isnan(LSE[n:2 * n]).all() and np.isposinf(O).any() and np.isneginf(O).any()
    assert np.isnan(LSE[2 * n:3 * n]).any() and np.isfinite(LSE[2 * n:3 * n]).any()


def test_scores_of_minus_infinity():
    """A key's infinity acts as the score that it makes: -infinity is a weight of 0, and a row with no other score
    is like one that sees nothing; +infinity and 0 * infinity make NaN of the row."""
    n = 3
    c = make(102, [200, 0, 40, 130], [n] * 4, 1, 128, 16)
    q = _bf16(c["rng"], 4 * n, 4, 128)
    q[..., 0] = 1.0
    q[3 * n:3 * n + 1, :, 0] = 0.0  # 0 * infinity
    q[3 * n + 1:3 * n + 2, :, 0] = -1.0
    for t in (0, 130, 202):
        c["kc"][sd.cell(c["table"][0], 16, t)][0, 0] = -INF
    for t in range(3):
        c["kc"][sd.cell(c["table"][1], 16, t)][0, 0] = -INF
    for t in range(43):
        c["kc"][sd.cell(c["table"][2], 16, t)][0, 0] = -INF
    c["kc"][sd.cell(c["table"][3], 16, 5)][0, 0] = -INF
    g = dev(c)
    o, lse = jfa.jfa_decode_tree(q.cuda(), *cache(g), g["offs"], scale=0.1, check=True)
    o, lse = np64(o), np64(lse)
    assert (o[n:3 * n] == 0).all() and np.isneginf(lse[n:3 * n]).all()
    assert np.isnan(o[3 * n:3 * n + 2]).all() and np.isnan(lse[3 * n:3 * n + 2]).all()
    # the rest as if those tokens were not there, to a bound far above what the definition's rounding takes
    with np.errstate(invalid="ignore"):
        O, LSE, absO, A = sd.decode_tree(np64(q), np64(c["kc"]), np64(c["vc"]), c["table"], c["lens"], c["offs"], 0.1)
    for r in list(range(n)) + [3 * n + 2]:
        assert (np.abs(lse[r] - LSE[r]) <= 1e-3).all()
        assert (np.abs(o[r] - O[r]) <= 2.0 ** -7 * absO[r] + 2.0 ** -7 * np.abs(O[r])).all()
