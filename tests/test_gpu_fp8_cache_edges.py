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
from tests.test_gpu_fp8_cache import _bf16, _cache, _case, _gpu

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
