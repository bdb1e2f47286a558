"""Calls of speculative decoding over the bf16 paged cache that other tests leave out: one token of a fused
projection rotated in place."""
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from tests.test_gpu_spec_decode import _bf16, cache, check_append, dev, make, tables

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,Hq,Hkv", [(128, 32, 8), (64, 6, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_one_token_of_a_fused_projection_in_place(d, Hq, Hkv, interleaved):
    """The row of a fused projection holds q, k and v; with one token its strides say nothing, and Q may turn where
    it lies, as a view of the whole row or cut out of it."""
    cos, sin = tables(100, d)
    gcos, gsin = (torch.from_numpy(x).cuda() for x in (cos, sin))
    for cut in ("heads", "columns"):
        c = make(200, [77], [1], Hkv, d, 16)
        g = dev(c)
        row = _bf16(c["rng"], 1, Hq + 2 * Hkv, d)
        q, k, v = row.split([Hq, Hkv, Hkv], dim=1)
        gr = row.cuda()
        if cut == "heads":
            gq, gk, gv = gr.split([Hq, Hkv, Hkv], dim=1)
        else:
            gq, gk, gv = (x.unflatten(1, (-1, d)) for x in gr.flatten(1).split([Hq * d, Hkv * d, Hkv * d], dim=1))
        out = jfa.jfa_cache_append_rope(gq, gk, gv, *cache(g), g["offs"], gcos, gsin, interleaved=interleaved, q_out=gq,
                                        check=True)
        assert out is gq and torch.equal(gr[:, Hq:].cpu(), row[:, Hq:])
        check_append(c, g, q, k, v, gq, cos, sin, None, interleaved, cut)
