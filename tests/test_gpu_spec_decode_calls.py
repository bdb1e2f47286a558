"""Calls of speculative decoding over the bf16 paged cache that other tests leave out: one token of a fused
projection rotated in place, more work than is numbered, and a captured turn whose batch changes between replays."""
import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from tests.test_gpu_spec_decode import _bf16, as_i64, cache, check_append, dev, make, tables, words
from tests.test_gpu_spec_decode_edges import _results, _same, _turn

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


def test_more_work_than_is_numbered():
    """Lines of more than 2^31 tiles together (here over shared pages): reported, and the rows are empty, as those of
    any sequence that is refused. Rows behind the last sequence stay."""
    P, H, d, B, mp = 1024, 1024, 64, 33, 8190
    kc = torch.zeros(1, P, H, d, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(B, mp, dtype=torch.int32, device="cuda")
    lens = torch.full((B,), mp * P, dtype=torch.int32, device="cuda")
    new = [2] + [1] * (B - 1)
    assert (mp * P // 128 + 3) * H * (B - 1) < 2 ** 31 <= (mp * P // 128 + 3) * H * B
    offs = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
    used = sum(new)
    q = torch.ones(used + 2, H, d, dtype=torch.bfloat16, device="cuda")
    o, lse = torch.full_like(q, 7), torch.full((used + 2, H), 7.0, device="cuda")
    with pytest.raises(jfa.JfaError, match="501"):
        jfa.jfa_decode_tree(q, kc, kc, table, lens, offs, max_q=2, o=o, lse=lse, check=True)
    assert (o[:used] == 0).all() and torch.isneginf(lse[:used]).all()
    assert (o[used:] == 7).all() and (lse[used:] == 7).all()


def _state(seed, before, new):
    """A turn's tensors for a batch of these lengths; batches of as many new tokens fill tensors of the same sizes."""
    need = [-(-(a + n) // 16) for a, n in zip(before, new)]
    c = make(seed, before, new, 2, 128, 16, spare=90 - sum(need), wide=60 - max(need))
    g, rng, n = dev(c), c["rng"], sum(new)
    s = {x: _bf16(rng, n, h, 128).cuda() for x, h in (("q", 8), ("k", 2), ("v", 2))}
    s["cos"], s["sin"] = (torch.from_numpy(x).cuda() for x in tables(1000, 128))
    s["mask"] = as_i64(words(rng, new, "tree"))
    s["count"] = torch.tensor([int(rng.integers(0, min(5, m) + 1)) for m in new], dtype=torch.int32).cuda()
    s["path"] = torch.from_numpy(np.stack([rng.integers(0, max(m, 1), 5) for m in new]).astype(np.int32)).cuda()
    s["qr"], s["o"] = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    s["lse"], s["left"] = torch.zeros(n, 8, device="cuda"), torch.zeros_like(g["lens"])
    return g, s


def test_captured_turn_replays_with_another_batch():
    """A graph reads lengths and offsets when it runs: the same turn for sequences of other lengths and other numbers of
    new tokens (lines, cuts and parts all move), for the first ones again, and for a batch that is partly empty."""
    batches = [([100, 700, 5, 33, 256], [12, 1, 0, 30, 7]), ([33, 5, 256, 700, 100], [0, 30, 12, 1, 7]),
               ([0, 640, 1, 300, 120], [1, 9, 33, 0, 7]), ([0, 0, 0, 0, 890], [0, 0, 0, 0, 50])]
    g, s = _state(210, *batches[0])
    _turn(g, s)  # sets the kernels up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _turn(g, s)
    for seed, which in enumerate((0, 1, 2, 3, 0)):
        g2, s2 = _state(220 + seed, *batches[which])
        for mine, other in ((g, g2), (s, s2)):
            for x in other:
                assert mine[x].shape == other[x].shape, x
                mine[x].copy_(other[x])
        _turn(g2, s2)
        graph.replay()
        assert _same(_results(g, s), _results(g2, s2)), which
