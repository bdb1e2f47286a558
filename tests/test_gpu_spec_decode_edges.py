"""Speculative decoding over the bf16 paged cache at its edges: batches of every shape against 64-bit
PyTorch on the device, caches past 2^31 elements, captured and replayed turns, other streams, calls
that run at the same time. The bounds are those of tests/test_gpu_spec_decode.py."""
import random

import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from tests.test_gpu_spec_decode import as_i64, cache, dev, make, tables, words

pytestmark = pytest.mark.gpu
bf16, i32 = torch.bfloat16, torch.int32


def reference(q, kc, vc, table, lens, offs, scale, mask=None):
    """O, LSE, sum_j P_j |v_j| and max_j scale sum_d |q_d k_jd| of every row, in 64 bits."""
    total, Hq, d = q.shape
    P, Hkv = kc.shape[1:3]
    G = Hq // Hkv
    f64 = dict(dtype=torch.float64, device=q.device)
    O, aO = torch.zeros(total, Hq, d, **f64), torch.zeros(total, Hq, d, **f64)
    LSE, A = torch.full((total, Hq), -torch.inf, **f64), torch.zeros(total, Hq, **f64)
    for b in range(len(lens)):
        o0, n, L = offs[b], offs[b + 1] - offs[b], lens[b]
        if n == 0:
            continue
        t = torch.arange(L, device=q.device)
        at = (table[b].long()[t // P], t % P)
        k, v = kc[at].double(), vc[at].double()
        see = torch.ones(n, L, dtype=torch.bool, device=q.device)
        if mask is None:
            see[:, L - n:] = torch.ones(n, n, device=q.device).tril().bool()
        else:
            j = torch.arange(n, device=q.device)
            see[:, L - n:] = (mask[o0:o0 + n, None] >> j & 1).bool()
        x = q[o0:o0 + n].double().view(n, Hkv, G, d)
        s = scale * torch.einsum("nhgd,thd->hngt", x, k)
        s = s.masked_fill(~see[None, :, None, :], -torch.inf)
        z = torch.logsumexp(s, -1)
        p = torch.exp(s - torch.where(torch.isinf(z), torch.zeros_like(z), z)[..., None])
        rows = slice(o0, o0 + n)
        O[rows] = torch.einsum("hngt,thd->nhgd", p, v).reshape(n, Hq, d)
        aO[rows] = torch.einsum("hngt,thd->nhgd", p, v.abs()).reshape(n, Hq, d)
        LSE[rows] = z.permute(1, 0, 2).reshape(n, Hq)
        A[rows] = (scale * torch.einsum("nhgd,thd->hngt", x.abs(), k.abs()).amax(-1)).permute(1, 0, 2).reshape(n, Hq)
    return O, LSE, aO, A


def close(o, lse, ref, longest, d, what=""):
    O, LSE, aO, A = ref
    n = O.shape[0]
    o, lse = o[:n].double(), lse[:n].double()
    ds = (d + 8) * 2.0 ** -23 * A + 2.0 ** -20
    bound = (2.0 ** -8 + longest / 16 * 2.0 ** -23 + 2.0 ** -13 + 2 * ds)[..., None] * aO + 2.0 ** -8 * O.abs() + 2.0 ** -134
    worst = ((o - O).abs() - bound).max().item() if O.numel() else -1
    assert worst <= 0, f"{what}: O over its bound by {worst:.3e}"
    none = torch.isneginf(LSE)
    assert torch.equal(torch.isneginf(lse), none) and (o[none] == 0).all(), what
    e = torch.where(none, 0.0, (lse - LSE).abs() - (ds + (LSE.abs() + 1) * 2.0 ** -21))
    assert (e <= 0).all(), f"{what}: LSE over its bound by {e.max().item():.3e}"


@pytest.mark.parametrize("seed", range(24))
def test_tree_of_any_shape(seed):
    rng = random.Random(seed)
    d, P = rng.choice([64, 128]), rng.choice([1, 2, 5, 8, 16, 16, 24, 40, 64, 128, 384])
    Hkv, G = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 7, 8, 12, 16, 33])
    B = rng.choice([1, 2, 7, 30, 200])
    most = rng.choice([1, 2, 8, 17, 33, 64])
    hi = rng.choice([0, 30, 128, 300, 1100, 5000]) // (1 if B < 100 else 4)
    new = [rng.choice([0, rng.randint(1, most), most]) for _ in range(B)]
    c = make(seed, [rng.randint(0, hi) for _ in range(B)], new, Hkv, d, P, wide=rng.choice([0, 3]))
    g = dev(c)
    q = torch.randn(sum(new), G * Hkv, d, generator=torch.Generator().manual_seed(seed)).to(bf16).cuda()
    kind = rng.choice(["tree", "bits", None])
    mask = None if kind is None else as_i64(words(c["rng"], new, kind))
    o, lse = jfa.jfa_decode_tree(q, *cache(g), g["offs"], mask, max_q=rng.choice([most, 64]), scale=0.15, check=True)
    for x in ("kc", "vc"):
        g[x].nan_to_num_(0)
    ref = reference(q, g["kc"], g["vc"], g["table"], c["lens"].tolist(), c["offs"].tolist(), 0.15, mask)
    close(o, lse, ref, max(c["lens"]), d, f"seed {seed}: B {B} most {most} Hkv {Hkv} G {G} d {d} P {P} {kind}")


def test_tree_long_and_many_rows():
    """Two sequences of tens of thousands of tokens, 1024 rows a KV head beside 16."""
    new = [64, 1]
    c = make(50, [40000, 65000], new, 1, 128, 64)
    g = dev(c)
    q = torch.randn(65, 16, 128, generator=torch.Generator().manual_seed(50)).to(bf16).cuda()
    mask = as_i64(words(c["rng"], new, "tree"))
    o, lse = jfa.jfa_decode_tree(q, *cache(g), g["offs"], mask, check=True)
    for x in ("kc", "vc"):
        g[x].nan_to_num_(0)
    close(o, lse, reference(q, g["kc"], g["vc"], g["table"], c["lens"].tolist(), c["offs"].tolist(), 128 ** -0.5, mask),
          65001, 128)


def test_append_of_many_tokens():
    """More tokens than get a block each: the form with a warp a token, padded and strided."""
    rng = np.random.default_rng(51)
    for d, Hq, Hkv, rot, inter, P in ((128, 5, 2, 128, False, 16), (64, 8, 8, 32, True, 3), (128, 1, 1, 96, False, 128)):
        new = [700, 0, 1, 1300, 64, 0]
        before = [0, 10, 500, 33, 128, 0]
        lens = [a + n for a, n in zip(before, new)]
        pages = sum(-(-x // P) for x in lens)
        table = torch.full((6, max(-(-x // P) for x in lens)), -1, dtype=i32)
        perm, at = torch.from_numpy(rng.permutation(pages)).to(i32), 0
        for b, x in enumerate(lens):
            table[b, :-(-x // P)] = perm[at:at - (-x // P)]
            at += -(-x // P)
        n = sum(new)
        qkv = torch.randn(n + 5, (Hq + 2 * Hkv) * d + 8, device="cuda").to(bf16)[:, :-8]
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([Hq * d, Hkv * d, Hkv * d], dim=1))
        kc, vc = (torch.full((pages, P, Hkv, d), 7.0, dtype=bf16, device="cuda") for _ in range(2))
        offs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=i32).cuda()
        cos, sin = (torch.from_numpy(x).cuda() for x in tables(2000, rot))
        out = torch.full((n + 5, Hq, d), 7.0, dtype=bf16, device="cuda")
        jfa.jfa_cache_append_rope(q, k, v, kc, vc, table.cuda(), torch.tensor(lens, dtype=i32).cuda(), offs, cos, sin,
                                  interleaved=inter, q_out=out, check=True)
        assert (out[n:] == 7).all()
        seen = torch.zeros(pages, P, dtype=torch.bool)
        lo, hi = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        for b in range(6):
            rows, t = slice(int(offs[b]), int(offs[b + 1])), torch.arange(before[b], lens[b])
            where = (table[b].long()[t // P], t % P)
            seen[where] = True
            assert torch.equal(vc[where], v[rows])
            for x, y in ((q[rows], out[rows]), (k[rows], kc[where])):
                x, y = x.double(), y.double()
                cc, ss = cos[t].double()[:, None], sin[t].double()[:, None]
                w = x.clone()
                w[..., lo], w[..., hi] = x[..., lo] * cc - x[..., hi] * ss, x[..., hi] * cc + x[..., lo] * ss
                top = x.abs().amax(-1, keepdim=True) if x.numel() else 0
                assert ((y - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -21 * top + 2.0 ** -134).all()
                assert torch.equal(y[..., rot:], x[..., rot:])
        assert (kc[~seen.cuda()] == 7).all() and (vc[~seen.cuda()] == 7).all()


def test_caches_past_2_31_elements():
    """Pages behind the 2^31st element of the caches: append, attention, accept."""
    P, H, d, pages = 16, 8, 128, 140_000
    kc = torch.zeros(pages, P, H, d, dtype=bf16, device="cuda")
    vc = torch.zeros(pages, P, H, d, dtype=bf16, device="cuda")
    assert kc.numel() > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(52)
    lens = [300, 45]
    table = torch.stack([pages - 1 - torch.arange(20), pages - 40 - torch.arange(20)]).to(i32).cuda()
    offs = torch.tensor([0, 300, 345], dtype=i32).cuda()
    k, v, q = (torch.randn(345, h, d, generator=gen, device="cuda").to(bf16) for h in (H, H, 32))
    seq = torch.tensor(lens, dtype=i32).cuda()
    jfa.jfa_cache_append_rope(None, k, v, kc, vc, table, seq, offs, None, None, check=True)
    assert int((kc[:pages - 100] != 0).sum()) == 0  # nothing went to the other end
    new = torch.tensor([0, 17, 20], dtype=i32).cuda()
    o, lse = jfa.jfa_decode_tree(q[:20], kc, vc, table, seq, new, check=True)
    close(o, lse, reference(q[:20], kc, vc, table, lens, [0, 17, 20], d ** -0.5), 300, d)
    path = torch.tensor([[2, 5, 16], [1, 2, 0]], dtype=i32).cuda()
    left = jfa.jfa_cache_accept(kc, vc, table, seq, new, path, torch.tensor([3, 2], dtype=i32).cuda(), check=True)
    assert left.tolist() == [286, 44]
    for b, first, rows in ((0, 283, [2, 5, 16]), (1, 42, [1, 2])):
        t = torch.arange(first, first + len(rows)).cuda()
        src = torch.tensor([int(offs[b]) + first + j for j in rows]).cuda()
        assert torch.equal(kc[table[b][t // P].long(), t % P], k[src])
        assert torch.equal(vc[table[b][t // P].long(), t % P], v[src])


def _turn(g, s, ws=None, stream=None):
    """One turn: drafts in, attention, accepted drafts kept."""
    ws = ws or [None] * 3
    jfa.jfa_cache_append_rope(s["q"], s["k"], s["v"], *cache(g), g["offs"], s["cos"], s["sin"], q_out=s["qr"],
                              workspace=ws[0], stream=stream)
    jfa.jfa_decode_tree(s["qr"], *cache(g), g["offs"], s["mask"], o=s["o"], lse=s["lse"], workspace=ws[1], stream=stream)
    jfa.jfa_cache_accept(*cache(g), g["offs"], s["path"], s["count"], new_seqlens=s["left"], workspace=ws[2], stream=stream)


def _turn_state(seed):
    new = [12, 1, 0, 30, 7]
    c = make(seed, [100, 700, 5, 33, 256], new, 2, 128, 16)
    g = dev(c)
    rng = c["rng"]
    n = sum(new)
    s = {x: torch.from_numpy(rng.standard_normal((n, h, 128)).astype(np.float32)).to(bf16).cuda()
         for x, h in (("q", 8), ("k", 2), ("v", 2))}
    s["cos"], s["sin"] = (torch.from_numpy(x).cuda() for x in tables(1000, 128))
    s["mask"] = as_i64(words(rng, new, "tree"))
    s["path"] = torch.from_numpy(np.stack([np.sort(rng.permutation(max(m, 5))[:5]) % max(m, 1) for m in new]).astype(np.int32)).cuda()
    s["count"] = torch.tensor([min(m, 1) * min(5, m) for m in new], dtype=i32).cuda()
    s["qr"], s["o"] = torch.zeros_like(s["q"]), torch.zeros_like(s["q"])
    s["lse"], s["left"] = torch.zeros(n, 8, device="cuda"), torch.zeros_like(g["lens"])
    return g, s


def _results(g, s):
    return [x.clone() for x in (g["kc"].nan_to_num(9), g["vc"].nan_to_num(9), s["qr"], s["o"], s["lse"], s["left"])]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_turn_replays_with_new_inputs():
    g, s = _turn_state(60)
    _turn(g, s)  # sets the kernels up
    torch.cuda.synchronize()
    start = {x: g[x].clone() for x in ("kc", "vc")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _turn(g, s)
    for seed in (61, 62):
        g2, s2 = _turn_state(seed)
        for x in ("kc", "vc"):
            start[x] = g2[x].clone()
        _turn(g2, s2)
        want = _results(g2, s2)
        # other pages, lengths as before: the graph reads what the tensors hold now
        if g["kc"].shape != g2["kc"].shape:
            continue
        for x in ("kc", "vc"):
            g[x].copy_(start[x])
        g["table"].copy_(g2["table"])
        for x in ("q", "k", "v", "mask", "path", "count"):
            s[x].copy_(s2[x])
        for _ in range(2):
            for x in ("kc", "vc"):
                g[x].copy_(start[x])
            graph.replay()
            assert _same(_results(g, s), want)


def test_turn_on_other_streams():
    g, s = _turn_state(63)
    was = {x: g[x].clone() for x in ("kc", "vc")}
    _turn(g, s)
    want = _results(g, s)
    for how in ("argument", "current"):
        for x in ("kc", "vc"):
            g[x].copy_(was[x])
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        if how == "argument":
            _turn(g, s, stream=side)
        else:
            with torch.cuda.stream(side):
                _turn(g, s)
        side.synchronize()
        assert _same(_results(g, s), want), how


def test_turns_at_the_same_time():
    """Two batches on two streams, again and again, with workspaces of their own that hold rubbish."""
    states = [_turn_state(64), _turn_state(65)]
    wants, ws, was = [], [], []
    for g, s in states:
        was.append({x: g[x].clone() for x in ("kc", "vc")})
        _turn(g, s)
        wants.append(_results(g, s))
        ws.append([torch.randint(0, 256, (n,), dtype=torch.uint8, device="cuda") for n in (256, 64 << 20, 256)])
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    for _ in range(10):
        for (g, s), w, old, side in zip(states, ws, was, streams):
            with torch.cuda.stream(side):
                for x in ("kc", "vc"):
                    g[x].copy_(old[x])
                _turn(g, s, w)
        torch.cuda.synchronize()
        for (g, s), want, w in zip(states, wants, ws):
            assert _same(_results(g, s), want)
            assert all(jfa.jfa_read_device_status(x) == (0, 0) for x in w)


def test_tree_events_and_status_of_a_reused_workspace():
    g, s = _turn_state(66)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    jfa.jfa_decode_tree(s["q"], *cache(g), g["offs"], s["mask"], workspace=ws, events=ev, check=True)
    torch.cuda.synchronize()
    assert 0 < ev[0].elapsed_time(ev[1]) < 1000
    lens = g["lens"].clone()
    g["lens"][0] = -1
    jfa.jfa_decode_tree(s["q"], *cache(g), g["offs"], s["mask"], workspace=ws)
    assert jfa.jfa_read_device_status(ws) == (6, 501)
    g["lens"].copy_(lens)
    jfa.jfa_decode_tree(s["q"], *cache(g), g["offs"], s["mask"], workspace=ws)
    assert jfa.jfa_read_device_status(ws) == (0, 0)
    with pytest.raises(ValueError, match="workspace"):
        jfa.jfa_decode_tree(s["q"], *cache(g), g["offs"], s["mask"], workspace=ws[:1024])


def test_captured_turns_keep_their_workspaces():
    """Two captured turns whose calls got workspaces of their own, replayed at the same time between calls
    and tensors that take and give back memory of every size."""
    runs = []
    for seed, explicit in ((67, False), (68, True)):
        g, s = _turn_state(seed)
        was = {x: g[x].clone() for x in ("kc", "vc")}
        _turn(g, s)
        want = _results(g, s)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            for x in ("kc", "vc"):
                g[x].copy_(was[x])
            _turn(g, s, stream=side if explicit else None)
        runs.append((g, s, want, side, graph, was))  # the graph reads was
    other, t = _turn_state(69)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(8):
        held = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (256, 512, 4 << 10, 1 << 20, 20 << 20, 80 << 20)]
        for g, s, want, side, graph, _ in runs:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
        _turn(other, t)
        torch.cuda.synchronize()
        assert all((x == 255).all() for x in held)
        for g, s, want, side, graph, _ in runs:
            assert _same(_results(g, s), want)


def test_turns_of_several_threads():
    """Calls from four host threads, each on its own stream."""
    import threading

    states = [_turn_state(70 + i) for i in range(4)]
    wants, was = [], []
    for g, s in states:
        was.append({x: g[x].clone() for x in ("kc", "vc")})
        _turn(g, s)
        wants.append(_results(g, s))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        g, s = states[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                for x in ("kc", "vc"):
                    g[x].copy_(was[i][x])
                _turn(g, s)
                if not _same(_results(g, s), wants[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    torch.cuda.synchronize()
    assert not wrong


def test_outputs_that_lie_over_inputs():
    """The tree decode may not write over Q, nor accept over what it reads; rotated Q may, row on row."""
    g, s = _turn_state(74)
    for o in (s["q"], torch.empty(0, device="cuda")):
        with pytest.raises((jfa.JfaError, TypeError)):
            jfa.jfa_decode_tree(s["q"], *cache(g), g["offs"], s["mask"], o=o)
    for name in ("count", "lens"):
        new = s["count"] if name == "count" else g["lens"]
        with pytest.raises(jfa.JfaError):
            jfa.jfa_cache_accept(*cache(g), g["offs"], s["path"], s["count"], new_seqlens=new)
    both = torch.zeros(s["q"].shape[0] + 1, 8, 128, dtype=bf16, device="cuda")
    with pytest.raises(jfa.JfaError):
        jfa.jfa_cache_append_rope(both[:-1], s["k"], s["v"], *cache(g), g["offs"], s["cos"], s["sin"], q_out=both[1:])
    jfa.jfa_cache_append_rope(both[:-1], s["k"], s["v"], *cache(g), g["offs"], s["cos"], s["sin"], q_out=both[:-1], check=True)
