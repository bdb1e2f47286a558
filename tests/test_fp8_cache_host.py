"""The 8-bit paged cache without a GPU: the fp64 oracle against closed forms, the
C structures, and the refusals of the C entry points and of the binding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import kv_cache as kvo
from oracle.attention import attention_forward, e4m3_decode
from varlen_flashattention_gb300 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA_INC = "/usr/local/cuda/include"
bf16, f32, i32, u8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


# ------------------------------------------------------------------ the oracle

def test_encode_matches_the_format():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    assert (kvo.e4m3_encode(e4m3_decode(codes)) == codes).all()  # every value is its own nearest
    x = np.random.default_rng(0).uniform(-448, 448, 4096).astype(np.float32)
    torch_codes = torch.from_numpy(x).to(torch.float8_e4m3fn).view(u8).numpy()
    assert (kvo.e4m3_encode(x.astype(np.float64)) == torch_codes).all()
    # midpoints go to the even code
    pos = kvo.E4M3
    mid = (pos[:-1] + pos[1:]) / 2
    assert (kvo.e4m3_encode(mid) % 2 == 0).all()


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (448.0001, 2.0), (1.0, 2.0 ** -8), (1.75, 2.0 ** -8),
                                        (1.7500001, 2.0 ** -7), (0.0, 2.0 ** -126), (2.0 ** -130, 2.0 ** -126)])
def test_block_scale(amax, scale):
    assert kvo.block_scale(amax) == scale


def _cache(rng, pages, P, block, H, d):
    kc, vc = (rng.integers(0, 127, (pages, P, H, d)).astype(np.uint8) for _ in range(2))
    ks, vs = (2.0 ** rng.integers(-12, -4, (pages, P // block, H)).astype(np.float64) for _ in range(2))
    return kc, vc, ks, vs


def test_oracle_decode_is_attention_over_the_values():
    rng = np.random.default_rng(1)
    kc, vc, ks, vs = _cache(rng, 4, 8, 4, 1, 16)
    table, L = np.array([[2, 0, 3]]), 19
    q = rng.standard_normal((1, L, 1, 16))  # every token a query: causal self-attention
    O, LSE, W, _, _, _ = kvo.decode(q, kc, vc, ks, vs, table, [L], 0.25, weights=np.ones((1, 1, 24)), decay=0.5)
    K, V = kvo.gather(kc, ks, table[0], L), kvo.gather(vc, vs, table[0], L)
    Oa, La = attention_forward(q[0], K, V, [0, L], 0.25, True)
    assert np.allclose(O[0], Oa, atol=1e-12) and np.allclose(LSE[0].T, La, atol=1e-12)
    assert np.isclose(W[0].sum(), L + 0.5 * L)  # every row's weights sum to one


def test_oracle_append_holds_values_within_half_a_step():
    rng = np.random.default_rng(2)
    kc, vc, ks, vs = _cache(rng, 6, 8, 4, 2, 16)
    k, v = (rng.standard_normal((11, 2, 16)) for _ in range(2))
    table = np.array([[5, 1, 0], [2, 3, 4]])
    before = kvo.gather(kc, ks, table[0], 3)
    kvo.append(k, v, kc, vc, ks, vs, table, [3 + 7, 4], [0, 7, 11])
    K = kvo.gather(kc, ks, table[0], 10)
    # e4m3 rounds within 2^-4, or half the smallest step 2^-10 of the block's scale
    step = np.repeat(ks[table[0][:2]].reshape(-1, 2), 4, 0)[:10, :, None] * 2.0 ** -10
    assert (np.abs(K[3:] - k[:7]) <= np.maximum(np.abs(k[:7]) * 2.0 ** -4, step[3:])).all()
    assert (np.abs(K[:3] - before) <= np.maximum(np.abs(before) * 2.0 ** -4, step[:3])).all()


def test_oracle_evict_keeps_the_largest_in_order():
    rng = np.random.default_rng(3)
    kc, vc, ks, vs = _cache(rng, 8, 4, 2, 1, 16)
    w = np.zeros((1, 1, 16), dtype=np.float32)
    w[0, 0, :13] = [0, 5, 1, 1, 1, np.nan, 9, 0, 1, 2, 0, 0, 0]
    table, new = np.array([[0, 1, 2, 3]]), np.array([[6, 7]])
    V = kvo.gather(vc, vs, table[0], 13)
    kept, lens, nw = kvo.evict(kc, vc, ks, vs, table, [13], w, 7, new, first=1, recent=2)
    assert kept[0, 0].tolist() == [0, 1, 2, 6, 9, 11, 12] and lens.tolist() == [7]
    assert nw[0, 0].tolist() == [0, 5, 1, 9, 2, 0, 0, 0]
    # a power-of-two scale moves codes unchanged but for subnormals of the new block
    got = kvo.gather(vc, vs, new[0], 7)
    tiny = np.repeat(vs[new[0]].reshape(-1, 1), 2, 0)[:7, :, None] * 2.0 ** -10
    assert (np.abs(got - V[kept[0, 0]]) <= np.where(np.abs(V[kept[0, 0]]) < tiny * 16, tiny, 0)).all()


# ------------------------------------------------------------------ the C ABI

@pytest.fixture(scope="module")
def lib():
    from __graft_entry__ import build
    build()
    return jfa.library()


STRUCTS = {"jfa_cache_append_fp8_args": _abi.CacheAppendFp8Args, "jfa_decode_fp8_args": _abi.DecodeFp8Args,
           "jfa_cache_evict_fp8_args": _abi.CacheEvictFp8Args}


def test_struct_layouts_match_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime_api.h")):
        pytest.skip("gcc or CUDA headers missing")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "jfa.h"', "int main(void) {"]
    for cname, py in STRUCTS.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        lines += [f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));' for f, _ in py._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0; }"]))
    subprocess.check_call([gcc, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INC, str(src), "-o", str(exe)])
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in subprocess.check_output([str(exe)], text=True).splitlines()}
    for cname, py in STRUCTS.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


FAKE = 0x10000  # aligned, never dereferenced: every call below returns before any CUDA work


def _decode_args(**kw):
    a = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, seqlens_k=FAKE, batch=4,
             q_len=1, q_heads=32, kv_heads=8, head_dim=128, page_size=16, block_size=16, num_pages=100, max_pages=10,
             scale=0.1, o=FAKE, lse=FAKE, weights=None, weights_out=None, decay=1.0, main_kernel_events=None)
    return _abi.DecodeFp8Args(**{**a, **kw})


def _append_args(**kw):
    a = dict(k=FAKE, v=FAKE, new_offsets=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE,
             page_table=FAKE, seqlens_k=FAKE, batch=4, kv_heads=8, head_dim=128, page_size=16, block_size=16,
             num_pages=100, max_pages=10, total_new=4, max_new=1, weights=None)
    return _abi.CacheAppendFp8Args(**{**a, **kw})


def _evict_args(**kw):
    a = dict(k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, page_table=FAKE, seqlens_k=FAKE, weights=FAKE,
             new_page_table=FAKE, batch=4, kv_heads=8, head_dim=128, page_size=16, block_size=16, num_pages=100,
             max_pages=10, new_max_pages=4, keep=64, first=4, recent=16, kept=FAKE, new_seqlens=2 * FAKE,
             new_weights=2 * FAKE)
    return _abi.CacheEvictFp8Args(**{**a, **kw})


ENTRIES = {"jfa_decode_fp8": _decode_args, "jfa_cache_append_fp8": _append_args, "jfa_cache_evict_fp8": _evict_args}


@pytest.mark.parametrize("entry", list(ENTRIES))
def test_cache_arguments_are_refused(lib, entry):
    call, make = getattr(lib, entry), ENTRIES[entry]
    assert call(None, FAKE, 1 << 40, None) == _abi.JFA_ERR_INVALID_ARG
    for bad in (dict(batch=-1), dict(kv_heads=0), dict(page_size=0), dict(block_size=0), dict(num_pages=-1),
                dict(max_pages=-1), dict(page_size=24, block_size=16), dict(k_cache=FAKE + 8), dict(v_cache=None),
                dict(k_scale=FAKE + 2), dict(v_scale=None), dict(page_table=FAKE + 2), dict(seqlens_k=None),
                dict(num_pages=1 << 27), dict(max_pages=1 << 27)):
        assert call(ctypes.byref(make(**bad)), FAKE, 1 << 40, None) == _abi.JFA_ERR_INVALID_ARG, bad
    for bad in (dict(head_dim=192), dict(head_dim=96), dict(block_size=256, page_size=256),
                dict(block_size=12, page_size=24)):
        assert call(ctypes.byref(make(**bad)), FAKE, 1 << 40, None) == _abi.JFA_ERR_UNSUPPORTED, bad
    a = make()
    assert call(ctypes.byref(a), FAKE + 16, 1 << 40, None) == _abi.JFA_ERR_INVALID_ARG
    need = getattr(lib, entry + "_workspace_size")(ctypes.byref(a))
    assert need >= 256
    assert call(ctypes.byref(a), FAKE, need - 1, None) == _abi.JFA_ERR_WORKSPACE_TOO_SMALL


def test_decode_arguments_are_refused(lib):
    for bad in (dict(q_len=0), dict(q_heads=0), dict(q_heads=30), dict(scale=0.0), dict(scale=float("nan")),
                dict(q=FAKE + 8), dict(o=None), dict(lse=FAKE + 2), dict(weights=FAKE),
                dict(weights=FAKE, weights_out=FAKE, decay=-0.5),
                dict(weights=FAKE, weights_out=FAKE, decay=float("inf")), dict(weights_out=FAKE + 2),
                dict(batch=1 << 30)):
        assert lib.jfa_decode_fp8(ctypes.byref(_decode_args(**bad)), FAKE, 1 << 60, None) == \
            _abi.JFA_ERR_INVALID_ARG, bad
    for bad in (dict(q_len=5), dict(kv_heads=1)):  # 20 and 32 rows
        assert lib.jfa_decode_fp8(ctypes.byref(_decode_args(**bad)), FAKE, 1 << 60, None) == \
            _abi.JFA_ERR_UNSUPPORTED, bad
    # the scores of every tile are kept for the weights: 4 sequences x 160 tokens x 32 heads
    size = lib.jfa_decode_fp8_workspace_size
    assert size(ctypes.byref(_decode_args(weights_out=FAKE))) - size(ctypes.byref(_decode_args())) >= 4 * 4 * 160 * 32
    assert size(None) == 0


def test_append_and_evict_arguments_are_refused(lib):
    for bad in (dict(total_new=-1), dict(max_new=-1), dict(batch=0), dict(new_offsets=None), dict(k=FAKE + 8), dict(v=None),
                dict(weights=FAKE + 2), dict(batch=1 << 25, max_new=1 << 20)):
        assert lib.jfa_cache_append_fp8(ctypes.byref(_append_args(**bad)), FAKE, 1 << 40, None) == \
            _abi.JFA_ERR_INVALID_ARG, bad
    for bad in (dict(keep=0), dict(first=-1), dict(recent=-1), dict(first=50), dict(new_max_pages=3),
                dict(new_max_pages=-1), dict(new_page_table=None), dict(kept=FAKE + 2), dict(new_seqlens=FAKE),
                dict(new_weights=FAKE), dict(weights=None)):
        assert lib.jfa_cache_evict_fp8(ctypes.byref(_evict_args(**bad)), FAKE, 1 << 40, None) == \
            _abi.JFA_ERR_INVALID_ARG, bad


def test_append_takes_any_bound_on_new_tokens(lib):
    """max_new, a bound, does not decide what is refused; an empty workspace ends the calls before any CUDA work."""
    call = lib.jfa_cache_append_fp8
    for good in (dict(max_new=2 ** 31 - 1), dict(batch=16384, kv_heads=64, total_new=16383 + 131072, max_new=131072),
                 dict(batch=1 << 20, kv_heads=128, total_new=1 << 20, max_new=1 << 20)):
        assert call(ctypes.byref(_append_args(**good)), FAKE, 0, None) == _abi.JFA_ERR_WORKSPACE_TOO_SMALL, good
    for bad in (dict(batch=1 << 25, max_new=1), dict(batch=1 << 20, kv_heads=256, total_new=1 << 20),
                dict(kv_heads=32767, total_new=2 ** 31 - 1, max_new=2 ** 31 - 1)):
        assert call(ctypes.byref(_append_args(**bad)), FAKE, 0, None) == _abi.JFA_ERR_INVALID_ARG, bad


# ------------------------------------------------------------------ the binding

def _t(B=3, P=16, block=8, H=2, d=64, pages=10, mp=4):
    kc = torch.zeros(pages, P, H, d, dtype=u8)
    ks = torch.ones(pages, P // block, H)
    return dict(k_cache=kc, v_cache=kc.clone(), k_scale=ks, v_scale=ks.clone(),
                page_table=torch.zeros(B, mp, dtype=i32), seqlens_k=torch.ones(B, dtype=i32))


CACHE_ERRORS = [
    (dict(v_cache=torch.zeros(9, 16, 2, 64, dtype=u8)), ValueError, "v_cache must have shape"),
    (dict(k_cache=torch.zeros(10, 16, 2, 64)), TypeError, "k_cache must be"),
    (dict(k_scale=torch.ones(10, 3, 2)), ValueError, "v_scale must have shape|divisor of the page size"),
    (dict(k_scale=torch.ones(10, 3, 2), v_scale=torch.ones(10, 3, 2)), ValueError, "divisor of the page size"),
    (dict(k_scale=torch.ones(10, 2, 1)), ValueError, "k_scale must have shape"),
    (dict(v_scale=torch.ones(10, 1, 2)), ValueError, "v_scale must have shape"),
    (dict(page_table=torch.zeros(2, 4, dtype=i32)), ValueError, "page_table must have shape"),
    (dict(seqlens_k=torch.ones(3, dtype=torch.int64)), TypeError, "seqlens_k must be"),
    (dict(page_table=torch.zeros(4, 3, dtype=i32).t()), ValueError, "page_table must be contiguous"),
    (dict(v_cache=torch.zeros(10, 2, 16, 64, dtype=u8).transpose(1, 2)), ValueError, "v_cache must be contiguous"),
    (dict(k_scale=None), TypeError, "k_scale must be a torch.Tensor"),
]


@pytest.mark.parametrize("bad,kind,match", CACHE_ERRORS)
def test_binding_checks_the_cache(bad, kind, match):
    t = {**_t(), **bad}
    k = torch.zeros(5, 2, 64, dtype=bf16)
    off = torch.tensor([0, 2, 4, 5], dtype=i32)
    w = torch.zeros(3, 2, 64)
    calls = [lambda: jfa.jfa_cache_append_fp8(k, k, **t, new_offsets=off, max_new=2),
             lambda: jfa.jfa_decode_fp8(torch.zeros(3, 1, 4, 64, dtype=bf16), **t),
             lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=16, new_page_table=torch.zeros(3, 1, dtype=i32))]
    for call in calls:
        with pytest.raises(kind, match=match):
            call()


def test_binding_checks_the_rest():
    t = _t()
    k = torch.zeros(5, 2, 64, dtype=bf16)
    off = torch.tensor([0, 2, 4, 5], dtype=i32)
    w = torch.zeros(3, 2, 64)
    q = torch.zeros(3, 1, 4, 64, dtype=bf16)
    new = torch.zeros(3, 1, dtype=i32)
    for match, call in [
        ("k must have shape", lambda: jfa.jfa_cache_append_fp8(torch.zeros(5, 1, 64, dtype=bf16), k, **t,
                                                               new_offsets=off, max_new=2)),
        ("v must have shape", lambda: jfa.jfa_cache_append_fp8(k, k[:4], **t, new_offsets=off, max_new=2)),
        ("new_offsets must have shape", lambda: jfa.jfa_cache_append_fp8(k, k, **t, new_offsets=off[:3], max_new=2)),
        ("weights must have shape", lambda: jfa.jfa_cache_append_fp8(k, k, **t, new_offsets=off, max_new=2,
                                                                     weights=w[:2])),
        ("q must have shape", lambda: jfa.jfa_decode_fp8(q[:2], **t)),
        ("q must have shape", lambda: jfa.jfa_decode_fp8(torch.zeros(3, 1, 4, 128, dtype=bf16), **t)),
        ("weights must have shape", lambda: jfa.jfa_decode_fp8(q, **t, weights=torch.zeros(3, 2, 63))),
        ("weights_out must have shape", lambda: jfa.jfa_decode_fp8(q, **t, weights=w, weights_out=w[:2])),
        ("lse must have shape", lambda: jfa.jfa_decode_fp8(q, **t, lse=torch.zeros(3, 4))),
        ("new_page_table must have shape", lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=16,
                                                                           new_page_table=new[:2])),
        ("new_page_table holds 16", lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=17, new_page_table=new)),
        ("first [+] recent at most", lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=16, new_page_table=new,
                                                                     first=9, recent=8)),
        ("kept must have shape", lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=16, new_page_table=new,
                                                                 kept=torch.zeros(3, 2, 8, dtype=i32))),
        # all in order: the only complaint is the device
        ("must be on a CUDA device", lambda: jfa.jfa_cache_append_fp8(k, k, **t, new_offsets=off, max_new=2,
                                                                      weights=w)),
        ("must be on a CUDA device", lambda: jfa.jfa_decode_fp8(q, **t, weights=w)),
        ("must be on a CUDA device", lambda: jfa.jfa_cache_evict_fp8(**t, weights=w, keep=16, new_page_table=new)),
    ]:
        with pytest.raises(ValueError, match=match):
            call()
