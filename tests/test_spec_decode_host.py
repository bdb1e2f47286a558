"""Speculative decoding over the bf16 paged cache without a GPU: the fp64 oracle against closed
forms, the C structures, and the refusals of the C entry points and of the binding."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import varlen_flashattention_gb300 as jfa
from oracle import attention as att
from oracle import spec_decode as sd
from varlen_flashattention_gb300 import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA_INC = "/usr/local/cuda/include"
bf16, f32, i32, i64 = torch.bfloat16, torch.float32, torch.int32, torch.int64


# ------------------------------------------------------------------ the oracle

def test_oracle_rotation():
    x = np.array([[1.0, 2.0, 3.0, 4.0, 9.0]])
    c, s = np.array([0.0, 0.6]), np.array([1.0, 0.8])  # a quarter turn, and (3, 4) / 5
    assert np.allclose(sd.rotate(x, c, s), [[-3.0, 0.6 * 2 - 0.8 * 4, 1.0, 0.6 * 4 + 0.8 * 2, 9.0]])
    assert np.allclose(sd.rotate(x, c, s, True), [[-2.0, 1.0, 0.6 * 3 - 0.8 * 4, 0.6 * 4 + 0.8 * 3, 9.0]])


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_depends_on_distance(interleaved):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 16))
    angle = np.arange(50)[:, None] * 10.0 ** (-np.arange(4) / 2.0)
    c, s = np.cos(angle), np.sin(angle)
    dots = [float((sd.rotate(q, c[p], s[p], interleaved) * sd.rotate(k, c[p - 7], s[p - 7], interleaved)).sum())
            for p in (7, 20, 49)]
    assert np.allclose(dots, dots[0])
    z = (q[0, 0] + 1j * q[0, 1 if interleaved else 4]) * np.exp(1j * angle[9, 0])
    y = sd.rotate(q, c[9], s[9], interleaved)
    assert np.allclose([y[0, 0], y[0, 1 if interleaved else 4]], [z.real, z.imag])


def test_oracle_tree_closed_form():
    # two cached tokens, drafts 0 and 1 both behind them: siblings do not see each other
    kc = np.zeros((3, 2, 1, 2))
    vc = np.zeros((3, 2, 1, 2))
    table, L = np.array([[2, 0]]), 4
    for t, (key, val) in enumerate([(0.0, 1.0), (0.0, 3.0), (np.log(2.0), 6.0), (np.log(6.0), 10.0)]):
        kc[sd.cell(table[0], 2, t)] = [[key, 0.0]]
        vc[sd.cell(table[0], 2, t)] = [[val, -val]]
    q = np.ones((2, 1, 2))
    O, LSE, absO, _ = sd.decode_tree(q, kc, vc, table, [L], [0, 2], 1.0, mask=[0b01, 0b10])
    assert np.allclose(O[:, 0, 0], [(1 + 3 + 2 * 6) / 4, (1 + 3 + 6 * 10) / 8]) and np.allclose(O[..., 1], -O[..., 0])
    assert np.allclose(LSE[:, 0], np.log([4.0, 8.0])) and np.allclose(absO, np.abs(O))


def test_oracle_chain_is_the_decode_of_the_last_tokens():
    rng = np.random.default_rng(1)
    B, n, Hq, Hkv, d, P = 2, 3, 4, 2, 128, 4
    kc, vc = rng.standard_normal((2, 8, P, Hkv, d))
    table, lens = np.array([[5, 1, 7], [0, 2, 3]]), [11, 3]
    q = rng.standard_normal((B * n, Hq, d))
    O, LSE, *_ = sd.decode_tree(q, kc, vc, table, lens, [0, n, 2 * n], 0.1)
    Or, Lr = att.decode_smallq_forward(q.reshape(B, n, Hq, d), kc, vc, table, np.array(lens), P, 0.1)
    assert np.allclose(O.reshape(Or.shape), Or, atol=1e-12) and np.allclose(LSE.reshape(Lr.shape), Lr, atol=1e-12)


def test_oracle_empty_rows_and_accept():
    rng = np.random.default_rng(2)
    kc, vc = rng.standard_normal((2, 2, 4, 1, 2))
    table = np.array([[1, 0]])
    O, LSE, *_ = sd.decode_tree(rng.standard_normal((2, 1, 2)), kc, vc, table, [2], [0, 2], 1.0, mask=[0, 2])
    assert (O[0] == 0).all() and LSE[0, 0] == -np.inf and np.allclose(O[1, 0], vc[1, 1, 0])
    was = sd.gather(kc, table[0], 7)
    lens = sd.accept(kc, vc, table, [7], [0, 5], [[1, 4, 3]], [3])
    assert lens[0] == 5 and (sd.gather(kc, table[0], 7) == was[[0, 1, 3, 6, 5, 5, 6]]).all()


# ------------------------------------------------------------------ C structures and refusals

STRUCTS = {"jfa_cache_append_rope_args": _abi.CacheAppendRopeArgs, "jfa_decode_tree_args": _abi.DecodeTreeArgs,
           "jfa_cache_accept_args": _abi.CacheAcceptArgs}


def test_struct_layouts_match_c(tmp_path):
    gcc = shutil.which("gcc")
    if gcc is None or not os.path.exists(os.path.join(CUDA_INC, "cuda_runtime_api.h")):
        pytest.skip("gcc or CUDA headers missing")
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "jfa.h"', "int main(void) {"]
    for cname, py in STRUCTS.items():
        lines.append(f'printf("{cname} size %zu\\n", sizeof({cname}));')
        for f, _ in py._fields_:
            lines.append(f'printf("{cname} {f} %zu\\n", offsetof({cname}, {f}));')
    lines.append("return 0; }")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.check_call([gcc, "-I", os.path.join(ROOT, "include"), "-I", CUDA_INC, str(src), "-o", str(exe)])
    got = {}
    for line in subprocess.check_output([str(exe)], text=True).split("\n"):
        if line:
            s, f, v = line.split()
            got[(s, f)] = int(v)
    for cname, py in STRUCTS.items():
        assert got[(cname, "size")] == ctypes.sizeof(py), cname
        for f, _ in py._fields_:
            assert got[(cname, f)] == getattr(py, f).offset, (cname, f)


@pytest.fixture(scope="module")
def lib():
    from __graft_entry__ import build
    build()
    return jfa.library()


X = 4096  # an aligned address that nothing reads
APPEND = dict(q=X, k=X, v=X, new_offsets=X, positions=None, cos_table=X, sin_table=X, q_out=8 * X, k_cache=X, v_cache=X,
              page_table=X, seqlens_k=X, q_stride=512, k_stride=256, v_stride=256, batch=2, q_heads=4, kv_heads=2,
              head_dim=128, rot_dim=128, interleaved=0, table_rows=100, page_size=16, num_pages=8, max_pages=4, total_new=5)
TREE = dict(q=X, k_cache=X, v_cache=X, page_table=X, seqlens_k=X, q_offsets=X, tree_mask=X, batch=2, q_heads=4,
            kv_heads=2, head_dim=128, page_size=16, num_pages=8, max_pages=4, total_q=5, max_q=64, scale=0.1, o=8 * X, lse=X,
            main_kernel_events=None)
ACCEPT = dict(k_cache=X, v_cache=X, page_table=X, seqlens_k=X, q_offsets=X, accepted=X, counts=X, batch=2, kv_heads=2,
              head_dim=128, page_size=16, num_pages=8, max_pages=4, width=4, new_seqlens=2 * X)
CACHE = [dict(batch=-1), dict(kv_heads=0), dict(page_size=0), dict(num_pages=-1), dict(max_pages=-1), dict(k_cache=None),
         dict(v_cache=X + 8), dict(page_table=None), dict(page_table=X + 2), dict(seqlens_k=None),
         dict(num_pages=2 ** 27, page_size=16), dict(max_pages=2 ** 27, page_size=16)]
INV, UNS, WS = _abi.JFA_ERR_INVALID_ARG, _abi.JFA_ERR_UNSUPPORTED, _abi.JFA_ERR_WORKSPACE_TOO_SMALL
BAD = [(n, c, INV) for n in ("append", "tree", "accept") for c in CACHE] + \
    [(n, dict(head_dim=192), UNS) for n in ("append", "tree", "accept")] + \
    [("append", c, INV) for c in (
        dict(new_offsets=None), dict(total_new=-1), dict(total_new=2 ** 31 - 1), dict(rot_dim=8), dict(rot_dim=144),
        dict(rot_dim=-16), dict(interleaved=2), dict(table_rows=-1), dict(q_heads=0), dict(k=None), dict(v=X + 8),
        dict(k_stride=248), dict(v_stride=260), dict(q_stride=504), dict(q_out=None), dict(q_out=X, q_stride=1024),
        dict(cos_table=None), dict(sin_table=X + 8), dict(positions=X + 1), dict(batch=0), dict(total_new=2 ** 31 - 100),
        dict(q_out=X + 1024), dict(q_out=X - 2048), dict(q_out=X + 5104))] + \
    [("tree", c, INV) for c in (
        dict(q_offsets=None), dict(q_heads=5), dict(q_heads=0), dict(total_q=-1), dict(max_q=0), dict(scale=0.0),
        dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(o=X + 8), dict(lse=X + 2),
        dict(tree_mask=X + 4), dict(total_q=2 ** 30),
        dict(o=X), dict(o=X + 5104), dict(o=X - 2048))] + \
    [("tree", dict(max_q=65), UNS), ("tree", dict(q_heads=258), UNS)] + \
    [("accept", c, INV) for c in (dict(q_offsets=None), dict(width=-1), dict(counts=None), dict(accepted=None),
                                  dict(new_seqlens=None), dict(new_seqlens=X), dict(batch=2 ** 29, kv_heads=2),
                                  dict(seqlens_k=2 * X), dict(counts=2 * X), dict(counts=2 * X - 4),
                                  dict(q_offsets=2 * X - 8), dict(accepted=2 * X - 28), dict(page_table=2 * X - 28))] + \
    [("accept", dict(width=65), UNS)]
CALLS = {"append": ("jfa_cache_append_rope", _abi.CacheAppendRopeArgs, APPEND),
         "tree": ("jfa_decode_tree", _abi.DecodeTreeArgs, TREE), "accept": ("jfa_cache_accept", _abi.CacheAcceptArgs, ACCEPT)}


@pytest.mark.parametrize("which,change,status", BAD, ids=lambda x: str(x))
def test_c_refusals(lib, which, change, status):
    name, struct, good = CALLS[which]
    a = struct(**{**good, **change})
    assert getattr(lib, name)(ctypes.byref(a), X, 1 << 40, None) == status


@pytest.mark.parametrize("which", list(CALLS))
def test_c_refuses_bad_workspaces(lib, which):
    name, struct, good = CALLS[which]
    f = getattr(lib, name)
    assert f(None, X, 1 << 40, None) == INV
    a = struct(**good)
    assert f(ctypes.byref(a), None, 1 << 40, None) == INV and f(ctypes.byref(a), X + 16, 1 << 40, None) == INV
    if which != "tree":  # the tree decode asks the device for its size first
        assert f(ctypes.byref(a), X, 128, None) == WS
    assert getattr(lib, name + "_workspace_size")(ctypes.byref(a)) >= 256
    assert getattr(lib, name + "_workspace_size")(None) == 0


def _tensors():
    z = torch.zeros
    return dict(k_cache=z(8, 16, 2, 128, dtype=bf16), v_cache=z(8, 16, 2, 128, dtype=bf16),
                page_table=z(3, 4, dtype=i32), seqlens_k=z(3, dtype=i32), offsets=z(4, dtype=i32))


def _call(which, **change):
    z = torch.zeros
    t = _tensors()
    if which == "append":
        t = dict(q=z(5, 4, 128, dtype=bf16), k=z(5, 2, 128, dtype=bf16), v=z(5, 2, 128, dtype=bf16), **t, cos=z(9, 64),
                 sin=z(9, 64), positions=None, q_out=None)
        f, names = jfa.jfa_cache_append_rope, ("q", "k", "v", "k_cache", "v_cache", "page_table", "seqlens_k", "offsets",
                                               "cos", "sin")
    elif which == "tree":
        t = dict(q=z(5, 4, 128, dtype=bf16), **t, tree_mask=z(5, dtype=i64), o=None, lse=None)
        f, names = jfa.jfa_decode_tree, ("q", "k_cache", "v_cache", "page_table", "seqlens_k", "offsets", "tree_mask")
    else:
        t = dict(**t, accepted=z(3, 4, dtype=i32), counts=z(3, dtype=i32), new_seqlens=None)
        f, names = jfa.jfa_cache_accept, ("k_cache", "v_cache", "page_table", "seqlens_k", "offsets", "accepted", "counts")
    t.update(change)
    args = [t.pop(n) for n in names]
    return f(*args, **t)


Z = torch.zeros
SHARED = [(dict(k_cache=Z(8, 16, 2, 128)), TypeError), (dict(v_cache=Z(8, 16, 1, 128, dtype=bf16)), ValueError),
          (dict(k_cache=Z(8, 16, 256, dtype=bf16)), ValueError), (dict(page_table=Z(2, 4, dtype=i32)), ValueError),
          (dict(page_table=Z(3, 4, dtype=i64)), TypeError), (dict(seqlens_k=Z(4, dtype=i32)), ValueError),
          (dict(offsets=Z(3, dtype=i32)), ValueError), (dict(offsets=None), TypeError),
          (dict(k_cache=Z(8, 2, 16, 128, dtype=bf16).transpose(1, 2)), ValueError)]


@pytest.mark.parametrize("which,change,error", [(n, c, e) for n in CALLS for c, e in SHARED] + [
    ("append", dict(q=Z(5, 4, 64, dtype=bf16)), ValueError), ("append", dict(q=Z(4, 4, 128, dtype=bf16)), ValueError),
    ("append", dict(k=Z(5, 2, 128)), TypeError), ("append", dict(k=None), TypeError),
    ("append", dict(v=Z(6, 2, 128, dtype=bf16)), ValueError),
    ("append", dict(k=Z(5, 128, 2, dtype=bf16).transpose(1, 2)), ValueError),
    ("append", dict(k=Z(5, 260, dtype=bf16)[:, :256].unflatten(1, (2, 128))), ValueError),
    ("append", dict(v=Z(1, 2, 128, dtype=bf16).expand(5, 2, 128)), ValueError),
    ("append", dict(cos=None), TypeError), ("append", dict(sin=Z(8, 64)), ValueError),
    ("append", dict(cos=Z(9, 72), sin=Z(9, 72)), ValueError), ("append", dict(cos=Z(9, 4), sin=Z(9, 4)), ValueError),
    ("append", dict(cos=Z(9, 64, dtype=bf16)), TypeError), ("append", dict(positions=Z(4, dtype=i32)), ValueError),
    ("append", dict(positions=Z(5, dtype=i64)), TypeError), ("append", dict(q=None, q_out=Z(5, 4, 128, dtype=bf16)), ValueError),
    ("append", dict(q_out=Z(5, 3, 128, dtype=bf16)), ValueError),
    ("tree", dict(q=Z(5, 4, 64, dtype=bf16)), ValueError), ("tree", dict(q=Z(5, 512, dtype=bf16)), ValueError),
    ("tree", dict(tree_mask=Z(5, dtype=i32)), TypeError), ("tree", dict(tree_mask=Z(6, dtype=i64)), ValueError),
    ("tree", dict(o=Z(4, 4, 128, dtype=bf16)), ValueError), ("tree", dict(lse=Z(4, 5)), ValueError),
    ("accept", dict(accepted=Z(2, 4, dtype=i32)), ValueError), ("accept", dict(accepted=Z(3, dtype=i32)), ValueError),
    ("accept", dict(counts=Z(3, dtype=i64)), TypeError), ("accept", dict(new_seqlens=Z(2, dtype=i32)), ValueError),
], ids=lambda x: str(list(x)) if isinstance(x, dict) else str(x))
def test_binding_refusals(which, change, error):
    with pytest.raises(error):
        _call(which, **change)


@pytest.mark.parametrize("which", list(CALLS))
def test_binding_asks_for_the_device(which):
    with pytest.raises(ValueError, match="CUDA"):
        _call(which)


@pytest.mark.parametrize("struct,pack", [(_abi.CacheAppendRopeArgs, _abi.pack_cache_append_rope),
                                         (_abi.DecodeTreeArgs, _abi.pack_decode_tree),
                                         (_abi.CacheAcceptArgs, _abi.pack_cache_accept)])
def test_packed_arguments_are_the_struct(struct, pack):
    values = [i + 1.5 if t is _abi.c_f32 else 7 * i + 1 for i, (_, t) in enumerate(struct._fields_)]
    packed = pack(*values)
    assert len(packed) == ctypes.sizeof(struct)
    back = struct.from_buffer_copy(packed)
    assert [getattr(back, f) for f, _ in struct._fields_] == values


@pytest.mark.parametrize("which,change", [("tree", dict(max_q=2 ** 40)), ("append", dict(k_stride=2 ** 63)),
                                          ("accept", dict(width=-2 ** 31 - 1))])
def test_packed_arguments_that_do_not_fit(which, change):
    struct, good = CALLS[which][1:]
    with pytest.raises(ValueError, match=struct.__name__):
        _abi.packer(struct)(*[{**good, **change}[f] or 0 for f, _ in struct._fields_])
