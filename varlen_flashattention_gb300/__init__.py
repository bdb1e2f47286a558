"""Jagged (varlen) FlashAttention for GB300: Python binding of libjfa.so.

The functions here carry the names of the C entry points and only marshal
arguments: they check shapes and dtypes, allocate outputs and the workspace
with PyTorch when the caller does not pass them, and call the library on the
current CUDA stream. Every step of the computation runs in the sm_103a
kernels; there is no CPU or PyTorch fallback.

    jfa_fwd               jagged self-attention forward -> (O, LSE)
    jfa_bwd               its recompute-based backward -> (dQ, dK, dV)
    jfa_fwd_broadcast_q   one dense Q shared by a jagged K/V batch -> (O, LSE)
    jfa_bwd_broadcast_q   its backward, dQ summed over the batch -> (dQ, dK, dV)
    jfa_decode_splitkv    split-KV decode over a paged GQA cache -> (O, LSE)
    jfa_fwd_varlen        separate query / key lengths, grouped KV heads -> (O, LSE)
    jfa_bwd_varlen        its backward -> (dQ, dK, dV)
    jfa_decode_smallq     paged split-KV decode of a few query tokens per sequence -> (O, LSE)
    jfa_fwd_fp8           jagged forward over FP8 (e4m3) inputs with per-tensor descales -> (O, LSE)
    jfa_fp8_quantize_v    bf16 V -> e4m3 V in the layout jfa_fwd_fp8 reads (its vt argument)
    jfa_cache_append_fp8  new tokens' K and V quantized into an 8-bit paged cache (block scales)
    jfa_decode_fp8        decode over the 8-bit paged cache, with accumulated attention weights -> (O, LSE)
    jfa_cache_evict_fp8   the tokens of the largest accumulated weights moved to new pages
    jfa_cache_append_rope new tokens' K and V written to a bf16 paged cache, Q and K rotated on the way
    jfa_decode_tree       attention of drafted trees (or chains) of up to 64 tokens over the paged cache -> (O, LSE)
    jfa_cache_accept      the accepted drafts moved to the places behind the earlier tokens
    jfa_trace_enable      registers a per-role event trace buffer (JFA_TRACE builds; see trace.py)
    jfa_trace_compiled    1 if the loaded library records traces
    jagged_attention      autograd wrapper of jfa_fwd / jfa_bwd
    varlen_attention      autograd wrapper of jfa_fwd_varlen / jfa_bwd_varlen
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _abi

__all__ = [
    "JfaError", "jfa_fwd", "jfa_bwd", "jfa_fwd_broadcast_q", "jfa_bwd_broadcast_q", "jfa_decode_splitkv",
    "jfa_read_device_status", "jagged_attention", "library", "jfa_fwd_varlen", "jfa_bwd_varlen",
    "varlen_attention", "jfa_decode_smallq", "jfa_selftest_wait_timeout", "jfa_fwd_fp8",
    "jfa_trace_enable", "jfa_trace_compiled", "jfa_fp8_quantize_v",
    "jfa_cache_append_fp8", "jfa_decode_fp8", "jfa_cache_evict_fp8",
    "jfa_cache_append_rope", "jfa_decode_tree", "jfa_cache_accept",
]


class JfaError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = library().jfa_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def library():
    return _abi.load()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, dtype, shape):
    """Type, dtype, shape (a tuple, or an int: the number of dimensions) and
    layout of one argument. The kernels address every tensor from the shapes
    of q (and k), so each buffer is checked against them here; the device is
    checked by _device once every tensor of the call is known."""
    if type(t) is torch.Tensor and t.dtype is dtype and (t.dim() if type(shape) is int else t.shape) == shape and \
            t.is_contiguous():
        return  # the usual case; what follows names what is wrong
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if isinstance(shape, int):
        if t.dim() != shape:
            raise ValueError(f"{name} must have {shape} dimensions, got {tuple(t.shape)}")
    elif t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_offsets(t, name):
    _need(t, name, torch.int32, 1)
    if t.numel() < 1:
        raise ValueError(f"{name} must hold batch + 1 >= 1 entries")


def _device(**tensors):
    """The one CUDA device that holds every given tensor (None entries are
    skipped); the call runs there, on that device's stream."""
    first = None
    for name, t in tensors.items():
        if t is None:
            continue
        i = t.get_device()  # -1 on the host
        if first is None:
            first, idx = t, i
        if i < 0:
            raise ValueError(f"{name} must be on a CUDA device")
        if i != idx:
            raise ValueError(f"{name} is on cuda:{i}, the other tensors on cuda:{idx}")
    return first.device


def _stream(stream):
    """The cudaStream_t of a torch stream, by default the current one (asked for by its
    handle: building torch's stream object costs several microseconds a call)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream


def _events(events):
    if events is None:
        return None, None
    for e in events:  # torch creates the CUDA event lazily, on its first record
        if not e.cuda_event:
            e.record()
    arr = (ctypes.c_void_p * 2)(events[0].cuda_event, events[1].cuda_event)
    return ctypes.cast(arr, ctypes.c_void_p), arr


def _workspace(nbytes, device, workspace):
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor")
    if workspace.get_device() != device.index:
        raise ValueError(f"workspace is on {workspace.device}, the call runs on {device}")
    if _nbytes(workspace) < nbytes:
        raise ValueError(f"workspace holds {_nbytes(workspace)} bytes, needs {nbytes}")
    return workspace


def _nbytes(t):
    return t.numel() * t.element_size()


_entries = {}  # the library's functions by name


def _entry(name):
    f = _entries.get(name)
    if f is None:
        f = _entries[name] = getattr(library(), name)
    return f


def _run(entry, size_entry, a, device, workspace, stream, check):
    """Sizes the workspace, calls the entry point on `device` and its stream,
    and with check=True reads the device status back (a stream sync)."""
    if device.index == torch.cuda.current_device():
        _run_here(entry, size_entry, a, device, workspace, stream, check)
    else:
        with torch.cuda.device(device):
            _run_here(entry, size_entry, a, device, workspace, stream, check)


def _run_here(entry, size_entry, a, device, workspace, stream, check):
    ref = ctypes.byref(a)
    need = _entry(size_entry)(ref)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device_index != device.index:
        raise ValueError(f"stream belongs to {stream.device}, the call runs on {device}")
    else:
        raw = stream.cuda_stream
    if workspace is None:
        nbytes = max(need, 256)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
        if stream is not None:
            ws.record_stream(stream)  # allocated on the current stream, used on this one
    else:
        ws = _workspace(need, device, workspace)
        nbytes = _nbytes(ws)
    status = _entry(entry)(ref, ws.data_ptr(), nbytes, raw)
    if status != _abi.JFA_OK:
        raise JfaError(status, entry)
    if check:
        _finish(ws, check, stream, entry)


def _run_packed(entry, packed, need, index, workspace, stream, check):
    """_run for the arguments of a call as the bytes of its struct, and a known workspace size.
    A workspace of its own comes from PyTorch's allocator without a tensor around it (half a
    microsecond against five beside a launch); it belongs to the call's stream."""
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _run_packed(entry, packed, need, index, workspace, stream, check)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device_index != index:
        raise ValueError(f"stream belongs to {stream.device}, the call runs on cuda:{index}")
    else:
        raw = stream.cuda_stream
    if workspace is not None:
        _workspace(need, torch.device("cuda", index), workspace)
        _started(entry, _abi.packed_entry(entry)(packed, workspace.data_ptr(), _nbytes(workspace), raw))
        if check:
            _finish(workspace, check, stream, entry)
        return
    ws = torch._C._cuda_cudaCachingAllocator_raw_alloc(need, raw)
    try:
        _started(entry, _abi.packed_entry(entry)(packed, ws, need, raw))
        if check:
            d = ctypes.c_int32(0)
            st = _entry("jfa_read_device_status")(ws, raw, ctypes.byref(d))
            if st != _abi.JFA_OK:
                raise JfaError(st, f"{entry} (device, detail {d.value})")
    finally:
        torch._C._cuda_cudaCachingAllocator_raw_delete(ws)


def _started(entry, status):
    if status != _abi.JFA_OK:
        raise JfaError(status, entry)


def _check(status, where):
    if status != _abi.JFA_OK:
        raise JfaError(status, where)


def jfa_read_device_status(workspace, stream=None):
    """Synchronises the stream; returns (status, detail) of the last call that used `workspace`."""
    d = ctypes.c_int32(0)
    st = library().jfa_read_device_status(_ptr(workspace), _stream(stream), ctypes.byref(d))
    return int(st), int(d.value)


def jfa_selftest_wait_timeout(budget_us=20000, workspace=None, stream=None):
    """Runs the failure-detection self-test (a pipeline wait whose input never
    arrives, bounded to budget_us). Returns (status, detail, second_stage_aborted)."""
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    _check(library().jfa_selftest_wait_timeout(int(budget_us), _ptr(ws), _stream(stream)), "jfa_selftest_wait_timeout")
    st, detail = jfa_read_device_status(ws, stream)
    aborted = int(ws[16:20].view(torch.int32).item())
    return st, detail, aborted


def jfa_trace_compiled():
    """1 if the loaded library was built with JFA_TRACE (it records traces), else 0."""
    return int(library().jfa_trace_compiled())


def jfa_trace_enable(buffer, records_per_warp=1024):
    """Registers `buffer` (a zeroed uint8 CUDA tensor of at least
    trace.buffer_bytes(SMs, records_per_warp) bytes) for the per-role event
    records of later calls; None turns recording off. Raises JfaError
    (unsupported) unless the library was built with JFA_TRACE."""
    if buffer is not None:
        if not isinstance(buffer, torch.Tensor) or not buffer.is_cuda or not buffer.is_contiguous():
            raise TypeError("buffer must be a contiguous CUDA tensor")
        _check(library().jfa_trace_enable(_ptr(buffer), _nbytes(buffer), int(records_per_warp)), "jfa_trace_enable")
    else:
        _check(library().jfa_trace_enable(None, 0, 0), "jfa_trace_enable")


def _finish(ws, check, stream, where):
    if check:
        st, detail = jfa_read_device_status(ws, stream)
        if st != _abi.JFA_OK:
            e = JfaError(st, f"{where} (device, detail {detail})")
            raise e


# ---------------------------------------------------------------- forward / backward

def jfa_fwd(q, k, v, offsets, max_seqlen, scale=None, causal=False, o=None, lse=None, workspace=None,
            stream=None, events=None, check=False):
    """Jagged self-attention forward. q, k, v: bf16 [total, H, d]; offsets: int32 [B+1] (CUDA).
    Returns O bf16 [total, H, d] and LSE fp32 [H, total] (natural log)."""
    _need(q, "q", torch.bfloat16, 3)
    total, H, d = q.shape
    _need(k, "k", torch.bfloat16, q.shape)
    _need(v, "v", torch.bfloat16, q.shape)
    _need_offsets(offsets, "offsets")
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (H, total))
    dev = _device(q=q, k=k, v=v, offsets=offsets, o=o, lse=lse)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((H, total), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.FwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(offsets), offsets.numel() - 1, H, d, int(max_seqlen),
                     total, scale, int(bool(causal)), _ptr(o), _ptr(lse), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_fwd", "jfa_fwd_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_bwd(q, k, v, o, dout, lse, offsets, max_seqlen, scale=None, causal=False, head_chunk=0,
            dq=None, dk=None, dv=None, workspace=None, stream=None, events=None, check=False):
    """Recompute-based backward of jfa_fwd. Returns dQ, dK, dV bf16 [total, H, d]."""
    _need(q, "q", torch.bfloat16, 3)
    total, H, d = q.shape
    for n, t in (("k", k), ("v", v), ("o", o), ("dout", dout)):
        _need(t, n, torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (H, total))
    _need_offsets(offsets, "offsets")
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        if t is not None:
            _need(t, n, torch.bfloat16, q.shape)
    dev = _device(q=q, k=k, v=v, o=o, dout=dout, lse=lse, offsets=offsets, dq=dq, dk=dk, dv=dv)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    a = _abi.BwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(offsets),
                     offsets.numel() - 1, H, d, int(max_seqlen), total, scale, int(bool(causal)), int(head_chunk),
                     _ptr(dq), _ptr(dk), _ptr(dv), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_bwd", "jfa_bwd_workspace_size", a, dev, workspace, stream, check)
    return dq, dk, dv


def jfa_fwd_broadcast_q(q, k, v, kv_offsets, max_seqlen_k, scale=None, o=None, lse=None, workspace=None,
                        stream=None, events=None, check=False):
    """Broadcast-Q forward. q: bf16 [Lq, H, d] shared by every sequence; k, v jagged [total_k, H, d].
    Returns O bf16 [B, Lq, H, d] and LSE fp32 [B, H, Lq]."""
    _need(q, "q", torch.bfloat16, 3)
    Lq, H, d = q.shape
    _need(k, "k", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, (k.shape[0], H, d))
    _need(v, "v", torch.bfloat16, k.shape)
    _need_offsets(kv_offsets, "kv_offsets")
    B = kv_offsets.numel() - 1
    if o is not None:
        _need(o, "o", torch.bfloat16, (B, Lq, H, d))
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, H, Lq))
    dev = _device(q=q, k=k, v=v, kv_offsets=kv_offsets, o=o, lse=lse)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty((B, Lq, H, d), dtype=torch.bfloat16, device=dev) if o is None else o
    lse = torch.empty((B, H, Lq), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.BcastFwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(kv_offsets), B, Lq, H, d, int(max_seqlen_k),
                          k.shape[0], scale, _ptr(o), _ptr(lse), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_fwd_broadcast_q", "jfa_bcast_fwd_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_bwd_broadcast_q(q, k, v, o, dout, lse, kv_offsets, max_seqlen_k, scale=None, dq=None, dk=None, dv=None,
                        workspace=None, stream=None, events=None, check=False):
    """Broadcast-Q backward. Returns dQ bf16 [Lq, H, d] summed over the batch, dK, dV [total_k, H, d]."""
    _need(q, "q", torch.bfloat16, 3)
    Lq, H, d = q.shape
    _need(k, "k", torch.bfloat16, 3)
    _need(k, "k", torch.bfloat16, (k.shape[0], H, d))
    _need(v, "v", torch.bfloat16, k.shape)
    _need_offsets(kv_offsets, "kv_offsets")
    B = kv_offsets.numel() - 1
    _need(o, "o", torch.bfloat16, (B, Lq, H, d))
    _need(dout, "dout", torch.bfloat16, (B, Lq, H, d))
    _need(lse, "lse", torch.float32, (B, H, Lq))
    if dq is not None:
        _need(dq, "dq", torch.bfloat16, q.shape)
    if dk is not None:
        _need(dk, "dk", torch.bfloat16, k.shape)
    if dv is not None:
        _need(dv, "dv", torch.bfloat16, k.shape)
    dev = _device(q=q, k=k, v=v, o=o, dout=dout, lse=lse, kv_offsets=kv_offsets, dq=dq, dk=dk, dv=dv)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    a = _abi.BcastBwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(kv_offsets),
                          B, Lq, H, d, int(max_seqlen_k), k.shape[0], scale, _ptr(dq), _ptr(dk), _ptr(dv), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_bwd_broadcast_q", "jfa_bcast_bwd_workspace_size", a, dev, workspace, stream, check)
    return dq, dk, dv


def jfa_fwd_fp8(q, k, v, offsets, max_seqlen, q_descale, k_descale, v_descale, scale=None, causal=False, o=None,
                lse=None, workspace=None, stream=None, events=None, check=False, vt=None):
    """Jagged forward over FP8 inputs. q, k, v: e4m3 codes [total, H, 128] (torch.uint8 or
    torch.float8_e4m3fn); byte x of q stands for e4m3(x) * q_descale (likewise k, v).
    vt (optional): V as jfa_fp8_quantize_v wrote it for these offsets and heads; v is then
    not read (it may be None) and the call makes no pass over V.
    Returns O bf16 [total, H, 128] and LSE fp32 [H, total]."""
    qkv = []
    for n, t in (("q", q), ("k", k), ("v", v)):
        if n == "v" and t is None and vt is not None:
            qkv.append(None)
            continue
        if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
            t = t.view(torch.uint8)
        _need(t, n, torch.uint8, 3)
        qkv.append(t)
    q, k, v = qkv
    total, H, d = q.shape
    _need(k, "k", torch.uint8, q.shape)
    if v is not None:
        _need(v, "v", torch.uint8, q.shape)
    _need_offsets(offsets, "offsets")
    if vt is not None:
        _need(vt, "vt", torch.uint8, (int(library().jfa_fp8_vt_bytes(offsets.numel() - 1, H, total)),))
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (H, total))
    dev = _device(q=q, k=k, v=v, offsets=offsets, o=o, lse=lse, vt=vt)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty((total, H, d), dtype=torch.bfloat16, device=dev) if o is None else o
    lse = torch.empty((H, total), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.FwdFp8Args(_ptr(q), _ptr(k), _ptr(v), _ptr(offsets), offsets.numel() - 1, H, d, int(max_seqlen), total,
                        scale, int(bool(causal)), float(q_descale), float(k_descale), float(v_descale), _ptr(o),
                        _ptr(lse), None, _ptr(vt))
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_fwd_fp8", "jfa_fwd_fp8_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_fp8_quantize_v(v, offsets, max_seqlen, v_descale, vt=None, workspace=None, stream=None, check=False):
    """bf16 V [total, H, 128] -> e4m3(v / v_descale) in the blocks jfa_fwd_fp8 reads (see
    include/jfa.h): returns the uint8 tensor of jfa_fp8_vt_bytes(batch, H, total) bytes, to
    pass as jfa_fwd_fp8(..., vt=...)."""
    _need(v, "v", torch.bfloat16, 3)
    total, H, d = v.shape
    _need_offsets(offsets, "offsets")
    nbytes = int(library().jfa_fp8_vt_bytes(offsets.numel() - 1, H, total))
    if vt is not None:
        _need(vt, "vt", torch.uint8, (nbytes,))
    dev = _device(v=v, offsets=offsets, vt=vt)
    vt = torch.empty(nbytes, dtype=torch.uint8, device=dev) if vt is None else vt
    a = _abi.Fp8QuantizeVArgs(_ptr(v), _ptr(offsets), offsets.numel() - 1, H, d, int(max_seqlen), total,
                              float(v_descale), _ptr(vt))
    _run("jfa_fp8_quantize_v", "jfa_fp8_quantize_v_workspace_size", a, dev, workspace, stream, check)
    return vt


# ---------------------------------------------------------------- varlen / GQA

def _var_inputs(q, k, v, q_offsets, k_offsets):
    _need(q, "q", torch.bfloat16, 3)
    total_q, Hq, d = q.shape
    _need(k, "k", torch.bfloat16, 3)
    total_k, Hkv, _ = k.shape
    _need(k, "k", torch.bfloat16, (total_k, Hkv, d))
    _need(v, "v", torch.bfloat16, k.shape)
    _need_offsets(q_offsets, "q_offsets")
    _need_offsets(k_offsets, "k_offsets")
    if q_offsets.numel() != k_offsets.numel():
        raise ValueError("q_offsets and k_offsets must have the same length")
    return total_q, Hq, d, total_k, Hkv


def jfa_fwd_varlen(q, k, v, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale=None, causal=False, o=None,
                   lse=None, workspace=None, stream=None, events=None, check=False):
    """Jagged attention with separate query / key packing and grouped KV heads.
    q: bf16 [total_q, Hq, d]; k, v: bf16 [total_k, Hkv, d] with Hq % Hkv == 0; q_offsets and
    k_offsets: int32 [B+1] (CUDA). causal aligns the mask to the bottom right (key j visible to
    query i iff j <= i + L_k - L_q). Returns O bf16 [total_q, Hq, d], LSE fp32 [Hq, total_q]."""
    total_q, Hq, d, total_k, Hkv = _var_inputs(q, k, v, q_offsets, k_offsets)
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (Hq, total_q))
    dev = _device(q=q, k=k, v=v, q_offsets=q_offsets, k_offsets=k_offsets, o=o, lse=lse)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((Hq, total_q), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.VarlenFwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(q_offsets), _ptr(k_offsets), q_offsets.numel() - 1,
                           Hq, Hkv, d, int(max_seqlen_q), int(max_seqlen_k), total_q, total_k, scale,
                           int(bool(causal)), _ptr(o), _ptr(lse), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_fwd_varlen", "jfa_varlen_fwd_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_bwd_varlen(q, k, v, o, dout, lse, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale=None,
                   causal=False, head_chunk=0, dq=None, dk=None, dv=None, workspace=None, stream=None, events=None,
                   check=False):
    """Backward of jfa_fwd_varlen. Returns dQ bf16 [total_q, Hq, d] and dK, dV bf16
    [total_k, Hkv, d] (a KV head's gradient summed over the query heads that read it)."""
    total_q, Hq, d, total_k, Hkv = _var_inputs(q, k, v, q_offsets, k_offsets)
    _need(o, "o", torch.bfloat16, q.shape)
    _need(dout, "dout", torch.bfloat16, q.shape)
    _need(lse, "lse", torch.float32, (Hq, total_q))
    if dq is not None:
        _need(dq, "dq", torch.bfloat16, q.shape)
    if dk is not None:
        _need(dk, "dk", torch.bfloat16, k.shape)
    if dv is not None:
        _need(dv, "dv", torch.bfloat16, k.shape)
    dev = _device(q=q, k=k, v=v, o=o, dout=dout, lse=lse, q_offsets=q_offsets, k_offsets=k_offsets, dq=dq, dk=dk,
                  dv=dv)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    a = _abi.VarlenBwdArgs(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(dout), _ptr(lse), _ptr(q_offsets),
                           _ptr(k_offsets), q_offsets.numel() - 1, Hq, Hkv, d, int(max_seqlen_q), int(max_seqlen_k),
                           total_q, total_k, scale, int(bool(causal)), int(head_chunk), _ptr(dq), _ptr(dk), _ptr(dv),
                           None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_bwd_varlen", "jfa_varlen_bwd_workspace_size", a, dev, workspace, stream, check)
    return dq, dk, dv


# ---------------------------------------------------------------- decode

def _cache_inputs(k_cache, v_cache, page_table, seqlens_k, B, d):
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    num_pages, P, Hkv, _ = k_cache.shape
    _need(k_cache, "k_cache", torch.bfloat16, (num_pages, P, Hkv, d))
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _need(page_table, "page_table", torch.int32, 2)
    _need(page_table, "page_table", torch.int32, (B, page_table.shape[1]))
    _need(seqlens_k, "seqlens_k", torch.int32, (B,))
    return num_pages, P, Hkv


def jfa_decode_splitkv(q, k_cache, v_cache, page_table, seqlens_k, num_splits, scale=None, o=None, lse=None,
                       split_bounds=None, workspace=None, stream=None, events=None, check=False):
    """Split-KV decode over a paged GQA cache. q: bf16 [B, Hq, 128]; caches bf16
    [num_pages, page_size, Hkv, 128]; page_table int32 [B, max_pages]; seqlens_k int32 [B].
    Returns O bf16 [B, Hq, 128] and LSE fp32 [B, Hq]. If `split_bounds` (int32 [B, S, 2])
    is given, the kernel writes each split's token range into it."""
    _need(q, "q", torch.bfloat16, 3)
    B, Hq, d = q.shape
    num_pages, P, Hkv = _cache_inputs(k_cache, v_cache, page_table, seqlens_k, B, d)
    if split_bounds is not None:
        _need(split_bounds, "split_bounds", torch.int32, (B, int(num_splits), 2))
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, Hq))
    dev = _device(q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, seqlens_k=seqlens_k, o=o, lse=lse,
                  split_bounds=split_bounds)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.DecodeArgs(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens_k),
                        B, Hq, Hkv, d, P, num_pages, page_table.shape[1], int(num_splits), scale,
                        _ptr(o), _ptr(lse), _ptr(split_bounds), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_decode_splitkv", "jfa_decode_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_decode_smallq(q, k_cache, v_cache, page_table, seqlens_k, num_splits, min_split_tokens=0, scale=None,
                      o=None, lse=None, split_bounds=None, split_counts=None, workspace=None, stream=None,
                      events=None, check=False):
    """Paged split-KV decode of q_len new tokens per sequence (speculative / chunked decode).
    q: bf16 [B, q_len, Hq, 128]; caches bf16 [num_pages, page_size, Hkv, 128]; page_table int32
    [B, max_pages]; seqlens_k int32 [B] (new tokens included: token i of q_len sits at key position
    L - q_len + i and sees keys up to it). Returns O bf16 [B, q_len, Hq, 128], LSE fp32 [B, q_len, Hq].
    With min_split_tokens > 0 each sequence uses clamp(ceil(L / min_split_tokens), 1, num_splits)
    splits; `split_counts` (int32 [B]) and `split_bounds` (int32 [B, S, 2]) receive them if given."""
    _need(q, "q", torch.bfloat16, 4)
    B, ql, Hq, d = q.shape
    num_pages, P, Hkv = _cache_inputs(k_cache, v_cache, page_table, seqlens_k, B, d)
    if split_bounds is not None:
        _need(split_bounds, "split_bounds", torch.int32, (B, int(num_splits), 2))
    if split_counts is not None:
        _need(split_counts, "split_counts", torch.int32, (B,))
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, ql, Hq))
    dev = _device(q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, seqlens_k=seqlens_k, o=o, lse=lse,
                  split_bounds=split_bounds, split_counts=split_counts)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, ql, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    a = _abi.DecodeSmallqArgs(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table), _ptr(seqlens_k),
                              B, ql, Hq, Hkv, d, P, num_pages, page_table.shape[1], int(num_splits),
                              int(min_split_tokens), scale, _ptr(o), _ptr(lse), _ptr(split_bounds),
                              _ptr(split_counts), None)
    ev, _keep = _events(events)
    a.main_kernel_events = ev
    _run("jfa_decode_smallq", "jfa_decode_smallq_workspace_size", a, dev, workspace, stream, check)
    return o, lse


# ---------------------------------------------------------------- 8-bit paged cache

def _codes(t, name, shape):
    """The uint8 view of an e4m3 cache (torch.uint8 or torch.float8_e4m3fn)."""
    if isinstance(t, torch.Tensor) and t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    _need(t, name, torch.uint8, shape)
    return t


def _fp8_cache_inputs(k_cache, v_cache, k_scale, v_scale, page_table, seqlens_k):
    """Shapes of an 8-bit cache and of the batch that reads it; the scales' second
    dimension gives the block size. Returns the caches as uint8 and (num_pages, page
    size, block size, KV heads, head dim, batch, max_pages)."""
    try:  # the usual case in one test; what follows it names what is wrong
        num_pages, P, Hkv, d = shape = k_cache.shape
        pages, blocks, heads = scale_shape = k_scale.shape
        B, mp = page_table.shape
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        if (k_cache.dtype is u8 and v_cache.dtype is u8 and k_scale.dtype is f32 and v_scale.dtype is f32 and
                page_table.dtype is i32 and seqlens_k.dtype is i32 and v_cache.shape == shape and
                v_scale.shape == scale_shape and seqlens_k.shape == (B,) and pages == num_pages and heads == Hkv and
                blocks > 0 and P % blocks == 0 and k_cache.is_contiguous() and v_cache.is_contiguous() and
                k_scale.is_contiguous() and v_scale.is_contiguous() and page_table.is_contiguous() and
                seqlens_k.is_contiguous()):
            return k_cache, v_cache, (num_pages, P, P // blocks, Hkv, d, B, mp)
    except (AttributeError, TypeError, ValueError):
        pass
    k_cache = _codes(k_cache, "k_cache", 4)
    num_pages, P, Hkv, d = k_cache.shape
    v_cache = _codes(v_cache, "v_cache", k_cache.shape)
    _need(k_scale, "k_scale", torch.float32, 3)
    blocks = k_scale.shape[1]
    _need(k_scale, "k_scale", torch.float32, (num_pages, blocks, Hkv))
    _need(v_scale, "v_scale", torch.float32, k_scale.shape)
    if blocks < 1 or P % blocks != 0:
        raise ValueError(f"k_scale must hold a divisor of the page size {P} in dimension 1, got {blocks}")
    _need(seqlens_k, "seqlens_k", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    B, mp = page_table.shape
    _need(page_table, "page_table", torch.int32, (seqlens_k.numel(), mp))
    return k_cache, v_cache, (num_pages, P, P // blocks, Hkv, d, B, mp)


def jfa_cache_append_fp8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, seqlens_k, new_offsets, max_new,
                         weights=None, workspace=None, stream=None, check=False):
    """Quantizes the K and V rows of new tokens into an 8-bit paged cache, in place (see include/jfa.h).
    k, v: bf16 [total_new, Hkv, d], sequence b's rows new_offsets[b] .. new_offsets[b+1]-1 becoming its
    last tokens (seqlens_k counts them already); caches: e4m3 codes [num_pages, page_size, Hkv, d]
    (torch.uint8 or torch.float8_e4m3fn); k_scale, v_scale: fp32 [num_pages, page_size / block, Hkv];
    page_table int32 [B, max_pages]; seqlens_k int32 [B]; new_offsets int32 [B+1]; max_new >= every
    sequence's count. weights (optional, fp32 [B, Hkv, max_pages * page_size]) is set to 0 at the new
    positions. Returns (k_cache, v_cache, k_scale, v_scale)."""
    kc, vc, (num_pages, P, block, Hkv, d, B, mp) = _fp8_cache_inputs(k_cache, v_cache, k_scale, v_scale, page_table,
                                                                     seqlens_k)
    _need(k, "k", torch.bfloat16, (k.shape[0] if isinstance(k, torch.Tensor) and k.dim() else 0, Hkv, d))
    _need(v, "v", torch.bfloat16, k.shape)
    _need(new_offsets, "new_offsets", torch.int32, (B + 1,))
    if weights is not None:
        _need(weights, "weights", torch.float32, (B, Hkv, mp * P))
    dev = _device(k=k, v=v, k_cache=kc, v_cache=vc, k_scale=k_scale, v_scale=v_scale, page_table=page_table,
                  seqlens_k=seqlens_k, new_offsets=new_offsets, weights=weights)
    a = _abi.CacheAppendFp8Args(_ptr(k), _ptr(v), _ptr(new_offsets), _ptr(kc), _ptr(vc), _ptr(k_scale), _ptr(v_scale),
                                _ptr(page_table), _ptr(seqlens_k), B, Hkv, d, P, block, num_pages, mp, k.shape[0],
                                int(max_new), _ptr(weights))
    _run("jfa_cache_append_fp8", "jfa_cache_append_fp8_workspace_size", a, dev, workspace, stream, check)
    return k_cache, v_cache, k_scale, v_scale


def jfa_decode_fp8(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens_k, scale=None, weights=None, decay=1.0,
                   weights_out=None, o=None, lse=None, workspace=None, stream=None, events=None, check=False):
    """Decode of the last q_len tokens of each sequence over an 8-bit paged cache. q: bf16
    [B, q_len, Hq, d], q_len * Hq / Hkv <= 16; the cache as in jfa_cache_append_fp8; seqlens_k
    counts the query tokens (token i sits at key position L - q_len + i and sees keys up to it).
    weights (optional, fp32 [B, Hkv, max_pages * page_size]): weights_out = decay * weights + each
    cached token's attention weight, summed over the group's query heads and the query tokens, for
    the tokens of each sequence; weights is updated in place if weights_out is not given, and
    weights_out alone receives the sums. With either the workspace holds 4 bytes per query row and
    slot of page_table, whatever the lengths are. Returns O bf16 [B, q_len, Hq, d], LSE fp32 [B, q_len, Hq]."""
    kc, vc, (num_pages, P, block, Hkv, d, B, mp) = _fp8_cache_inputs(k_cache, v_cache, k_scale, v_scale, page_table,
                                                                     seqlens_k)
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        _need(q, "q", torch.bfloat16, 4)
    _, ql, Hq, _ = q.shape
    _need(q, "q", torch.bfloat16, (B, ql, Hq, d))
    if weights is not None:
        _need(weights, "weights", torch.float32, (B, Hkv, mp * P))
    if weights_out is None:
        weights_out = weights
    else:
        _need(weights_out, "weights_out", torch.float32, (B, Hkv, mp * P))
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, ql, Hq))
    dev = _device(q=q, k_cache=kc, v_cache=vc, k_scale=k_scale, v_scale=v_scale, page_table=page_table,
                  seqlens_k=seqlens_k, weights=weights, weights_out=weights_out, o=o, lse=lse)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((B, ql, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    if stream is not None:  # new memory belongs to the current stream
        o.record_stream(stream)
        lse.record_stream(stream)
    a = _abi.DecodeFp8Args(_ptr(q), _ptr(kc), _ptr(vc), _ptr(k_scale), _ptr(v_scale), _ptr(page_table),
                           _ptr(seqlens_k), B, ql, Hq, Hkv, d, P, block, num_pages, mp, scale, _ptr(o), _ptr(lse),
                           _ptr(weights), _ptr(weights_out), float(decay), None)
    if events is not None:
        a.main_kernel_events, _keep = _events(events)
    _run("jfa_decode_fp8", "jfa_decode_fp8_workspace_size", a, dev, workspace, stream, check)
    return o, lse


def jfa_cache_evict_fp8(k_cache, v_cache, k_scale, v_scale, page_table, seqlens_k, weights, keep, new_page_table,
                        first=0, recent=0, kept=None, new_seqlens=None, new_weights=None, workspace=None, stream=None,
                        check=False):
    """Cuts every sequence of an 8-bit paged cache to at most `keep` tokens: each KV head keeps its
    first `first` and last `recent` tokens and the largest weights of the rest (ties: the lower
    position), in order, in the pages of new_page_table (int32 [B, new_max_pages], room for `keep`
    tokens a row, pages that no sequence of the call holds). weights: fp32 [B, Hkv, max_pages *
    page_size], as jfa_decode_fp8 accumulates them. Returns kept int32 [B, Hkv, keep] (old positions,
    -1 past the end), new_seqlens int32 [B] and new_weights fp32 [B, Hkv, new_max_pages * page_size]."""
    kc, vc, (num_pages, P, block, Hkv, d, B, mp) = _fp8_cache_inputs(k_cache, v_cache, k_scale, v_scale, page_table,
                                                                     seqlens_k)
    keep, first, recent = int(keep), int(first), int(recent)
    _need(weights, "weights", torch.float32, (B, Hkv, mp * P))
    nmp = new_page_table.shape[1] if isinstance(new_page_table, torch.Tensor) and new_page_table.dim() == 2 else 0
    _need(new_page_table, "new_page_table", torch.int32, (B, nmp))
    if keep < 1 or first < 0 or recent < 0 or first + recent > keep:
        raise ValueError(f"keep must be >= 1 and first + recent at most keep, got {keep}, {first}, {recent}")
    if nmp * P < keep:
        raise ValueError(f"new_page_table holds {nmp * P} tokens a sequence, keep is {keep}")
    if kept is not None:
        _need(kept, "kept", torch.int32, (B, Hkv, keep))
    if new_seqlens is not None:
        _need(new_seqlens, "new_seqlens", torch.int32, (B,))
    if new_weights is not None:
        _need(new_weights, "new_weights", torch.float32, (B, Hkv, nmp * P))
    dev = _device(k_cache=kc, v_cache=vc, k_scale=k_scale, v_scale=v_scale, page_table=page_table,
                  seqlens_k=seqlens_k, weights=weights, new_page_table=new_page_table, kept=kept,
                  new_seqlens=new_seqlens, new_weights=new_weights)
    kept = torch.empty((B, Hkv, keep), dtype=torch.int32, device=dev) if kept is None else kept
    new_seqlens = torch.empty_like(seqlens_k) if new_seqlens is None else new_seqlens
    if new_weights is None:
        new_weights = torch.empty((B, Hkv, nmp * P), dtype=torch.float32, device=dev)
    if stream is not None:  # new memory belongs to the current stream
        for t in (kept, new_seqlens, new_weights):
            t.record_stream(stream)
    a = _abi.CacheEvictFp8Args(_ptr(kc), _ptr(vc), _ptr(k_scale), _ptr(v_scale), _ptr(page_table), _ptr(seqlens_k),
                               _ptr(weights), _ptr(new_page_table), B, Hkv, d, P, block, num_pages, mp, nmp, keep,
                               first, recent, _ptr(kept), _ptr(new_seqlens), _ptr(new_weights))
    _run("jfa_cache_evict_fp8", "jfa_cache_evict_fp8_workspace_size", a, dev, workspace, stream, check)
    return kept, new_seqlens, new_weights


# ---------------------------------------------------------------- speculative decoding

def _adr(t):
    return 0 if t is None else t.data_ptr()


def _paged_ok(k_cache, v_cache, page_table, seqlens_k, offsets, B):
    """The usual case of a bf16 paged cache and a batch over it, in one test: types, layouts and one
    CUDA device. What is not usual is named by _paged_inputs."""
    bf16, i32, i = torch.bfloat16, torch.int32, k_cache.get_device()
    return (i >= 0 and k_cache.dtype is bf16 and v_cache.dtype is bf16 and page_table.dtype is i32 and
            seqlens_k.dtype is i32 and offsets.dtype is i32 and v_cache.shape == k_cache.shape and
            seqlens_k.shape == (B,) and offsets.shape == (B + 1,) and v_cache.get_device() == i and
            page_table.get_device() == i and seqlens_k.get_device() == i and offsets.get_device() == i and
            k_cache.is_contiguous() and v_cache.is_contiguous() and page_table.is_contiguous() and
            seqlens_k.is_contiguous() and offsets.is_contiguous())


def _paged_inputs(k_cache, v_cache, page_table, seqlens_k, offsets, offsets_name):
    """Shapes of a bf16 paged cache and of the batch over it: (num_pages, page size, KV heads,
    head dim, batch, max_pages)."""
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    num_pages, P, Hkv, d = k_cache.shape
    _need(v_cache, "v_cache", torch.bfloat16, k_cache.shape)
    _need(seqlens_k, "seqlens_k", torch.int32, 1)
    _need(page_table, "page_table", torch.int32, 2)
    B, mp = page_table.shape
    _need(page_table, "page_table", torch.int32, (seqlens_k.numel(), mp))
    _need(offsets, offsets_name, torch.int32, (B + 1,))
    return num_pages, P, Hkv, d, B, mp


def _need_rows(t, name, heads, d, rows):
    """bf16 [rows, heads, d] whose rows may lie apart (a view of a fused projection's
    output); returns the row stride in elements."""
    if type(t) is torch.Tensor and t.dtype is torch.bfloat16 and t.dim() == 3 and \
            t.shape == (t.shape[0] if rows is None else rows, heads, d):
        stride, inner, last = t.stride()
        if last == 1 and inner == d and stride >= heads * d and stride % 8 == 0:
            return stride  # the usual case; what follows names what is wrong
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1:] != (heads, d) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must have shape {('rows' if rows is None else rows, heads, d)}, got {tuple(t.shape)}")
    stride, inner, last = t.stride()
    if t.shape[0] <= 1 or t.is_contiguous():
        stride = heads * d
    if t.numel() and (last != 1 or (heads > 1 and inner != d) or stride < heads * d or stride % 8 != 0):
        raise ValueError(f"{name}: a row's heads must be contiguous and its stride a multiple of 8, got {t.stride()}")
    return stride


def _same_device(index, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != index:
            return False
    return True


def jfa_cache_append_rope(q, k, v, k_cache, v_cache, page_table, seqlens_k, new_offsets, cos, sin, positions=None,
                          interleaved=False, q_out=None, workspace=None, stream=None, check=False):
    """Writes the K and V rows of new tokens into a bf16 paged cache, K rotated by its position on the
    way, and rotates Q (see include/jfa.h). q: bf16 [total_new, Hq, d] or None; k, v: bf16 [total_new,
    Hkv, d]; the rows of the three may be strided (views of a fused projection's output). Sequence b's
    rows new_offsets[b] .. new_offsets[b+1]-1 (int32 [B+1]) become its last tokens (seqlens_k, int32 [B],
    counts them already); caches bf16 [num_pages, page_size, Hkv, d] with d 64 or 128; page_table int32 [B,
    max_pages]. cos, sin: fp32 [positions, rot_dim / 2] with rot_dim a multiple of 16 up to d, or both
    None (nothing turns). positions (optional, int32 [total_new]): the tables' rows, by default the
    tokens' places in their sequences. Pairs are columns (j, j + rot_dim / 2), or neighbours if
    interleaved. Returns the rotated Q (q_out, which may be q itself, and no part of k or v; None
    without q); its rows behind new_offsets[B] are not written."""
    try:
        num_pages, P, Hkv, d = k_cache.shape
        B, mp = page_table.shape
        usual = _paged_ok(k_cache, v_cache, page_table, seqlens_k, new_offsets, B)
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        num_pages, P, Hkv, d, B, mp = _paged_inputs(k_cache, v_cache, page_table, seqlens_k, new_offsets, "new_offsets")
    ks = _need_rows(k, "k", Hkv, d, None)
    total = k.shape[0]
    vs = _need_rows(v, "v", Hkv, d, total)
    Hq = qs = 0
    if q is not None:
        Hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        qs = _need_rows(q, "q", Hq, d, total)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    rows = rot = 0
    if cos is not None or sin is not None:
        _need(cos, "cos", torch.float32, 2)
        rows, rot = cos.shape
        rot *= 2
        _need(sin, "sin", torch.float32, cos.shape)
        if rot > d or rot % 16 != 0:
            raise ValueError(f"cos must hold a multiple of 8 up to {d // 2} columns, got {cos.shape[1]}")
    if positions is not None:
        _need(positions, "positions", torch.int32, (total,))
    if q_out is not None:
        _need(q_out, "q_out", torch.bfloat16, q.shape)
    if not usual or not _same_device(k_cache.get_device(), k, v, q, cos, sin, positions, q_out):
        _device(k=k, v=v, q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, seqlens_k=seqlens_k,
                new_offsets=new_offsets, cos=cos, sin=sin, positions=positions, q_out=q_out)
    dev = k_cache.device
    if q is not None and q_out is None:
        q_out = torch.empty((total, Hq, d), dtype=torch.bfloat16, device=dev)
        if stream is not None:  # new memory belongs to the current stream
            q_out.record_stream(stream)
    packed = _abi.pack_cache_append_rope(
        _adr(q), k.data_ptr(), v.data_ptr(), new_offsets.data_ptr(), _adr(positions), _adr(cos), _adr(sin), _adr(q_out),
        k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), seqlens_k.data_ptr(), qs, ks, vs, B, Hq, Hkv, d,
        rot, 1 if interleaved else 0, rows, P, num_pages, mp, total)
    _run_packed("jfa_cache_append_rope", packed, 256, dev.index, workspace, stream, check)
    return q_out


_tree_workspaces = {}  # bytes of the workspace by device, group, head dim and max_q


def jfa_decode_tree(q, k_cache, v_cache, page_table, seqlens_k, q_offsets, tree_mask=None, max_q=64, scale=None, o=None,
                    lse=None, workspace=None, stream=None, events=None, check=False):
    """Attention of each sequence's new tokens over its bf16 paged cache, which holds them already (see
    include/jfa.h). q: bf16 [total_q, Hq, d], sequence b's rows q_offsets[b] .. q_offsets[b+1]-1 (int32
    [B+1]), at most max_q <= 64 of them; the cache as in jfa_cache_append_rope, seqlens_k counting the new
    tokens. A row sees all tokens before the new ones and new token j iff bit j of its tree_mask (int64 or
    uint64 [total_q]) is set: its ancestors in the tree and itself; without tree_mask j <= i. Returns O bf16
    [total_q, Hq, d] and LSE fp32 [total_q, Hq]; rows behind q_offsets[B] are not written."""
    try:
        num_pages, P, Hkv, d = k_cache.shape
        B, mp = page_table.shape
        total, Hq, qd = q.shape
        usual = (_paged_ok(k_cache, v_cache, page_table, seqlens_k, q_offsets, B) and q.dtype is torch.bfloat16 and
                 qd == d and q.is_contiguous() and q.get_device() == k_cache.get_device())
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        num_pages, P, Hkv, d, B, mp = _paged_inputs(k_cache, v_cache, page_table, seqlens_k, q_offsets, "q_offsets")
        _need(q, "q", torch.bfloat16, 3)
        total, Hq, _ = q.shape
        _need(q, "q", torch.bfloat16, (total, Hq, d))
    if tree_mask is not None:
        mask_type = torch.uint64 if isinstance(tree_mask, torch.Tensor) and tree_mask.dtype is torch.uint64 else torch.int64
        _need(tree_mask, "tree_mask", mask_type, (total,))
    if o is not None:
        _need(o, "o", torch.bfloat16, q.shape)
    if lse is not None:
        _need(lse, "lse", torch.float32, (total, Hq))
    if not usual or not _same_device(k_cache.get_device(), tree_mask, o, lse):
        _device(q=q, k_cache=k_cache, v_cache=v_cache, page_table=page_table, seqlens_k=seqlens_k,
                q_offsets=q_offsets, tree_mask=tree_mask, o=o, lse=lse)
    dev = k_cache.device
    max_q = int(max_q)
    scale = d ** -0.5 if scale is None else float(scale)
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((total, Hq), dtype=torch.float32, device=dev) if lse is None else lse
    if stream is not None:  # new memory belongs to the current stream
        o.record_stream(stream)
        lse.record_stream(stream)
    ev = 0
    if events is not None:
        _, _keep = _events(events)
        ev = ctypes.addressof(_keep)
    args = (q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), seqlens_k.data_ptr(),
            q_offsets.data_ptr(), _adr(tree_mask), B, Hq, Hkv, d, P, num_pages, mp, total, max_q, scale, o.data_ptr(),
            lse.data_ptr(), ev)
    need = _tree_workspaces.get((dev, Hq, Hkv, d, max_q))
    if need is None:
        with torch.cuda.device(dev):  # the size depends on the device's number of SMs
            need = _entry("jfa_decode_tree_workspace_size")(ctypes.byref(_abi.DecodeTreeArgs(*args)))
        _tree_workspaces[dev, Hq, Hkv, d, max_q] = need
    _run_packed("jfa_decode_tree", _abi.pack_decode_tree(*args), need, dev.index, workspace, stream, check)
    return o, lse


def jfa_cache_accept(k_cache, v_cache, page_table, seqlens_k, q_offsets, accepted, counts, new_seqlens=None,
                     workspace=None, stream=None, check=False):
    """Keeps the accepted ones of each sequence's new tokens in a bf16 paged cache: the K and V rows of new
    tokens accepted[b][k], k < counts[b] (int32 [B, width <= 64] and [B]; 0 .. n_b - 1, n_b = q_offsets[b+1] -
    q_offsets[b]), move to the places behind the tokens before the new ones, in that order. Returns
    new_seqlens int32 [B] = seqlens_k - n_b + counts."""
    try:
        num_pages, P, Hkv, d = k_cache.shape
        B, mp = page_table.shape
        usual = _paged_ok(k_cache, v_cache, page_table, seqlens_k, q_offsets, B)
    except (AttributeError, TypeError, ValueError):
        usual = False
    if not usual:
        num_pages, P, Hkv, d, B, mp = _paged_inputs(k_cache, v_cache, page_table, seqlens_k, q_offsets, "q_offsets")
    width = accepted.shape[1] if isinstance(accepted, torch.Tensor) and accepted.dim() == 2 else 0
    _need(accepted, "accepted", torch.int32, (B, width))
    _need(counts, "counts", torch.int32, (B,))
    if new_seqlens is not None:
        _need(new_seqlens, "new_seqlens", torch.int32, (B,))
    if not usual or not _same_device(k_cache.get_device(), accepted, counts, new_seqlens):
        _device(k_cache=k_cache, v_cache=v_cache, page_table=page_table, seqlens_k=seqlens_k, q_offsets=q_offsets,
                accepted=accepted, counts=counts, new_seqlens=new_seqlens)
    dev = k_cache.device
    if new_seqlens is None:
        new_seqlens = torch.empty_like(seqlens_k)
        if stream is not None:  # new memory belongs to the current stream
            new_seqlens.record_stream(stream)
    packed = _abi.pack_cache_accept(k_cache.data_ptr(), v_cache.data_ptr(), page_table.data_ptr(), seqlens_k.data_ptr(),
                                    q_offsets.data_ptr(), accepted.data_ptr(), counts.data_ptr(), B, Hkv, d, P,
                                    num_pages, mp, width, new_seqlens.data_ptr())
    _run_packed("jfa_cache_accept", packed, 256, dev.index, workspace, stream, check)
    return new_seqlens


# ---------------------------------------------------------------- autograd

class _JaggedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, offsets, max_seqlen, scale, causal):
        o, lse = jfa_fwd(q, k, v, offsets, max_seqlen, scale, causal)
        ctx.save_for_backward(q, k, v, o, lse, offsets)
        ctx.max_seqlen, ctx.scale, ctx.causal = max_seqlen, scale, causal
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, offsets = ctx.saved_tensors
        dq, dk, dv = jfa_bwd(q, k, v, o, do.contiguous(), lse, offsets, ctx.max_seqlen, ctx.scale, ctx.causal)
        return dq, dk, dv, None, None, None, None


def jagged_attention(q, k, v, offsets, max_seqlen, scale=None, causal=False):
    """Differentiable jagged attention (bf16 [total, H, d] tensors, int32 offsets)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _JaggedAttention.apply(q, k, v, offsets, max_seqlen, scale, causal)


class _VarlenAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale, causal):
        o, lse = jfa_fwd_varlen(q, k, v, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale, causal)
        ctx.save_for_backward(q, k, v, o, lse, q_offsets, k_offsets)
        ctx.args = (max_seqlen_q, max_seqlen_k, scale, causal)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, q_offsets, k_offsets = ctx.saved_tensors
        mq, mk, scale, causal = ctx.args
        dq, dk, dv = jfa_bwd_varlen(q, k, v, o, do.contiguous(), lse, q_offsets, k_offsets, mq, mk, scale, causal)
        return dq, dk, dv, None, None, None, None, None, None


def varlen_attention(q, k, v, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale=None, causal=False):
    """Differentiable varlen / GQA attention (see jfa_fwd_varlen for layouts and the causal alignment)."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    return _VarlenAttention.apply(q, k, v, q_offsets, k_offsets, max_seqlen_q, max_seqlen_k, scale, causal)
