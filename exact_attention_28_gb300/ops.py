"""ctypes binding of libfa_gb300.so: the C entry points under the same names.

Argument marshalling only -- every step of the computation runs in the CUDA
library.  There is no fallback: a missing library or a failing call raises.
"""
from __future__ import annotations

import array
import ctypes
import math
import os
import struct
import threading
import weakref

import torch

from .build import LIB_PATH

(FA_OK, FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED, FA_ERR_MISALIGNED, FA_ERR_CUDA, FA_ERR_TIMEOUT,
 FA_ERR_TOO_LARGE) = range(7)

_lib = None


class FAError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def load_library(path: str | None = None):
    """Load the compiled library (build it first with __graft_entry__.build())."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise FileNotFoundError(
            f"{path} is missing: the CUDA library has not been built (run __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.fa_fwd.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd.restype = i
    lib.fa_fwd_host.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_host.restype = i
    lib.fa_host_groups.argtypes = [i, i, i, i, i, i]
    lib.fa_host_groups.restype = i
    lib.fa_fwd_test_missing_load.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_test_missing_load.restype = i
    lib.fa_fwd_splitkv.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, ctypes.c_size_t, vp]
    lib.fa_fwd_splitkv.restype = i
    lib.fa_fwd_splitkv_noalloc.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp]
    lib.fa_fwd_splitkv_noalloc.restype = i
    lib.fa_splitkv_workspace.argtypes = [i, i, i, i, i, i, vp, vp]
    lib.fa_splitkv_workspace.restype = i
    lib.fa_fwd_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_paged.restype = i
    lib.fa_fwd_paged_splitkv.argtypes = [vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, f, i, i, vp,
                                         ctypes.c_size_t, vp]
    lib.fa_fwd_paged_splitkv.restype = i
    lib.fa_quantize_fp8.argtypes = [vp, vp, vp, i, i, i, i, vp, i, vp]
    lib.fa_quantize_fp8.restype = i
    lib.fa_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp]
    lib.fa_fwd_fp8.restype = i
    lib.fa_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, vp, ctypes.c_size_t, vp]
    lib.fa_bwd.restype = i
    lib.fa_bwd_workspace.argtypes = [i, i, i, i, i, vp]
    lib.fa_bwd_workspace.restype = i
    z = ctypes.c_size_t
    i64 = ctypes.c_int64
    lib.fa_block_tables.argtypes = [vp] * 9 + [i] * 5 + [vp]
    lib.fa_block_tables.restype = i
    lib.fa_rope.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, i, vp, i64, i64, i, i, i, i, i, vp, vp, i, i, vp]
    lib.fa_rope.restype = i
    lib.fa_paged_append.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, i, vp, vp, i, vp, vp, vp, vp, i64, i, i, i, i,
                                    i, i, vp, vp, i, vp]
    lib.fa_paged_append.restype = i
    lib.fa_decode_paged.argtypes = [vp, vp, vp, vp, i, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, i, i, i, f, i, vp,
                                    z, vp]
    lib.fa_decode_paged.restype = i
    lib.fa_decode_paged_workspace.argtypes = [i, i, i, i, i, vp]
    lib.fa_decode_paged_workspace.restype = i
    lib.fa_check_device_status.argtypes = [vp]
    lib.fa_check_device_status.restype = i
    lib.fa_schedule.argtypes = [i, i, i, i, i, i, i, i, vp, ctypes.c_int64, vp]
    lib.fa_schedule.restype = i
    lib.fa_status_string.argtypes = [i]
    lib.fa_status_string.restype = ctypes.c_char_p
    if path == LIB_PATH:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().fa_status_string(status).decode()


def _check(status: int):
    if status != FA_OK:
        raise FAError(status, status_string(status))


def _stream_handle(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(getattr(stream, "cuda_stream", stream))


def _shape(q, k):
    B, H, Nq, d = q.shape
    Nk = k.shape[2]
    return B, H, Nq, Nk, d


def fa_fwd(q, k, v, o=None, lse=None, scale=None, causal=False, stream=None):
    """O, LSE = attention(q, k, v) on the GPU through the C ABI.

    q: bf16 [B,H,Nq,d], k/v: bf16 [B,H,Nk,d], contiguous CUDA tensors.
    Returns (o, lse); o bf16 [B,H,Nq,d], lse fp32 [B,H,Nq].
    """
    for t in (q, k, v):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise TypeError("q, k, v must be contiguous bf16 CUDA tensors")
    B, H, Nq, Nk, d = _shape(q, k)
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load_library().fa_fwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(stream)))
    return o, lse


def fa_fwd_host(hq, hk, hv, ho, hlse, dq, dk, dv, do, dlse, scale, causal=False, stream=None):
    """End-to-end call from (pinned) host tensors through caller-owned device buffers."""
    B, H, Nq, Nk, d = _shape(hq, hk)
    _check(load_library().fa_fwd_host(hq.data_ptr(), hk.data_ptr(), hv.data_ptr(), ho.data_ptr(),
                                      hlse.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                                      do.data_ptr(), dlse.data_ptr(), B, H, Nq, Nk, d, scale,
                                      int(bool(causal)), _stream_handle(stream)))


def fa_fwd_test_missing_load(q, k, v, item=0, scale=None, causal=False, stream=None):
    """fa_fwd with the first K tile of work item `item` never loaded (tests the
    bounded waits); returns the launch status, and the device status word then
    reads FA_ERR_TIMEOUT."""
    B, H, Nq, Nk, d = _shape(q, k)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return int(load_library().fa_fwd_test_missing_load(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                        lse.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)),
                                                        item, _stream_handle(stream)))


def host_groups(B, H, Nq, Nk, d, num_sms):
    """Number of head groups fa_fwd_host pipelines for these shapes (1: none)."""
    return int(load_library().fa_host_groups(B, H, Nq, Nk, d, num_sms))


def fa_fwd_paged(q, k_cache, v_cache, block_table, seq_lens, o=None, lse=None, scale=None, causal=False,
                 stream=None, num_splits=None, workspace=None):
    """Attention over a paged cache: k_cache, v_cache [num_blocks, H, block_size, d] bf16,
    block_table int32 [B, max_blocks], seq_lens int32 [B] (all CUDA tensors).

    num_splits: None runs fa_fwd_paged; an int (0 = the library's choice)
    runs fa_fwd_paged_splitkv with that many key slices, allocating the
    workspace unless one is given."""
    B, H, Nq, d = q.shape
    num_blocks, Hc, block_size, dc = k_cache.shape
    if Hc != H or dc != d or v_cache.shape != k_cache.shape:
        raise ValueError("cache shape mismatch")
    if block_table.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise TypeError("block_table and seq_lens must be int32")
    max_blocks = block_table.shape[1]
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if num_splits is None:
        _check(load_library().fa_fwd_paged(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                           block_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                           B, H, Nq, max_blocks, num_blocks, block_size, d, scale,
                                           int(bool(causal)), _stream_handle(stream)))
        return o, lse
    splits, nbytes = splitkv_workspace(B, H, Nq, max_blocks * block_size, d, causal, num_splits)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(load_library().fa_fwd_paged_splitkv(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                               block_table.data_ptr(), seq_lens.data_ptr(), o.data_ptr(),
                                               lse.data_ptr(), B, H, Nq, max_blocks, num_blocks, block_size, d,
                                               scale, int(bool(causal)), splits, workspace.data_ptr(),
                                               workspace.numel() * workspace.element_size(), _stream_handle(stream)))
    return o, lse


def quantize_fp8(x, signs=None, transpose=False, stream=None):
    """E4M3 codes (torch.uint8) and per-head descale (fp32 [B, H]) of a bf16
    [B, H, N, d] CUDA tensor; `signs` (fp32 [d] of +-1, CUDA) rotates rows by
    diag(signs) H / sqrt(d); transpose gives [B, H, d, ceil16(N)]."""
    if not (x.is_cuda and x.dtype == torch.bfloat16 and x.is_contiguous()):
        raise TypeError("x must be a contiguous bf16 CUDA tensor")
    B, H, N, d = x.shape
    if transpose:
        x8 = torch.empty((B, H, d, -(-N // 16) * 16), dtype=torch.uint8, device=x.device)
    else:
        x8 = torch.empty((B, H, N, d), dtype=torch.uint8, device=x.device)
    descale = torch.empty((B, H), dtype=torch.float32, device=x.device)
    _check(load_library().fa_quantize_fp8(x.data_ptr(), x8.data_ptr(), descale.data_ptr(), B, H, N, d,
                                          None if signs is None else signs.data_ptr(), int(bool(transpose)),
                                          _stream_handle(stream)))
    return x8, descale


def fa_fwd_fp8(q8, k8, vt8, descale_q, descale_k, descale_v, o=None, lse=None, scale=None, causal=False,
               stream=None):
    """Attention on E4M3 codes: q8 [B,H,Nq,d], k8 [B,H,Nk,d], vt8 [B,H,d,ceil16(Nk)]
    (torch.uint8 CUDA tensors) with per-head descales; returns bf16 O and fp32 LSE."""
    B, H, Nq, d = q8.shape
    Nk = k8.shape[2]
    if k8.shape != (B, H, Nk, d) or vt8.shape != (B, H, d, -(-Nk // 16) * 16):
        raise ValueError("shape mismatch")
    if o is None:
        o = torch.empty((B, H, Nq, d), dtype=torch.bfloat16, device=q8.device)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q8.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load_library().fa_fwd_fp8(q8.data_ptr(), k8.data_ptr(), vt8.data_ptr(), descale_q.data_ptr(),
                                     descale_k.data_ptr(), descale_v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                     B, H, Nq, Nk, d, scale, int(bool(causal)), _stream_handle(stream)))
    return o, lse


def fa_bwd(q, k, v, o, lse, do, dq=None, dk=None, dv=None, scale=None, causal=False, workspace=None,
           stream=None):
    """dQ, dK, dV of the attention forward (o, lse from fa_fwd) for upstream gradient do."""
    B, H, Nq, Nk, d = _shape(q, k)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    nb = ctypes.c_size_t(0)
    _check(load_library().fa_bwd_workspace(B, H, Nq, Nk, d, ctypes.byref(nb)))
    if workspace is None:
        workspace = torch.empty(nb.value, dtype=torch.uint8, device=q.device)
    _check(load_library().fa_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                 do.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, Nq, Nk, d,
                                 scale, int(bool(causal)), workspace.data_ptr(), workspace.numel(),
                                 _stream_handle(stream)))
    return dq, dk, dv


class _Attention(torch.autograd.Function):
    """Autograd wrapper: forward through fa_fwd (saving O and LSE), backward
    through fa_bwd.  Marshalling only; both directions run in the library."""

    @staticmethod
    def forward(ctx, q, k, v, scale, causal):
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        o, lse = fa_fwd(q, k, v, scale=scale, causal=causal)
        ctx.save_for_backward(q, k, v, o, lse)
        ctx.scale, ctx.causal = scale, causal
        ctx.mark_non_differentiable(lse)
        return o, lse

    @staticmethod
    def backward(ctx, do, _dlse):
        q, k, v, o, lse = ctx.saved_tensors
        dq, dk, dv = fa_bwd(q, k, v, o, lse, do.contiguous(), scale=ctx.scale, causal=ctx.causal)
        return dq, dk, dv, None, None


def flash_attention(q, k, v, causal=False, scale=None, return_lse=False):
    """softmax(scale * q k^T) v for bf16 CUDA tensors [B, H, N, d] (d = 64 or
    128), differentiable with respect to q, k and v.  scale defaults to
    1/sqrt(d); causal applies the top-left mask (key j visible to query i iff
    j <= i).  Returns O, or (O, LSE) with return_lse."""
    if scale is None:
        scale = 1.0 / math.sqrt(q.shape[-1])
    o, lse = _Attention.apply(q, k, v, float(scale), bool(causal))
    return (o, lse) if return_lse else o


# ---------------------------------------------------- serving, rotary positions

class Rotary:
    """Frequencies and axes of a rotary embedding, laid out once for fa_rope,
    fa_paged_append and apply_rotary.

    d: head dimension (64 or 128); rot: how many leading elements turn (a
    multiple of 16, default d); base: pair c turns by base^(-2c/rot) radians
    per position, unless inv_freq gives the rot/2 frequencies; sections: pairs
    that follow each axis, in order (they add up to rot/2; default one axis),
    or pair_axis: the axis of every pair, one by one; interleaved: pairs are
    elements (2c, 2c+1) instead of (c, c + rot/2).
    """

    def __init__(self, d, base=10000.0, rot=None, sections=None, interleaved=False, inv_freq=None, pair_axis=None):
        rot = d if rot is None else rot
        if d not in (64, 128) or rot % 16 or not 16 <= rot <= d:
            raise ValueError("d must be 64 or 128 and rot a multiple of 16 from 16 to d")
        pairs = rot // 2
        if inv_freq is None:
            inv_freq = [base ** (-2.0 * c / rot) for c in range(pairs)]
        if sections is not None and pair_axis is not None:
            raise ValueError("sections and pair_axis say the same thing: give one of them")
        if pair_axis is None:
            pair_axis = []
            for a, n in enumerate((pairs,) if sections is None else sections):
                pair_axis += [a] * n
        inv_freq, pair_axis = array.array("d", inv_freq), array.array("i", pair_axis)
        if len(inv_freq) != pairs or len(pair_axis) != pairs:
            raise ValueError(f"{pairs} frequencies and {pairs} pairs in the sections are needed")
        if not all(map(math.isfinite, inv_freq)):
            raise ValueError("the frequencies must be finite")
        axes = max(max(pair_axis) + 1, len(sections) if sections is not None else 1)
        if min(pair_axis) < 0 or axes > 4:
            raise ValueError("axes are 0 to 3")
        self.d, self.rot, self.axes, self.interleaved = d, rot, axes, bool(interleaved)
        self.inv_freq, self.pair_axis = tuple(inv_freq), tuple(pair_axis)
        self._freq = (ctypes.c_double * pairs).from_buffer(inv_freq)
        self._axis = (ctypes.c_int * pairs).from_buffer(pair_axis)


# what torch.cuda.current_device() and current_stream(dev).cuda_stream come to, without the objects in between
# (0.1 us instead of 0.3 and 2.9 on a Grace core); a tensor on the device exists by then, so CUDA is set up
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_PACK_STRIDES = {n: struct.Struct(f"{n}q").pack for n in (2, 3)}   # int64 arrays for the C side


def _refuse(name, t, dtype, dev, shape, what="a contiguous"):
    kind = str(dtype).removeprefix("torch.")
    if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype):
        raise TypeError(f"{name} must be {what} {kind} CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"tensors on different devices: {name} on {t.device}, others on cuda:{dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"shape mismatch: {name} {tuple(t.shape)}, expected {tuple(shape)}")
    raise TypeError(f"{name} must be {what} {kind} CUDA tensor")


def _device_of(name, t):
    """Index of the CUDA device of a tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _whole(name, t, dtype, dev, shape=None):
    """Address of a contiguous tensor of this type and device (and shape)."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, dev, shape)


def _flat(name, t, dtype, dev, n):
    """Address of a contiguous tensor of n elements."""
    try:
        if t.dtype is dtype and t.numel() == n and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(name, t, dtype, dev, (n,))


def _strided(name, t, dev, shape=None):
    """(address, strides of every dimension but the last; None: contiguous) of a bf16 tensor whose last
    dimension is contiguous."""
    try:
        if t.dtype is _BF16 and t.get_device() == dev and (shape is None or t.shape == shape):
            if t.is_contiguous():
                return t.data_ptr(), None
            st = t.stride()
            if st[-1] == 1:
                return t.data_ptr(), _PACK_STRIDES[len(st) - 1](*st[:-1])
    except AttributeError:
        pass
    _refuse(name, t, _BF16, dev, shape, "with a contiguous last dimension a")


def _call(dev, stream, fn, *args):
    """fn(*args, stream) with device `dev` current; stream None: the current one of that device."""
    if dev != _current_device():
        with torch.cuda.device(dev):
            return _call(dev, stream, fn, *args)
    status = fn(*args, _raw_stream(dev) if stream is None else int(getattr(stream, "cuda_stream", stream)))
    if status != FA_OK:
        _check(status)


def _new(shape, dtype, dev, stream, fill=None):
    """A tensor of the allocator's pool of the stream that uses it (and cleared on it)."""
    make = torch.empty if fill is None else torch.zeros
    if stream is None:
        return make(shape, dtype=dtype, device=dev)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=dev)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=dev)


def fa_block_tables(block_table, ctx_lens, new_lens, free_blocks, block_size, num_tokens, seq_lens=None,
                    query_start=None, slots=None, positions=None, counts=None, stream=None):
    """Block table, slots and positions of a step from the requests' lengths.

    block_table int32 [B, max_blocks] is updated in place; ctx_lens, new_lens
    int32 [B]; free_blocks int32 [num_free], or None (all contiguous CUDA tensors).
    num_tokens is the room for new tokens; those behind the last one get slot
    -1 and position 0.  Returns (seq_lens [B], query_start [B+1], slots
    [num_tokens], positions [num_tokens], counts [2]: tokens, blocks needed)."""
    dev = _device_of("block_table", block_table)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_blocks]")
    B, max_blocks = block_table.shape
    num_free = 0 if free_blocks is None else free_blocks.numel()
    if seq_lens is None:
        seq_lens = _new(B, _I32, dev, stream)
    if query_start is None:
        query_start = _new(B + 1, _I32, dev, stream)
    if slots is None:
        slots = _new(num_tokens, _I32, dev, stream)
    if positions is None:
        positions = _new(num_tokens, _I32, dev, stream)
    if counts is None:
        counts = _new(2, _I32, dev, stream)
    _call(dev, stream, (_lib or load_library()).fa_block_tables, _whole("block_table", block_table, _I32, dev),
          _flat("ctx_lens", ctx_lens, _I32, dev, B), _flat("new_lens", new_lens, _I32, dev, B),
          None if free_blocks is None else _flat("free_blocks", free_blocks, _I32, dev, num_free),
          _flat("seq_lens", seq_lens, _I32, dev, B), _flat("query_start", query_start, _I32, dev, B + 1),
          _flat("slots", slots, _I32, dev, num_tokens), _flat("positions", positions, _I32, dev, num_tokens),
          _flat("counts", counts, _I32, dev, 2), B, max_blocks, block_size, num_free, num_tokens)
    return seq_lens, query_start, slots, positions, counts


def _rope_positions(positions, dev, axes, lead):
    """(address, axis stride, batch stride) of int32 positions [axes, *lead] (the axis may be left out when
    there is one; [axes, N] is shared by the batches of lead = (B, N))."""
    if not isinstance(positions, torch.Tensor) or positions.dtype is not _I32 or positions.get_device() != dev:
        _refuse("positions", positions, _I32, dev, None)
    shape, st = positions.shape, positions.stride()
    if not st or (st[-1] != 1 and shape[-1] > 1):
        raise TypeError("positions must be contiguous in its last dimension")
    full = len(lead) + 1
    if len(st) == full and shape == (axes, *lead):
        return positions.data_ptr(), st[0], st[1] if full == 3 else 0
    if axes == 1 and shape == lead:
        return positions.data_ptr(), 0, st[0] if full == 3 else 0
    if full == 3 and shape == (axes, lead[1]):
        return positions.data_ptr(), st[0], 0
    if full == 3 and axes == 1 and shape == lead[1:]:
        return positions.data_ptr(), 0, 0
    raise ValueError(f"positions {tuple(shape)} do not fit {axes} axes of {lead}")


def fa_rope(q, k, positions, rotary, q_out=None, k_out=None, inverse=False, stream=None):
    """q and k (None: q alone) turned by their positions: bf16 [B, H, N, d], any strides whose last is 1.

    positions int32 [axes, B, N] or [axes, N] (the axis may be left out when there is one); rotary: a
    Rotary.  inverse turns back (the gradient).  q_out, k_out may be q, k
    themselves.  Without tokens (B or N is 0) nothing is launched.  Returns
    (q_out, k_out)."""
    dev = _device_of("q", q)
    B, Hq, N, d = q.shape
    if d != rotary.d:
        raise ValueError(f"head dimension {d}, rotary made for {rotary.d}")
    if q_out is None:
        q_out = _new((B, Hq, N, d), _BF16, dev, stream)
    qp, qs = _strided("q", q, dev)
    qop, qos = _strided("q_out", q_out, dev, q.shape)
    kp = kop = ks = kos = None
    Hk = 0
    if k is not None:
        Hk = k.shape[1]
        if k_out is None:
            k_out = _new((B, Hk, N, d), _BF16, dev, stream)
        kp, ks = _strided("k", k, dev, (B, Hk, N, d))
        kop, kos = _strided("k_out", k_out, dev, (B, Hk, N, d))
    elif k_out is not None:
        raise ValueError("k_out without k")
    pos, axis_stride, batch_stride = _rope_positions(positions, dev, rotary.axes, (B, N))
    if B == 0 or N == 0:
        return q_out, k_out
    _call(dev, stream, (_lib or load_library()).fa_rope, qp, qs, qop, qos, Hq, kp, ks, kop, kos, Hk, pos, axis_stride,
          batch_stride, B, N, d, rotary.rot, rotary.axes, rotary._freq, rotary._axis, rotary.interleaved, bool(inverse))
    return q_out, k_out


class _Trail:
    """Where the graph of one rotation begins: its device, its stream, and the edges to what its inputs came from."""
    __slots__ = ("dev", "stream", "edges", "mixed", "__weakref__")


# The trails of the rotations whose graphs are alive: {device: {stream: WeakSet}}.
#
# The gradient node of a leaf keeps the stream of the graph that made it for as
# long as any graph of the leaf lives.  A captured backward that reaches a node
# of another stream makes that stream wait inside the capture, which ends the
# process.  A node does not tell its stream, so a captured backward looks for
# the living rotations of other streams that come from the same leaves, through
# views, projections and whatever else lies between, and refuses.  That search
# walks whole graphs, so it is left to captures: an eager call leaves its trail,
# and its stream on the node of an input that is a leaf itself (where a graph of
# another function may keep it longer than this one lives).
_trails, _trails_lock = {}, threading.Lock()


def _leaves_behind(edges):
    """The gradient nodes of all leaves that a function's inputs came from."""
    seen, leaves, todo = set(), set(), [node for node, _ in edges if node is not None]
    while todo:
        node = todo.pop()
        if node in seen:
            continue
        seen.add(node)
        if type(node).__name__ == "AccumulateGrad":
            leaves.add(node)
        else:
            todo.extend(n for n, _ in node.next_functions if n is not None)
    return leaves


def _living(trail, apart):
    """The other living trails on this device whose leaves' nodes may belong to another stream than `apart`."""
    with _trails_lock:
        return [t for stream, live in _trails.get(trail.dev, {}).items() for t in live
                if t is not trail and (stream != apart or t.mixed)]


def _leave_trail(edges, dev):
    """The trail of a rotation on the current stream.  `mixed`: nodes of its leaves may be another stream's all the
    same, made by a rotation that was alive then."""
    trail = _Trail()
    stream = _raw_stream(dev)
    trail.dev, trail.stream, trail.edges = dev, stream, edges
    for node, _ in edges:
        if type(node).__name__ == "AccumulateGrad":
            node.metadata.setdefault("fa_stream", stream)
    with _trails_lock:
        streams = _trails.setdefault(dev, {})
        if stream not in streams:
            streams[stream] = weakref.WeakSet()
        trail.mixed = len(streams) > 1 and any(live for s, live in streams.items() if s != stream)
        streams[stream].add(trail)
    if trail.mixed and torch.cuda.is_current_stream_capturing():
        trail.mixed = _meets(trail)
    return trail


def _meets(trail):
    """Whether a leaf behind this trail may have a node of another stream than the trail's."""
    leaves = _leaves_behind(trail.edges)
    return (any(node.metadata.get("fa_stream", trail.stream) != trail.stream for node in leaves) or
            any(not leaves.isdisjoint(_leaves_behind(t.edges)) for t in _living(trail, trail.stream)))


class _Rotation(torch.autograd.Function):
    """The rotation of q and k; its gradient is the rotation by the negative angles."""

    @staticmethod
    def forward(ctx, q, k, positions, rotary, inverse):
        ctx.save_for_backward(positions)
        ctx.rotary, ctx.inverse = rotary, inverse
        q_out, k_out = fa_rope(_rows(q), None if k is None else _rows(k), positions, rotary, inverse=inverse)
        edges = ctx.next_functions
        if edges:
            ctx.trail = _leave_trail(edges, positions.get_device())
        return q_out if k is None else (q_out, k_out)

    @staticmethod
    def backward(ctx, gq, gk=None):
        positions, = ctx.saved_tensors
        if torch.cuda.is_current_stream_capturing() and _meets(ctx.trail):
            raise RuntimeError("apply_rotary: this backward is being captured while a graph of the same leaf, "
                               "made on another stream, is alive; drop that graph (its outputs) first")
        if torch.is_grad_enabled():     # a graph of the backward itself is asked for
            out = _Rotation.apply(gq, gk, positions, ctx.rotary, not ctx.inverse)
            gq, gk = (out, None) if gk is None else out
        else:
            gq, gk = fa_rope(_rows(gq), None if gk is None else _rows(gk), positions, ctx.rotary,
                             inverse=not ctx.inverse)
        return gq, gk, None, None, None


def _rows(t):
    """t itself where its rows start on 16-byte boundaries, else a contiguous copy."""
    if t.data_ptr() % 16 == 0:
        if t.is_contiguous():
            return t
        st = t.stride()
        if st[-1] == 1 and all(s % 8 == 0 or n == 1 for s, n in zip(st[:-1], t.shape)):
            return t
    return t.clone(memory_format=torch.contiguous_format)


def apply_rotary(q, k, positions, rotary):
    """fa_rope as a function differentiable with respect to q and k (bf16 CUDA tensors [B, H, N, d] of any
    strides; k may be None): what goes in front of flash_attention.  Returns (q, k) turned, or q alone
    when k is None.  Differentiable any number of times.

    Capturing its backward into a CUDA graph takes what PyTorch asks of any
    captured backward: warm up on the capture's stream, and let no eager graph
    of the same leaves live on another one.  A captured backward of a rotation
    raises RuntimeError where a living rotation of another stream comes from a
    leaf that its q or k comes from too, be q and k that leaf, views of it or
    results of it.  Graphs that went through no rotation are not seen."""
    return _Rotation.apply(q, k, positions, rotary, False)


def _cache(k_cache, v_cache, k_descale, v_descale, d, dev):
    """(k and v addresses, 0 (bf16) or 1 (E4M3 codes, torch.uint8), descale addresses, num_blocks, Hkv, block_size)
    of a paged cache [num_blocks, Hkv, block_size, d]."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise TypeError("the cache must be CUDA tensors [num_blocks, Hkv, block_size, d]")
    dtype, shape = k_cache.dtype, k_cache.shape
    if dtype is not _BF16 and dtype is not _U8:
        raise TypeError("the cache must be bfloat16 or uint8 (E4M3 codes)")
    num_blocks, Hkv, block_size, width = shape
    kp, vp = _flat("k_cache", k_cache, dtype, dev, k_cache.numel()), _whole("v_cache", v_cache, dtype, dev, shape)
    if width != d:
        raise ValueError(f"cache shape mismatch: {tuple(shape)} for head dimension {d}")
    if dtype is _BF16:
        if k_descale is not None or v_descale is not None:
            raise ValueError("k_descale and v_descale belong to an E4M3 cache")
        return kp, vp, 0, None, None, num_blocks, Hkv, block_size
    return (kp, vp, 1, _flat("k_descale", k_descale, _F32, dev, Hkv),
            _flat("v_descale", v_descale, _F32, dev, Hkv), num_blocks, Hkv, block_size)


def fa_paged_append(q, k, v, k_cache, v_cache, slots, positions=None, rotary=None, q_out=None, k_descale=None,
                    v_descale=None, stream=None):
    """Writes new tokens into the paged cache: k (turned by `rotary` at
    `positions`, if given) and v at their slots, and q, turned, to q_out.

    q bf16 [T, Hq, d] or None; k, v bf16 [T, Hkv, d] (any strides whose last
    is 1: views of one projection's output); caches [num_blocks, Hkv, block_size,
    d], bf16 or E4M3 codes (uint8) with k_descale, v_descale fp32 [Hkv];
    slots int32 [T], negative: the token is skipped and its q_out row left as
    it was; positions int32 [axes, T] or [T].  Without tokens (T = 0) nothing is
    launched.  Returns q_out (None without q)."""
    dev = _device_of("k", k)
    T, Hkv, d = k.shape
    kp, ks = _strided("k", k, dev)
    vp, vs = _strided("v", v, dev, k.shape)
    kcp, vcp, kind, kdp, vdp, num_blocks, heads, block_size = _cache(k_cache, v_cache, k_descale, v_descale, d, dev)
    if heads != Hkv:
        raise ValueError(f"cache shape mismatch: {heads} heads in the cache, {Hkv} in k")
    Hq, qp, qop, qs, qos = 0, None, None, None, None
    if q is not None:
        Hq = q.shape[1]
        if q_out is None:
            q_out = _new((T, Hq, d), _BF16, dev, stream, fill=0)   # skipped tokens read as 0
        qp, qs = _strided("q", q, dev, (T, Hq, d))
        qop, qos = _strided("q_out", q_out, dev, q.shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rot, axes, freq, axis, interleaved, pos, axis_stride = 0, 0, None, None, False, None, 0
    if rotary is not None:
        if positions is None or rotary.d != d:
            raise ValueError("rotary needs positions, and the head dimension it was made for")
        rot, axes, freq, axis, interleaved = rotary.rot, rotary.axes, rotary._freq, rotary._axis, rotary.interleaved
        pos, axis_stride, _ = _rope_positions(positions, dev, axes, (T,))
    slots_p = _flat("slots", slots, _I32, dev, T)
    if T == 0:
        return q_out
    _call(dev, stream, (_lib or load_library()).fa_paged_append, qp, qs, qop, qos, Hq, kp, ks, vp, vs, Hkv, kcp, vcp,
          kind, kdp, vdp, slots_p, pos, axis_stride, T, num_blocks, block_size, d, rot,
          axes, freq, axis, interleaved)
    return q_out


def decode_paged_workspace(B, Hq, Hkv, Nq, d):
    """Workspace bytes of fa_decode_paged, whatever the lengths."""
    nb = ctypes.c_size_t(0)
    _check(load_library().fa_decode_paged_workspace(B, Hq, Hkv, Nq, d, ctypes.byref(nb)))
    return nb.value


def fa_decode_paged(q, k_cache, v_cache, block_table, seq_lens, o=None, lse=None, scale=None, causal=False,
                    k_descale=None, v_descale=None, workspace=None, stream=None):
    """Attention of the newest Nq (1 to 16) tokens of each sequence over a paged cache, query heads in groups.

    q bf16 [B, Hq, Nq, d], any strides whose last is 1; caches [num_blocks,
    Hkv, block_size, d] with Hkv dividing Hq, bf16 or E4M3 codes (uint8) with
    k_descale, v_descale fp32 [Hkv]; block_table int32 [B, max_blocks],
    seq_lens int32 [B].  o may be q itself.  `workspace`: a contiguous CUDA
    uint8 tensor of decode_paged_workspace bytes (allocated here if None).
    Without sequences (B = 0) nothing is launched.  Returns (o, lse)."""
    dev = _device_of("q", q)
    B, Hq, Nq, d = q.shape
    qp, qs = _strided("q", q, dev)
    kcp, vcp, kind, kdp, vdp, num_blocks, Hkv, block_size = _cache(k_cache, v_cache, k_descale, v_descale, d, dev)
    table = _whole("block_table", block_table, _I32, dev)
    if block_table.dim() != 2 or block_table.shape[0] != B:
        raise ValueError("block_table must be [B, max_blocks]")
    if o is None:
        o = _new((B, Hq, Nq, d), _BF16, dev, stream)
    if lse is None:
        lse = _new((B, Hq, Nq), _F32, dev, stream)
    op, os_ = _strided("o", o, dev, q.shape)
    lens, lsep = _flat("seq_lens", seq_lens, _I32, dev, B), _flat("lse", lse, _F32, dev, B * Hq * Nq)
    if B == 0:
        return o, lse
    if workspace is None:
        workspace = _new(decode_paged_workspace(B, Hq, Hkv, Nq, d), _U8, dev, stream)
    nbytes = workspace.numel()
    _call(dev, stream, (_lib or load_library()).fa_decode_paged, qp, qs, kcp, vcp, kind, kdp, vdp, table,
          lens, op, os_, lsep, B, Hq, Hkv, Nq, block_table.shape[1], num_blocks, block_size, d,
          1.0 / math.sqrt(d) if scale is None else scale, bool(causal),
          _flat("workspace", workspace, _U8, dev, nbytes), nbytes)
    return o, lse


def check_device_status(stream=None):
    """Synchronise and raise if a kernel of the library hit a wait limit."""
    _check(load_library().fa_check_device_status(_stream_handle(stream)))


def schedule(B, H, Nq, Nk, d, causal, num_sms, num_splits=1):
    """The kernel's work list: int32 array [n_items, 8] of (cta, round,
    batch*head, first query row, first KV tile, end KV tile of query tile 0,
    of query tile 1 (-1 if absent), key slice)."""
    import numpy as np
    lib = load_library()
    n = ctypes.c_int64(0)
    args = (B, H, Nq, Nk, d, int(bool(causal)), num_sms, num_splits)
    _check(lib.fa_schedule(*args, None, 0, ctypes.byref(n)))
    out = np.zeros((n.value, 8), dtype=np.int32)
    _check(lib.fa_schedule(*args, out.ctypes.data, n.value, ctypes.byref(n)))
    return out


def splitkv_workspace(B, H, Nq, Nk, d, causal=False, num_splits=0):
    """(num_splits, workspace bytes) for fa_fwd_splitkv; num_splits=0 lets the library choose."""
    ns = ctypes.c_int(num_splits)
    nb = ctypes.c_size_t(0)
    _check(load_library().fa_splitkv_workspace(B, H, Nq, Nk, d, int(bool(causal)), ctypes.byref(ns), ctypes.byref(nb)))
    return ns.value, nb.value


def fa_fwd_splitkv(q, k, v, o=None, lse=None, scale=None, causal=False, num_splits=0, workspace=None,
                   stream=None):
    """Split-key attention forward; `workspace` is a CUDA uint8 tensor (allocated here if None)."""
    B, H, Nq, Nk, d = _shape(q, k)
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    num_splits, nbytes = splitkv_workspace(B, H, Nq, Nk, d, causal, num_splits)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    _check(load_library().fa_fwd_splitkv(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(),
                                         B, H, Nq, Nk, d, scale, int(bool(causal)), num_splits,
                                         workspace.data_ptr(), workspace.numel(), _stream_handle(stream)))
    return o, lse


def fa_fwd_splitkv_noalloc(q, k, v, o, lse, scale=None, causal=False, num_splits=0, stream=None):
    """Split-key forward whose partials live in the library's fixed scratch area
    (no allocation anywhere on this call; o and lse are caller-provided:
    o bf16 like q, lse fp32 [B, H, Nq], both contiguous on q's device)."""
    for t in (q, k, v):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.bfloat16 and t.is_contiguous()):
            raise TypeError("q, k, v must be contiguous bf16 CUDA tensors")
    B, H, Nq, Nk, d = _shape(q, k)
    if k.shape != (B, H, Nk, d) or v.shape != (B, H, Nk, d):
        raise ValueError(f"shape mismatch: q {tuple(q.shape)} k {tuple(k.shape)} v {tuple(v.shape)}")
    if not (isinstance(o, torch.Tensor) and o.dtype == torch.bfloat16 and o.shape == q.shape
            and o.is_contiguous() and o.device == q.device):
        raise TypeError("o must be a contiguous bf16 tensor shaped like q on q's device")
    if not (isinstance(lse, torch.Tensor) and lse.dtype == torch.float32 and lse.shape == (B, H, Nq)
            and lse.is_contiguous() and lse.device == q.device):
        raise TypeError("lse must be a contiguous fp32 tensor [B, H, Nq] on q's device")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check(load_library().fa_fwd_splitkv_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                                 lse.data_ptr(), B, H, Nq, Nk, d, scale, int(bool(causal)),
                                                 num_splits, _stream_handle(stream)))
    return o, lse


def raw_fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale, causal, stream_handle=0) -> int:
    """The C call with raw integers; returns the status code (argument tests)."""
    return load_library().fa_fwd(q_ptr, k_ptr, v_ptr, o_ptr, lse_ptr, B, H, Nq, Nk, d, scale,
                                 int(causal), stream_handle)
