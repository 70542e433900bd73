"""Torch-facing wrappers of the serving operators: rotary positions, the paged key/value cache
and the attention over it (argument marshalling only, as ``api.py``).

A cache is a dict of CUDA tensors, made by ``new_cache`` or by the caller:
  k, v                [pages, kv_heads, page_size, head_dim] float16 or bfloat16 (bits = 16), or
                      [pages, kv_heads, page_size, head_dim * bits / 8] uint8 codes (bits = 8, 4)
  k_scales, v_scales  [pages, kv_heads, page_size] float32 (bits = 8, 4)
  k_zeros, v_zeros    [pages, kv_heads, page_size] uint8 (bits = 8, 4)
Slot s of the cache is row s % page_size of page s // page_size.  A value is
scale * (code - zero), the form of the library's quantized weights, one scale and zero point per
token, head and side.

The plain case of each call (outputs made here, the current stream) goes through the native front of
``csrc/binding.cpp``, which checks, allocates and launches; anything else, and everything that is wrong,
through the Python below, which says what.  So does every call where the front cannot be loaded (with a warning).
"""

from __future__ import annotations

import contextlib
import ctypes

import torch

from ._native import front, lib
from .api import _DTYPE, _check, _need, _need_cuda

SCALING = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_PARTS = ("k", "v", "cache k_scales", "cache k_zeros", "cache v_scales", "cache v_zeros")
_SIDE = (torch.float32, torch.uint8, torch.float32, torch.uint8)


def _on(stream):
    """Outputs made here belong to the stream that fills them."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _heads(x, what, dtype=None):
    """[tokens, heads, head_dim] of one argument: 16-bit, unit stride inside a head."""
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError(f"{what} must be a [tokens, heads, head_dim] tensor")
    if x.dtype not in (torch.float16, torch.bfloat16) or (dtype is not None and x.dtype != dtype):
        raise ValueError(f"{what} must be {dtype or 'float16 or bfloat16'}, got {x.dtype}")
    st = x.stride()
    if st[2] != 1 and x.shape[2] > 1:
        raise ValueError(f"{what} must be contiguous inside a head")
    return x.shape, (st[0] if x.shape[0] > 1 else 0), (st[1] if x.shape[1] > 1 else 0)


def _here(dev, *ts):
    """CUDA tensors of the current device (strided ones allowed)."""
    for t in ts:
        if t.get_device() != dev:
            if not t.is_cuda:
                raise ValueError("tensors must be CUDA tensors")
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{dev}")


def _plain(dev, t, what, dtype, shape):
    """A contiguous tensor of one dtype and shape on the current device: one look where it is, the reasons
    where it is not (single-token calls are as long as their checks)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return
    _need(t, what, (dtype,), shape)
    _need_cuda(t)


def _device():
    return torch.cuda.current_device() if torch.cuda.is_initialized() or torch.cuda.is_available() else -2


def _raw_stream(stream, dev):
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _six(cache, bits):
    """A cache's tensors for the native front (which answers None where one is not there)."""
    if cache.__class__ is not dict:
        return (None,) * 6
    get = cache.get
    if bits == 16:
        return get("k"), get("v"), None, None, None, None
    return get("k"), get("v"), get("k_scales"), get("k_zeros"), get("v_scales"), get("v_zeros")


def _cache(cache, bits, kv_heads, head_dim, dtype, dev):
    """Pointers of a cache's tensors after checking them, and (pages, page_size, kv_heads, head_dim).
    kv_heads, head_dim and dtype (of 16 bits) are checked where given."""
    if bits not in (16, 8, 4):
        raise ValueError("bits must be 16, 8 or 4")
    try:
        k, v = cache["k"], cache["v"]
        side = () if bits == 16 else (cache["k_scales"], cache["k_zeros"], cache["v_scales"], cache["v_zeros"])
    except (KeyError, TypeError):
        raise ValueError("a cache needs k and v, and scales and zeros of both below 16 bits") from None
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("cache k must be a [pages, kv_heads, page_size, row] tensor")
    pages, H, P, row = k.shape
    D = row if bits == 16 else row * 8 // bits
    if bits == 16:
        want = dtype if dtype is not None else (k.dtype if k.dtype is torch.float16 else torch.bfloat16)
    else:
        want = torch.uint8
    heads, d = kv_heads or H, head_dim or D
    _plain(dev, k, "cache k", want, (pages, heads, P, d if bits == 16 else d * bits // 8))
    _plain(dev, v, "cache v", want, k.shape)
    if bits == 16:
        return (k.data_ptr(), v.data_ptr(), None, None, None, None), pages, P, H, D
    vectors = (pages, H, P)
    for t, name, dt in zip(side, _PARTS[2:], _SIDE):
        _plain(dev, t, name, dt, vectors)
    return (k.data_ptr(), v.data_ptr(), *[t.data_ptr() for t in side]), pages, P, H, D


def new_cache(pages, kv_heads, head_dim, page_size=64, bits=16, dtype=torch.bfloat16, device=None):
    """An empty cache (zeros).  16 bits: values of `dtype`; 8 or 4 bits: codes, scales, zeros."""
    if bits not in (16, 8, 4):
        raise ValueError("bits must be 16, 8 or 4")
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("dtype must be float16 or bfloat16")
    device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    shape = (pages, kv_heads, page_size)
    if bits == 16:
        return {s: torch.zeros(*shape, head_dim, dtype=dtype, device=device) for s in ("k", "v")}
    cache = {s: torch.zeros(*shape, head_dim * bits // 8, dtype=torch.uint8, device=device) for s in ("k", "v")}
    for s in ("k", "v"):
        cache[s + "_scales"] = torch.zeros(shape, dtype=torch.float32, device=device)
        cache[s + "_zeros"] = torch.zeros(shape, dtype=torch.uint8, device=device)
    return cache


def rotary_frequencies(rotary_dim, base=10000.0, scaling=None, factor=1.0, original_len=0, beta_fast=32.0,
                       beta_slow=1.0, device=None):
    """(inv_freq float64 [rotary_dim / 2] on the device, attention_factor) of ``rotary``.

    scaling None, "linear", "ntk" or "yarn" (gptq_rotary_frequencies), for contexts `factor` times as
    long as the model's own; "yarn" needs that length as original_len."""
    if scaling not in SCALING:
        raise ValueError(f"scaling must be one of {list(SCALING)}")
    if not isinstance(rotary_dim, int) or rotary_dim <= 0 or rotary_dim % 2:
        raise ValueError("rotary_dim must be a positive even number")
    freq = (ctypes.c_double * (rotary_dim // 2))()
    a = ctypes.c_float()
    st = lib().gptq_rotary_frequencies(rotary_dim, float(base), SCALING[scaling], float(factor), int(original_len),
                                       float(beta_fast), float(beta_slow), freq, ctypes.byref(a))
    _check(st, "gptq_rotary_frequencies")
    device = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    return torch.tensor(list(freq), dtype=torch.float64).to(device), a.value


def rotary(q, k, positions, inv_freq, attention_factor=1.0, interleaved=False, out=None, stream=None):
    """Rotary positions of q [tokens, heads, head_dim] and k [tokens, kv_heads, head_dim] (or None).

    The first 2 * len(inv_freq) values of each head turn, in pairs (i, i + r/2), or (2i, 2i + 1) if
    `interleaved`, by positions[t] * inv_freq[i]; the rest is copied.  q and k may be strided views
    of a fused projection.  Returns (q, k) as new tensors, or written to out = (q_out, k_out), which
    may be (q, k) themselves."""
    if out is None and stream is None:
        r = front().rotary(q, k, positions, inv_freq, attention_factor, interleaved)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(r, "gptq_rotary")
    (T, Hq, D), qt, qh = _heads(q, "q")
    Hk, kt, kh = 0, 0, 0
    if k is not None:
        (Tk, Hk, Dk), kt, kh = _heads(k, "k", q.dtype)
        if (Tk, Dk) != (T, D):
            raise ValueError("k must have q's tokens and head_dim")
    dev = _device()
    _plain(dev, positions, "positions", torch.int32, (T,))
    if not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must be a 1-D float64 tensor")
    _plain(dev, inv_freq, "inv_freq", torch.float64, inv_freq.shape)
    if out is None:
        _here(dev, q) if k is None else _here(dev, q, k)
        with _on(stream):
            qo = q.new_empty((T, Hq, D))
            ko = None if k is None else q.new_empty((T, Hk, D))
        qot, qoh, kot, koh = Hq * D, D, Hk * D, D
    else:
        if not isinstance(out, (tuple, list)) or len(out) != 2 or (out[1] is None) != (k is None):
            raise ValueError("out must be a pair (q_out, k_out)")
        qo, ko = out
        shape, qot, qoh = _heads(qo, "out q", q.dtype)
        kot = koh = 0
        if tuple(shape) != (T, Hq, D):
            raise ValueError("out q must have q's shape")
        if k is not None:
            shape, kot, koh = _heads(ko, "out k", q.dtype)
            if tuple(shape) != (T, Hk, D):
                raise ValueError("out k must have k's shape")
        _here(dev, *(t for t in (q, k, qo, ko) if t is not None))
    st = lib().gptq_rotary(q.data_ptr(), None if k is None else k.data_ptr(), _DTYPE[q.dtype], T, Hq, Hk, D,
                           2 * inv_freq.shape[0], 1 if interleaved else 0, qt, qh, kt, kh, positions.data_ptr(),
                           inv_freq.data_ptr(), attention_factor, qo.data_ptr(),
                           None if ko is None else ko.data_ptr(), qot, qoh, kot, koh, _raw_stream(stream, dev))
    _check(st, "gptq_rotary")
    return qo, ko


def cache_write(k, v, cache, slots, bits=16, stream=None):
    """Store k and v [tokens, kv_heads, head_dim] of each token in its slot (int32 [tokens]), quantized
    below 16 bits.  A slot outside the cache (-1 for a padded token) is left out; the others must
    differ.  Returns the cache."""
    if stream is None:
        r = front().cache_write(k, v, *_six(cache, bits), slots, bits)
        if r is True:
            return cache
        if r is not None:
            _check(r, "gptq_cache_write")
    (T, H, D), kt, kh = _heads(k, "k")
    shape, vt, vh = _heads(v, "v", k.dtype)
    if tuple(shape) != (T, H, D):
        raise ValueError("v must have k's shape")
    dev = _device()
    ptrs, pages, P, _, _ = _cache(cache, bits, H, D, k.dtype, dev)
    _plain(dev, slots, "slots", torch.int32, (T,))
    _here(dev, k, v)
    st = lib().gptq_cache_write(k.data_ptr(), v.data_ptr(), _DTYPE[k.dtype], T, H, D, kt, kh, vt, vh, *ptrs, bits,
                                pages, P, slots.data_ptr(), _raw_stream(stream, dev))
    _check(st, "gptq_cache_write")
    return cache


def cache_read(cache, slots, bits=16, dtype=None, stream=None):
    """(k, v) [len(slots), kv_heads, head_dim] of the slots (int32), each value rounded once to `dtype`
    (default: the cache's own, bfloat16 below 16 bits).  A slot outside the cache reads as zeros."""
    if dtype is None:
        own = cache["k"].dtype if isinstance(cache, dict) and isinstance(cache.get("k"), torch.Tensor) else None
        dtype = own if own in (torch.float16, torch.bfloat16) else torch.bfloat16
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("dtype must be float16 or bfloat16")
    if stream is None:
        r = front().cache_read(*_six(cache, bits), slots, bits, dtype is torch.float16)
        if r.__class__ is tuple:
            return r
        if r is not None:
            _check(r, "gptq_cache_read")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be a 1-D int32 tensor")
    dev = _device()
    ptrs, pages, P, H, D = _cache(cache, bits, None, None, dtype, dev)
    _plain(dev, slots, "slots", torch.int32, slots.shape)
    n = slots.shape[0]
    with _on(stream):
        k = slots.new_empty((n, H, D), dtype=dtype)
        v = slots.new_empty((n, H, D), dtype=dtype)
    st = lib().gptq_cache_read(*ptrs, bits, pages, P, slots.data_ptr(), n, H, D, _DTYPE[dtype], k.data_ptr(),
                               v.data_ptr(), _raw_stream(stream, dev))
    _check(st, "gptq_cache_read")
    return k, v


def paged_attention(q, cache, page_table, kv_lens, q_starts, bits=16, max_q_len=None, causal=True, scale=None,
                    out=None, stream=None):
    """Attention of new tokens over a paged cache that already holds their keys and values.

    q:          [tokens, heads, head_dim], the rows of sequence s being q_starts[s] .. q_starts[s+1]-1
    page_table: int32 [seqs, width], the pages of each sequence in order
    kv_lens:    int32 [seqs], keys of each sequence, its new tokens included
    q_starts:   int32 [seqs + 1]
    max_q_len:  the most rows of one sequence, if known (1 for single-token steps); default: tokens
    causal:     row i of n sees the keys 0 .. kv_len - n + i, else all of its sequence's keys
    scale:      of the scores, default head_dim ** -0.5
    Rows that see no key are zeros; rows of no sequence are left as they were in `out`."""
    if out is None and stream is None:
        r = front().paged_attention(q, *_six(cache, bits), page_table, kv_lens, q_starts, bits, max_q_len, causal, scale)
        if isinstance(r, torch.Tensor):
            return r
        if r is not None:
            _check(r, "gptq_paged_attention")
    (T, Hq, D), qt, qh = _heads(q, "q")
    dev = _device()
    ptrs, pages, P, H, _ = _cache(cache, bits, None, D, q.dtype, dev)
    if Hq % H:
        raise ValueError("heads must be a multiple of the cache's kv_heads")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [seqs, width] int32 tensor")
    S, width = page_table.shape
    _plain(dev, page_table, "page_table", torch.int32, page_table.shape)
    _plain(dev, kv_lens, "kv_lens", torch.int32, (S,))
    _plain(dev, q_starts, "q_starts", torch.int32, (S + 1,))
    _here(dev, q)
    if out is None:
        with _on(stream):
            out = q.new_empty((T, Hq, D))
    else:
        _plain(dev, out, "out", q.dtype, (T, Hq, D))
    if max_q_len is not None and (not isinstance(max_q_len, int) or max_q_len < 0):
        raise ValueError("max_q_len must be a number of rows")
    st = lib().gptq_paged_attention(q.data_ptr(), _DTYPE[q.dtype], T, Hq, H, D, qt, qh, *ptrs, bits, pages, P,
                                    page_table.data_ptr(), width, kv_lens.data_ptr(), q_starts.data_ptr(), S,
                                    T if max_q_len is None else min(max_q_len, T), 1 if causal else 0,
                                    D ** -0.5 if scale is None else scale, out.data_ptr(), _raw_stream(stream, dev))
    _check(st, "gptq_paged_attention")
    return out
