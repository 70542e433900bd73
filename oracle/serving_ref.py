"""Float64 NumPy restatement of the serving operators: rotary positions, the quantized vectors
of a paged key/value cache, and attention over it.  Test infrastructure; nothing here is shared
with the library."""

from __future__ import annotations

import math

import numpy as np


def rotary_frequencies(r, base=10000.0, scaling=None, factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """(angle per position of each pair, factor on the rotated values)."""
    i = np.arange(r // 2, dtype=np.float64)
    if scaling == "ntk":
        base = base * factor ** (r / (r - 2))
    f = base ** (-2.0 * i / r)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "yarn":
        return f, 1.0

    def pair(turns):  # the pair that turns so often within original_len
        return r / 2 * math.log(original_len / (2 * math.pi * turns)) / math.log(base)

    lo, hi = max(math.floor(pair(beta_fast)), 0), min(math.ceil(pair(beta_slow)), r - 1)
    slow = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return f / factor * slow + f * (1 - slow), (0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0)


def rotary(x, positions, freq, factor=1.0, interleaved=False):
    """x [tokens, heads, d] with the pairs of its first 2 len(freq) values turned."""
    x = np.asarray(x, dtype=np.float64)
    r = 2 * len(freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(freq)[None]
    c, s = factor * np.cos(ang)[:, None], factor * np.sin(ang)[:, None]
    ia, ib = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
    y = x.copy()
    y[..., ia] = x[..., ia] * c - x[..., ib] * s
    y[..., ib] = x[..., ib] * c + x[..., ia] * s
    return y


def quantize_vectors(x, bits):
    """(codes, scales float32, zeros) of each vector of the last axis; the code nearest to the exact
    quotient, half to even.  A vector that is not finite, or whose range is not: scale NaN, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    maxq = 2 ** bits - 1
    with np.errstate(all="ignore"):
        lo, hi = np.minimum(x.min(-1), 0.0), np.maximum(x.max(-1), 0.0)
        flat = (lo == 0) & (hi == 0)
        lo, hi = np.where(flat, -1.0, lo), np.where(flat, 1.0, hi)
        s = ((hi - lo).astype(np.float32).astype(np.float64) / maxq).astype(np.float32)
        bad = ~np.isfinite(x).all(-1) | ~np.isfinite(s)
        sd = np.where(bad, 1.0, s.astype(np.float64))
        xs, ls = np.where(bad[..., None], 0.0, x), np.where(bad, 0.0, lo)
        z = np.clip(np.rint(-ls / sd), 0, maxq)
        c = np.clip(np.rint(xs / sd[..., None]) + z[..., None], 0, maxq)
    s = np.where(bad, np.float32(np.nan), s).astype(np.float32)
    return np.where(bad[..., None], 0, c).astype(np.uint8), s, np.where(bad, 0, z).astype(np.uint8)


def pack_vector_codes(c, bits):
    """Codes of the last axis in bytes, least significant bits first."""
    return c if bits == 8 else (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack_vector_codes(b, bits):
    if bits == 8:
        return b
    out = np.empty(b.shape[:-1] + (b.shape[-1] * 2,), dtype=np.uint8)
    out[..., 0::2], out[..., 1::2] = b & 15, b >> 4
    return out


def vector_values(codes, scales, zeros):
    """float32(scale * (code - zero)), as float64."""
    d = codes.astype(np.float32) - zeros.astype(np.float32)[..., None]
    return (scales[..., None] * d).astype(np.float32).astype(np.float64)


def attention(q, k, v, causal=True, scale=None):
    """q [n, heads, d] over one sequence's k, v [L, kv_heads, d]: (out, slack) where slack[i, h] =
    (sum_j p_j |v_j|, largest scale * sum |q||k_j| over the keys seen) bounds what roundings do."""
    n, Hq, d = q.shape
    L, H, _ = k.shape
    scale = d ** -0.5 if scale is None else scale
    out, mass, size = np.zeros((n, Hq, d)), np.zeros((n, Hq, d)), np.zeros((n, Hq))
    for i in range(n):
        m = max(0, min(L, L - n + i + 1)) if causal else L
        if m == 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // (Hq // H)], v[:m, h // (Hq // H)]
            s = scale * (kk @ q[i, h])
            p = np.exp(s - s.max())
            p /= p.sum()
            out[i, h], mass[i, h] = p @ vv, p @ np.abs(vv)
            size[i, h] = scale * (np.abs(kk) @ np.abs(q[i, h])).max()
    return out, mass, size
