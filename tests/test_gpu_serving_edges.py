"""Attention over a paged cache at the edges of its inputs: sizes and strides that the common cases do not have, and
values at the ends of the types' ranges, against the float64 oracle.

Bounds, tighter than those of test_gpu_serving, from the roundings that each kernel makes (u = half a step of the
16-bit type, 2^-8 bfloat16, 2^-11 float16; size = largest scale * sum|q||k| over the keys seen; mass = sum p |v|):
* scores: fp32 sums of exact products, D 2^-24 size.  Few rows over codes: the products are with 1024 + code (64 +
  code of 4 bits), whose sums are off by D 2^-24 (1024 + 255) s sum|q| (s the largest key scale), and a query element is
  rounded where it is under 2^-14 of its row's largest, by 2^-25 of that.  With d of the scores, probabilities move by
  expm1(2 d): their own score's error and the sum's.
* probabilities: u of the products' type (float16 for few rows over codes, otherwise the call's), 2^-20 for exp2 and
  the fp32 sums.  Float16 has no steps below 2^-24: a weight there is off by 2^-25 of what the type's range leaves
  above the largest (few rows 2^15; more 2^7 above a maximum that may be 2^8 behind), summed over the keys seen.
* values: u of the call's type where many rows meet codes, none otherwise; then u |o| for the output.
"""

import numpy as np
import pytest
import torch

import post_weight_quantization_layer_b200 as gq
from oracle import serving_ref as R
from tests.gpu_util import device
from tests.test_gpu_serving import U, _attend, _case, _np, _randn

pytestmark = pytest.mark.gpu


def _bound(c, s, q, rows, ref, mass, size, dtype, bits, scale=None):
    """Of the rows q [n, heads, D] of sequence s; rows: the sequence's rows of a kv head."""
    k, v = c["vals"][s]
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    few = rows <= 16
    u = U[dtype]
    up = 2.0 ** -11 if few and bits < 16 else u
    ds = (D + 8) * 2.0 ** -24 * size
    if few and bits < 16:
        big = np.abs(k).max() / (7.5 if bits == 4 else 127.5)  # the range holds 0: at least half of it is one value's
        ds = ds + scale * (D * 2.0 ** -24 * 1279 * big * np.abs(q).sum(-1)
                           + 2.0 ** -25 * np.abs(q).max(-1) * np.abs(k).sum(-1).max())
    rel = up + (0.0 if few or bits == 16 else u) + 2.0 ** -20 + np.expm1(2 * ds)
    flush = 0.0
    if up == 2.0 ** -11:
        flush = 2.0 ** (-40 if few else -32) * len(k) * np.abs(v).max()
    return u * np.maximum(np.abs(ref), torch.finfo(dtype).tiny) + rel[..., None] * mass + flush


def _check(c, out, new, dtype, bits, scale=None, causal=True):
    at = 0
    for s, n in enumerate(new):
        if n:
            k, v = c["vals"][s]
            q = _np(c["q"][at:at + n])
            ref, mass, size = R.attention(q, k, v, causal, scale)
            err = np.abs(_np(out[at:at + n]) - ref)
            most = _bound(c, s, q, n * q.shape[1] // max(k.shape[1], 1), ref, mass, size, dtype, bits, scale)
            assert np.all(err <= most), (s, float(np.nanmax(err / most)))
        at += n


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("group", [1, 3, 5])
def test_few_items_share_clusters_with_heads_of_64(bits, group):
    """Odd numbers of rows of 16 pieces each: half a warp has one piece less than the other when the CTAs of a
    cluster meet."""
    have, new = [1000, 511, 30], [1, 3, 1]
    c = _case(have, new, 2, 64, 64, bits, torch.bfloat16, 40 + bits + group, Hq=2 * group)
    out = _attend(c, bits, max_q_len=3)
    _check(c, out, new, torch.bfloat16, bits)
    for _ in range(5):
        assert torch.equal(out, _attend(c, bits, max_q_len=3))
    assert gq.device_status() == 0
