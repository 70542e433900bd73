"""Attention over a paged cache at the edges of its inputs: sizes and strides that the common cases do not have, and
values at the ends of the types' ranges, against the float64 oracle.

Bounds, tighter than those of test_gpu_serving, from the roundings that each kernel makes (u = half a step of the
16-bit type, 2^-8 bfloat16, 2^-11 float16; size = largest scale * sum|q||k| over the keys seen; mass = sum p |v|):
* scores: fp32 sums of exact products, D 2^-24 size.  Few rows over codes: the products are with 1024 + code (64 +
  code of 4 bits), whose sums are off by D 2^-24 (1024 + 255) s sum|q| (s the largest key scale), and a query element is
  rounded where it is under 2^-28 of its row's largest, by 2^-39 of that.  With d of the scores, probabilities move by
  expm1(2 d): their own score's error and the sum's.
* probabilities: u of the products' type (float16 for few rows over codes, otherwise the call's), 2^-20 for exp2 and
  the fp32 sums.  Float16 has no steps below 2^-24: a weight there is off by 2^-25 of what the type's range leaves
  above the largest (few rows 2^15; more 2^7 above a maximum that may be 2^8 behind), summed over the keys seen.
* values: none, behind codes neither; then u |o| for the output.
"""

import numpy as np
import pytest
import torch

import post_weight_quantization_layer_b200 as gq
from oracle import serving_ref as R
from tests.gpu_util import device
from tests.test_gpu_serving import CHUNK, GUESS, LATE, STEP, U, _attend, _case, _np, _randn

pytestmark = pytest.mark.gpu


def _bound(c, s, q, rows, ref, mass, size, dtype, bits, scale=None):
    """Of the rows q [n, heads, D] of sequence s; rows: the sequence's rows of a kv head."""
    k, v = c["vals"][s]
    if not len(k):
        return np.zeros_like(ref)  # no keys: zeros
    D = q.shape[-1]
    scale = D ** -0.5 if scale is None else scale
    few = rows <= 16
    u = U[dtype]
    up = 2.0 ** -11 if few and bits < 16 else u
    ds = (D + 8) * 2.0 ** -24 * size
    if few and bits < 16:
        big = np.abs(k).max() / (7.5 if bits == 4 else 127.5)  # the range holds 0: at least half of it is one value's
        ds = ds + scale * (D * 2.0 ** -24 * 1279 * big * np.abs(q).sum(-1)
                           + 2.0 ** -39 * np.abs(q).max(-1) * np.abs(k).sum(-1).max())
    rel = up + 2.0 ** -20 + np.expm1(np.minimum(2 * ds, 700))
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


# ------------------------------------------------------------------ values at the ends of the types' ranges
def _outside(kind, L, n, H, group, D, seed):
    """Keys [L, H, D], queries [n, H * group, D] (bfloat16) and the scale; scores of ordinary size from operands that
    are not."""
    g = torch.Generator().manual_seed(seed)
    k, q = torch.randn(L, H, D, generator=g), torch.randn(n, H * group, D, generator=g)
    scale = None
    if kind == "key_80000":  # a first key that the first row sees alone
        k[:, :, 0] = 0.0
        k[0] = 0.0
        k[0, :, 0] = 80000.0
        q[..., 0] = -1e-4
    elif kind == "keys_1e5":  # every key, in one channel
        k[..., 0] = 1e5 * (1 + 0.1 * torch.rand(L, H, generator=g))
        q[..., 0] = -1e-3
    elif kind == "keys_1e5_up":
        k[..., 0] = 1e5 * (1 + 0.1 * torch.rand(L, H, generator=g))
        q[..., 0] = 1e-3
    elif kind == "queries_1e5":
        k[..., 0] = 1e-4 * torch.rand(L, H, generator=g)
        q[..., 0] = -1e5
    elif kind == "queries_1e-7":
        q *= 1e-7
        scale = 1e6
    elif kind == "small_keys":
        k *= 1e-9
        q *= 1e9
    elif kind == "large_keys":
        k *= 1e9
        q *= 1e-9
    elif kind == "queries_2^127":
        k *= 2.0 ** -124
        q[..., 0] = 1.5 * 2.0 ** 127
        q[..., 1:] *= 2.0 ** 120
    return q.bfloat16(), k.bfloat16(), scale


KINDS = ["key_80000", "keys_1e5", "keys_1e5_up", "queries_1e5", "queries_1e-7", "small_keys", "large_keys", "queries_2^127"]


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40, 300])
@pytest.mark.parametrize("kind", KINDS)
def test_codes_outside_float16(bits, D, n, kind):
    """Queries and keys behind codes may have any size that their types have, in a prompt as token by token."""
    H, group, L, dtype = 1, 4, max(n, 150), torch.bfloat16
    q, k, scale = _outside(kind, L, n, H, group, D, 5 + D + bits)
    c = _case([L], [n], H, D, 32, bits, dtype, 5, kv=lambda s, L: (k, _randn((L, H, D), 6, dtype)), Hq=H * group)
    c["q"] = q.to(device())
    _check(c, _attend(c, bits, scale=scale), [n], dtype, bits, scale)
    assert gq.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("first", [16, 64, 200])
@pytest.mark.parametrize("have,n", [(300, 1), (300, 4), (5000, 3), (300, 90)])
def test_scores_of_minus_infinity(dtype, first, have, n):
    """Keys whose scores are -infinity weigh nothing, wherever they lie: the rest is the answer; a row with no other
    key is zeros."""
    D, bits, group = 64, 16, 4

    def kv(s, L):
        k, v = _randn((L, 1, D), 1, dtype), _randn((L, 1, D), 2, dtype)
        k[:first, 0, 3] = -float("inf")
        return k, v

    c = _case([have], [n], 1, D, 16, bits, dtype, 4, kv=kv, Hq=group)
    c["q"][:, :, 3] = c["q"][:, :, 3].abs() + 0.25
    out = _attend(c, bits)
    k, v = c["vals"][0]
    c["vals"][0] = (k[first:], v[first:])
    _check(c, out, [n], dtype, bits)
    c = _case([first], [min(n, first)], 1, D, 16, bits, dtype, 4, kv=kv, Hq=group)
    c["q"][:, :, 3] = c["q"][:, :, 3].abs() + 0.25
    assert not _attend(c, bits).any()


@pytest.mark.parametrize("dtype,bits", [(torch.float16, 16), (torch.float16, 8), (torch.float16, 4), (torch.bfloat16, 8),
                                        (torch.bfloat16, 4), (torch.bfloat16, 16)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_many_small_weights_beside_a_large_one(dtype, bits, n):
    """A first key that outweighs each of 8191 others by 2^26, and whose value is zero: the others, 2^-13 together, are
    the answer.  Sequences enough that a CTA meets many keys of one of them."""
    D, L, H, group, S = 64, 8192, 8, 4, 16

    def kv(s, L):
        k, v = torch.zeros(L, H, D, dtype=dtype), torch.ones(L, H, D, dtype=dtype)
        k[0], v[0] = 1.126, 0.0  # score 0.125 * 64 * 2 * 1.126 = 26 ln 2
        return k, v

    c = _case([L], [n], H, D, 64, bits, dtype, 4, kv=kv, Hq=H * group)
    dev = device()
    c["table"] = c["table"].expand(S, -1).contiguous()
    c["lens"] = torch.full((S,), L, dtype=torch.int32, device=dev)
    c["starts"] = torch.arange(S + 1, dtype=torch.int32, device=dev) * n
    c["q"] = torch.full((S * n, H * group, D), 2.0, dtype=dtype, device=dev)
    out = _attend(c, bits, max_q_len=n)
    k, v = c["vals"][0]
    few = n * group <= 16
    ref = np.empty(n)  # the same of every head and value
    for i in range(n):
        score = 0.125 * k[:L - n + i + 1, 0] @ np.full(D, 2.0)
        w = np.exp(score - score[0])
        ref[i] = w @ v[:len(w), 0, 0] / w.sum()
    rel = U[dtype] + (2.0 ** -11 if few and bits < 16 else U[dtype]) + 2.0 ** -12  # 2^-12: scores of 26, in float32
    err = np.abs(_np(out).reshape(S, n, -1) - ref[:, None])
    assert np.all(err <= rel * ref[:, None] + L * 2.0 ** (-40 if few else -32))


# ------------------------------------------------------------------ the common cases, closer; shapes at the ends
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("H,group,D,P", [(2, 1, 128, 64), (2, 4, 64, 16), (1, 8, 128, 32), (1, 5, 64, 256)])
@pytest.mark.parametrize("lens", [STEP, GUESS, CHUNK, LATE], ids=["step", "guess", "chunk", "late"])
def test_attention_within_its_own_roundings(dtype, bits, H, group, D, P, lens):
    have, new = lens
    c = _case(have, new, H, D, P, bits, dtype, 70 + D + bits, Hq=H * group)
    _check(c, _attend(c, bits, max_q_len=max(new)), new, dtype, bits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("n", [1, 24])
def test_long_context_within_its_own_roundings(dtype, bits, n):
    """131072 keys that weigh much the same.  Roundings are many and independent: the 2-norm of the error is held to 4
    times the quadrature sum of the relative errors' spreads, u / sqrt(3) each of the output and of the probabilities
    (of the products' type)."""
    D, L, group = 128, 131072, 4
    g = torch.Generator().manual_seed(bits)

    def kv(s, L):
        return (0.7 * torch.randn(L, 1, D, generator=g)).to(dtype), torch.randn(L, 1, D, generator=g).to(dtype)

    c = _case([L], [n], 1, D, 128, bits, dtype, 3, kv=kv, Hq=group)
    out = _np(_attend(c, bits))
    k, v = c["vals"][0]
    q = _np(c["q"])
    ref = np.empty_like(q)
    for i in range(n):
        m = L - n + i + 1
        s = q[i] @ k[:m, 0].T / np.sqrt(D)
        p = np.exp(s - s.max(-1, keepdims=True))
        ref[i] = p @ v[:m, 0] / p.sum(-1, keepdims=True)
    u, few = U[dtype], n * group <= 16
    up = 2.0 ** -11 if few and bits < 16 else u
    most = 4 * np.sqrt((u ** 2 + up ** 2) / 3)
    assert np.linalg.norm(out - ref) <= most * np.linalg.norm(ref)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("group,D", [(16, 64), (17, 128), (32, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("have,new", [([300, 1, 129], [1, 1, 1]), ([200, 40, 3, 0], [9, 30, 3, 0])],
                         ids=["tokens", "chunks"])
def test_groups_to_64(bits, group, D, have, new):
    """Heads of a kv head up to 64: beyond 16 even single tokens are many rows."""
    c = _case(have, new, 2, D, 16, bits, torch.bfloat16, 80 + group, Hq=2 * group)
    _check(c, _attend(c, bits, max_q_len=max(new)), new, torch.bfloat16, bits)
    assert gq.device_status() == 0


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("have,new", [([300, 70], [1, 2]), ([300, 70], [200, 33])], ids=["tokens", "chunks"])
@pytest.mark.parametrize("order", ["heads first", "part of a wider row", "one head for all", "one token for all"])
def test_queries_of_any_strides(bits, have, new, order):
    """Queries laid out heads first, with gaps, or repeated (strides of zero)."""
    H, group, D, dtype = 2, 3, 64, torch.bfloat16
    c = _case(have, new, H, D, 32, bits, dtype, 90, Hq=H * group)
    T = sum(new)
    if order == "heads first":
        c["q"] = _randn((H * group, T, D), 91, dtype).to(device()).transpose(0, 1)
    elif order == "part of a wider row":
        c["q"] = _randn((T + 3, H * group + 2, 2 * D), 91, dtype).to(device())[3:, 1:-1, D:]
    elif order == "one head for all":
        c["q"] = _randn((T, 1, D), 91, dtype).to(device()).expand(T, H * group, D)
    else:
        c["q"] = _randn((1, H * group, D), 91, dtype).to(device()).expand(T, H * group, D)
    _check(c, _attend(c, bits, max_q_len=max(new)), new, dtype, bits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("lens", [STEP, GUESS, CHUNK], ids=["step", "guess", "chunk"])
def test_attention_gives_the_same_bits_again(dtype, bits, lens):
    """Every form, with other work and other contents of the workspace between."""
    have, new = lens
    c = _case(have, new, 2, 64, 32, bits, dtype, 95, Hq=6)
    other = _case([900, 20], [700, 20], 2, 128, 16, bits, dtype, 96, Hq=8)
    want = _attend(c, bits, max_q_len=max(new))
    for _ in range(4):
        _attend(other, bits)
        assert torch.equal(want, _attend(c, bits, max_q_len=max(new)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n", [1, 300])
def test_error_over_codes_is_that_of_the_output_and_the_weights(dtype, bits, n):
    """The 2-norm of the error beside that of an exact answer rounded once.  A weight's relative rounding is spread as
    the output's; for values of random signs the expected square of sum p v is sum p^2 v^2, and so the square of what
    the weights' roundings make of it is expected to be as large as that of the output's own: 2 together, where weights
    are of the call's type (1 + 2^-6 for few rows of a bfloat16 call, whose weights are float16).  Values rounded to the
    call's type would bring as much again, 3.  Over 1024 outputs and more the squares are held to half-way between,
    2.5 (1.5)."""
    D, L, H, group = 128, 1500, 2, 4
    c = _case([L], [n], H, D, 64, bits, dtype, 17 + bits, Hq=H * group)
    out = _np(_attend(c, bits))
    ref, _, _ = R.attention(_np(c["q"]), *c["vals"][0])
    once = np.linalg.norm(_np(torch.from_numpy(ref).to(dtype)) - ref)
    assert np.linalg.norm(out - ref) <= np.sqrt(1.5 if n * group <= 16 and dtype is torch.bfloat16 else 2.5) * once


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("n", [1, 3, 40, 300])
@pytest.mark.parametrize("size", [2.0 ** -120, 2.0 ** -60, 1e-7, 1e7, 2.0 ** 100, "mixed"])
def test_values_behind_codes_of_any_size(bits, n, size):
    """Values from the smallest to the largest that bfloat16 has, one size or all in one sequence."""
    D, H, group, L, dtype = 64, 1, 4, max(n, 150), torch.bfloat16
    v = _randn((L, H, D), 6, torch.float32)
    v *= torch.logspace(-8, 8, L, base=10.0)[torch.randperm(L)][:, None, None] if size == "mixed" else size
    c = _case([L], [n], H, D, 16, bits, dtype, 5, kv=lambda s, L: (_randn((L, H, D), 5, dtype), v.to(dtype)), Hq=H * group)
    _check(c, _attend(c, bits), [n], dtype, bits)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 40, 200])
def test_float16_calls_over_values_past_their_range(bits, D, n):
    """Values behind codes of 1e5, 2^40 in one channel of one key: the answer is in float16's range where they weigh
    little, and infinite where not."""
    H, group, L, dtype = 1, 4, max(n, 220), torch.bfloat16

    def kv(s, L):
        k, v = _randn((L, H, D), 5, dtype), _randn((L, H, D), 6, dtype)
        v[7] *= 1e5
        k[7] = 0.0
        v[11, :, 3] = 2.0 ** 40
        return k, v

    c = _case([L], [n], H, D, 32, bits, dtype, 5, kv=kv, Hq=H * group)
    c["q"] = c["q"].half()
    out, (k, v) = _attend(c, bits), c["vals"][0]
    q = _np(c["q"][:n])
    ref, mass, size = R.attention(q, k, v)
    most = _bound(c, 0, q, n * group, ref, mass, size, torch.float16, bits)
    out = _np(out)
    over = np.abs(ref) - most > 65520
    assert over.any() and np.all(np.isinf(out[over]) & (np.sign(out[over]) == np.sign(ref[over])))
    fine = np.abs(ref) + most < 65504
    assert fine.any() and np.all(np.abs(out - ref)[fine] <= most[fine])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("have,n", [(260, 200), (40, 4), (3000, 2)])
def test_unseen_minus_infinity(dtype, bits, have, n):
    """As test_attention_unseen_nonfinite, with -infinity: it reaches the rows that see it and no others."""
    D, H, bad = 64, 2, have - n // 2

    def kv(s, L):
        k, v = _randn((L, H, D), 1, dtype), _randn((L, H, D), 2, dtype)
        k[bad, 0, 3] = v[bad] = -float("inf")
        return k, v

    c = _case([have], [n], H, D, 16, bits, dtype, 3, kv=kv, Hq=4)
    out, first = _np(_attend(c, bits)), bad - (have - n)
    k, v = c["vals"][0]
    c["vals"][0] = k[:bad], v[:bad]
    q = _np(c["q"][:first])
    ref, mass, size = R.attention(q, k[:bad], v[:bad])
    assert np.all(np.abs(out[:first] - ref) <= _bound(c, 0, q, n * 2, ref, mass, size, dtype, bits))
    assert not np.isfinite(out[first:]).any()
