"""GPU parity of the serving operators (rotary, cache_write, cache_read, paged_attention) against
the float64 oracle.

Bounds, from the roundings of each operator (u = half a step of the 16-bit type: 2^-8 bfloat16,
2^-11 float16):
* rotary: the reduced angle is rounded to fp32 (in units of pi, at most 1: pi 2^-25 of angle), sine and
  cosine have two units in the last place (2^-22), products and their sum three more roundings:
  together below 2^-20 A (|a| + |b|), then one rounding u |y|.
* cache: codes, scales and zero points are equal; values read back are the fp32 product rounded once.
* attention: scores carry the fp32 sums' error d 2^-24 scale sum|q||k|, and u of the same for codes whose
  values are rounded to 16 bits; each probability moves by at most twice that (its own score and the
  sum), plus its own rounding (2^-8 where the products of probabilities and values run in bf16, u
  otherwise; 2^-20 for exp2 and the sums); values behind codes another u; then u |o|.
With integer values and q = 0 every probability is 1 and every sum exact, so there the outcome is the
mean rounded once (after a division: two roundings), which shows every missing or repeated key.
"""

import numpy as np
import pytest
import torch

import post_weight_quantization_layer_b200 as gq
from oracle import serving_ref as R
from post_weight_quantization_layer_b200 import api
from tests.gpu_util import device

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _np(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, seed, dtype, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * mult).to(dtype)


# ------------------------------------------------------------------ rotary
def _rotary_check(y, x, pos, f, a, inter, dtype):
    xn, r = _np(x), 2 * len(f)
    ref = R.rotary(xn, pos.cpu().numpy(), f.cpu().numpy(), a, inter)
    ia, ib = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
    amp = np.zeros_like(xn)
    amp[..., ia] = amp[..., ib] = np.abs(xn[..., ia]) + np.abs(xn[..., ib])
    # below the type's normal range its steps stop shrinking: half a step of the smallest normal
    bound = U[dtype] * np.maximum(np.abs(ref), torch.finfo(dtype).tiny) + 2.0 ** -20 * a * amp
    assert np.all(np.abs(_np(y) - ref) <= bound)
    assert torch.equal(y[..., r:].cpu(), x[..., r:].cpu())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,r", [(1, 32, 32, 128, 128), (7, 12, 12, 64, 32), (603, 5, 1, 64, 64), (3, 4, 2, 80, 20),
                                         (600, 3, 3, 24, 6), (33, 64, 8, 128, 96)])
def test_rotary(dtype, inter, T, Hq, Hk, D, r):
    dev = device()
    qkv = _randn((T, Hq + 2 * Hk, D), T + D + r, dtype).to(dev)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]  # strided views of a fused projection
    before = qkv.clone()
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g).int().to(dev)
    f, a = gq.rotary_frequencies(r, scaling="yarn", factor=16.0, original_len=2048)
    yq, yk = gq.rotary(q, k, pos, f, a, inter)
    assert torch.equal(qkv, before)  # new tensors: the inputs stay
    _rotary_check(yq, q, pos, f, a, inter, dtype)
    _rotary_check(yk, k, pos, f, a, inter, dtype)
    oq, ok = gq.rotary(q, k, pos, f, a, inter, out=(q, k))  # in place, through the views
    assert oq is q and torch.equal(q, yq) and torch.equal(k, yk)
    assert torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_rotary_alone_and_empty():
    dev = device()
    x = _randn((9, 4, 64), 1, torch.float16).to(dev)
    pos = torch.arange(9, dtype=torch.int32, device=dev)
    f, a = gq.rotary_frequencies(64)
    y, none = gq.rotary(x, None, pos, f, a)
    assert none is None
    _rotary_check(y, x, pos, f, a, False, torch.float16)
    flat = x.clone().reshape(9, 256)
    api.rope_(flat, 4, 9)  # the whole-sequence form is the same formula
    _rotary_check(flat.view(9, 4, 64), x, pos, f, a, False, torch.float16)
    back, _ = gq.rotary(y, None, -pos, f, a)
    assert np.allclose(_np(back), _np(x), atol=4 * 2.0 ** -11 * 5)  # three roundings of values below 5
    e, _ = gq.rotary(x[:0], None, pos[:0], f, a)
    assert e.shape == (0, 4, 64)


# ------------------------------------------------------------------ cache
def _fill(cache, bits):
    """Everything outside the slots that a test writes: NaN, so that a stray read shows."""
    for s in ("k", "v"):
        if bits == 16:
            cache[s].fill_(float("nan"))
        else:
            cache[s].fill_(0xA5)
            cache[s + "_scales"].fill_(float("nan"))
            cache[s + "_zeros"].fill_(7)
    return cache


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [4, 8, 16])
@pytest.mark.parametrize("T,H,D,P", [(1, 1, 64, 16), (37, 3, 128, 16), (130, 8, 64, 128), (65, 2, 128, 256)])
def test_cache_write_and_read(dtype, bits, T, H, D, P):
    dev = device()
    pages = -(-T // P) + 2
    cache = _fill(gq.new_cache(pages, H, D, P, bits, dtype), bits)
    kv = _randn((T, 2, H, D), T * D + bits, dtype, 3.0)
    kv[0] *= 1e-3
    if T > 8:
        kv[1, 0] = 0.0                        # an all-zero vector: range [-1, 1]
        kv[2, :, 0] = kv[2, :, 0].abs()       # one-sided ranges
        kv[3, :, 0] = -kv[3, :, 0].abs()
        kv[4, 0, 0, 5] = float("nan")
        kv[5, 1, 0, 6] = -float("inf")
        kv[6, :, 0] = torch.finfo(dtype).smallest_normal / 64  # subnormal
        kv[7, 0, 0, :2] = torch.tensor([1.0, -1.0]) * torch.finfo(dtype).max
        kv[8] = torch.arange(D) % 16 - 7.5 if bits == 4 else torch.arange(D) % 255 - 127  # ties
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * P, generator=g)[:T].int()
    bad = [i for i in range(T) if i % 11 == 9]
    keep = np.array([i for i in range(T) if i % 11 != 9])
    for j, i in enumerate(bad):
        slots[i] = (-1, pages * P, 2147483647, -2147483648)[j % 4]
    kd = kv.to(dev)
    before = {n: t.clone() for n, t in cache.items()}
    assert gq.cache_write(kd[:, 0], kd[:, 1], cache, slots.to(dev), bits) is cache
    page, off = slots.numpy()[keep] // P, slots.numpy()[keep] % P
    for n in before:  # nothing else moved
        t, b = cache[n].clone(), before[n].clone()
        for x in (t, b):
            x[torch.from_numpy(page).long(), :, torch.from_numpy(off).long()] = 0
        assert torch.equal(t.view(torch.uint8), b.view(torch.uint8)), n
    rk, rv = gq.cache_read(cache, slots.to(dev), bits, dtype)
    for side, got, x in (("k", rk, kv[:, 0]), ("v", rv, kv[:, 1])):
        assert torch.all(got.cpu()[bad] == 0)
        got = got.cpu()[keep]
        if bits == 16:
            assert torch.equal(got.view(torch.int16), x[keep].view(torch.int16))
            continue
        c, s, z = R.quantize_vectors(_np(x)[keep], bits)
        assert np.array_equal(cache[side + "_scales"].cpu().numpy()[page, :, off], s, equal_nan=True)
        assert np.array_equal(cache[side + "_zeros"].cpu().numpy()[page, :, off], z)
        assert np.array_equal(cache[side].cpu().numpy()[page, :, off], R.pack_vector_codes(c, bits))
        val = torch.from_numpy(R.vector_values(c, s, z)).float().to(dtype)
        assert np.array_equal(_np(got), _np(val), equal_nan=True)


def test_cache_empty_calls():
    dev = device()
    cache = gq.new_cache(2, 2, 64, 16, 8)
    k = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    gq.cache_write(k, k, cache, none, 8)
    assert gq.cache_read(cache, none, 8)[0].shape == (0, 2, 64)


# ------------------------------------------------------------------ attention
def _case(have, new, H, D, P, bits, dtype, seed, kv=None, pad_rows=0, Hq=None):
    """A cache holding the sequences' keys and values in shuffled pages, all else NaN; the values as
    the cache stores them (float64), and the call's index tensors."""
    dev = device()
    g = torch.Generator().manual_seed(seed)
    need = [-(-L // P) for L in have]
    pages = sum(need) + 2
    cache = _fill(gq.new_cache(pages, H, D, P, bits, dtype), bits)
    order = torch.randperm(pages, generator=g)
    width = max(max(need), 1) + 1
    table = torch.full((len(have), width), -7, dtype=torch.int32)  # unused entries: not a page
    at, vals, slots_all, ks, vs = 0, [], [], [], []
    for s, L in enumerate(have):
        table[s, :need[s]] = order[at:at + need[s]]
        at += need[s]
        j = torch.arange(L)
        slots = table[s].long()[j // P] * P + j % P
        k, v = kv(s, L) if kv else (_randn((L, H, D), seed + 10 * s, dtype), _randn((L, H, D), seed + 10 * s + 1, dtype))
        ks.append(k)
        vs.append(v)
        slots_all.append(slots.int())
        if bits == 16:
            vals.append((_np(k), _np(v)))
        else:
            vals.append(tuple(R.vector_values(*R.quantize_vectors(_np(x), bits)) if L else _np(x) for x in (k, v)))
    gq.cache_write(torch.cat(ks).to(dev), torch.cat(vs).to(dev), cache, torch.cat(slots_all).to(dev), bits)
    starts = torch.tensor([0] + list(new)).cumsum(0).int()
    T = int(starts[-1])
    q = _randn((T + pad_rows, (Hq or H) + 1, D), seed + 5, dtype).to(dev)[:, :-1]  # a strided view
    return dict(cache=cache, table=table.to(dev), lens=torch.tensor(have, dtype=torch.int32).to(dev),
                starts=starts.to(dev), q=q, vals=vals, T=T)


def _attend(c, bits, **kw):
    return gq.paged_attention(c["q"], c["cache"], c["table"], c["lens"], c["starts"], bits=bits, **kw)


def _bound(ref, mass, size, dtype, bits, D):
    u = U[dtype]
    up = u if bits == 16 else max(u, 2.0 ** -8)
    ds = (D * 2.0 ** -24 + (u if bits < 16 else 0.0)) * size
    rel = up + (u if bits < 16 else 0.0) + 2.0 ** -20 + np.expm1(2 * ds)
    return u * np.maximum(np.abs(ref), torch.finfo(dtype).tiny) + rel[..., None] * mass


def _check_all(c, out, new, dtype, bits, D, causal=True, scale=None):
    at = 0
    for s, n in enumerate(new):
        k, v = c["vals"][s]
        ref, mass, size = R.attention(_np(c["q"][at:at + n]), k, v, causal, scale)
        got = _np(out[at:at + n])
        at += n
        err = np.abs(got - ref)
        assert np.all(err <= _bound(ref, mass, size, dtype, bits, D)), (s, float(err.max()))


# (keys, new rows) per sequence
STEP = ([700, 33, 1, 64, 65, 1300, 16, 257], [1] * 8)
GUESS = ([130, 3, 0, 40, 515], [3, 3, 2, 0, 4])  # a row that sees one key, rows that see none, no rows
CHUNK = ([300, 513, 64, 129, 77, 9], [300, 100, 64, 128, 1, 9])
LATE = ([20, 200], [50, 130])                    # more rows than keys: the first ones see nothing


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("H,group,D,P", [(2, 1, 128, 64), (2, 4, 64, 16), (1, 8, 128, 32), (1, 5, 64, 256)])
@pytest.mark.parametrize("lens", [STEP, GUESS, CHUNK, LATE], ids=["step", "guess", "chunk", "late"])
def test_attention(dtype, bits, H, group, D, P, lens):
    have, new = lens
    c = _case(have, new, H, D, P, bits, dtype, 7 + D + bits, Hq=H * group)
    _check_all(c, _attend(c, bits, max_q_len=max(new)), new, dtype, bits, D)
    assert gq.device_status() == 0


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens", [STEP, CHUNK], ids=["step", "chunk"])
def test_attention_all_keys_and_scale(bits, lens):
    have, new = lens
    c = _case(have, new, 2, 128, 32, bits, torch.bfloat16, 90 + bits, Hq=6)
    _check_all(c, _attend(c, bits, causal=False, scale=0.2), new, torch.bfloat16, bits, 128, False, 0.2)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("group,D", [(1, 128), (4, 64), (16, 128)])
@pytest.mark.parametrize("have,new", [([3001, 17, 128], [1, 1, 1]), ([2500], [1]), ([900, 333], [900, 100])])
def test_attention_counts_every_key_once(bits, group, D, have, new):
    """q = 0 and integer values: the mean of the keys seen, from exact sums."""
    dtype = torch.bfloat16
    g = torch.Generator().manual_seed(D + bits)

    def kv(s, L):
        k = _randn((L, 2, D), 50 + s, dtype)
        # 0 .. maxq with both ends in each vector: scale 1, zero 0, every code exact
        v = torch.randint(0, 16, (L, 2, D), generator=g)
        v[..., 0], v[..., 1] = 0, 15 if bits == 4 else 255
        return k, v.to(dtype)

    c = _case(have, new, 2, D, 64, bits, dtype, 11, kv=kv, Hq=2 * group)
    c["q"] = torch.zeros_like(c["q"])
    out, at = _np(_attend(c, bits, max_q_len=max(new))), 0
    for s, (L, n) in enumerate(zip(have, new)):
        v = c["vals"][s][1]
        assert np.array_equal(v, np.rint(v))
        sums = np.cumsum(v, 0)
        for i in range(n):
            m = L - n + i + 1
            ref = np.repeat(sums[m - 1] / m, group, 0)
            assert np.all(np.abs(out[at + i] - ref) <= (2.0 ** -8 + 2.0 ** -21) * np.abs(ref))
        at += n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("n", [1, 24])
def test_attention_long_context(dtype, bits, n):
    """60000 keys that weigh much the same: the answer is some 200 times smaller than the values, and
    errors that grow with the number of keys or with an offset of the codes would show.  Roundings here are
    many and independent: the 2-norm of the error is held to 4 times the quadrature sum of the relative errors'
    spreads, u / sqrt(3) of the probability, of values and keys behind codes (the scores' error is theirs times
    their spread, below 2 here), and of the output."""
    D, L, group = 128, 60001, 4
    g = torch.Generator().manual_seed(bits)

    def kv(s, L):
        return (0.7 * torch.randn(L, 1, D, generator=g)).to(dtype), torch.randn(L, 1, D, generator=g).to(dtype)

    c = _case([L], [n], 1, D, 64, bits, dtype, 3, kv=kv, Hq=group)
    out = _np(_attend(c, bits))
    k, v = c["vals"][0]
    q = _np(c["q"])
    ref = np.empty_like(q)
    for i in range(n):
        m = L - n + i + 1
        s = q[i] @ k[:m, 0].T / np.sqrt(D)
        p = np.exp(s - s.max(-1, keepdims=True))
        ref[i] = p @ v[:m, 0] / p.sum(-1, keepdims=True)
    u = U[dtype]
    up = max(u, 2.0 ** -8) if bits < 16 else u
    codes = (u * 2, u) if bits < 16 else (0.0, 0.0)
    most = 4 * np.sqrt((u ** 2 + up ** 2 + codes[0] ** 2 + codes[1] ** 2) / 3)
    assert np.linalg.norm(out - ref) <= most * np.linalg.norm(ref)


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("n", [1, 2, 200])
def test_attention_finds_the_key(bits, n):
    """A key that outweighs all others by 2^-40: the answer is its value alone."""
    D, L, H, dtype = 128, 777, 1, torch.float16
    want = [(31 * i) % (L - n + 1) for i in range(n)]

    def kv(s, L):
        return _randn((L, H, D), 1, dtype), _randn((L, H, D), 2, dtype)

    c = _case([L], [n], H, D, 16, bits, dtype, 3, kv=kv, Hq=4)
    k, v = c["vals"][0]
    c["q"] = torch.from_numpy(np.repeat(8 * k[want], 4, 1)).to(dtype).to(device())  # |k|^2 ~ 128, others ~ 11
    out = _np(_attend(c, bits))
    ref, mass, size = R.attention(_np(c["q"]), k, v)
    assert np.all(np.abs(ref - np.repeat(v[want], 4, 1)) < 1e-6)
    up = 2.0 ** -8 if bits < 16 else U[dtype]
    assert np.all(np.abs(out - ref) <= (U[dtype] + up + (U[dtype] if bits < 16 else 0)) * np.abs(ref) + 2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("have,new", [([260], [200]), ([40], [4]), ([3000], [2])])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_attention_unseen_nonfinite(dtype, bits, have, new, what):
    """Keys and values that are not finite reach the rows that see them and no others."""
    D, H, (L,), (n,) = 64, 2, have, new
    bad = L - n // 2  # seen by the later half of the rows

    def kv(s, L):
        k, v = _randn((L, H, D), 1, dtype), _randn((L, H, D), 2, dtype)
        k[bad, 0, 3] = what
        v[bad] = what
        return k, v

    c = _case(have, new, H, D, 16, bits, dtype, 3, kv=kv, Hq=4)
    out = _np(_attend(c, bits))
    first = bad - (L - n)
    ref, mass, size = _masked_reference(c, L, n, bad)
    assert np.all(np.abs(out[:first] - ref) <= _bound(ref, mass, size, dtype, bits, D))
    assert not np.isfinite(out[first:]).any()


def _masked_reference(c, L, n, bad):
    """The rows before the one at position `bad`, from the keys before it."""
    first = bad - (L - n)
    k, v = c["vals"][0]
    return R.attention(_np(c["q"][:first]), k[:bad], v[:bad])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("rows", [1, 5])
def test_attention_many_sequences_share_pages(bits, rows):
    """More sequences than threads of a CTA, of all short lengths, all over the same few pages; a group of 4, so
    that 5 rows are a chunk."""
    D, H, P, dtype, S = 64, 2, 16, torch.bfloat16, 700
    c = _case([130], [1], H, D, P, bits, dtype, 8, Hq=4 * H)
    k, v = c["vals"][0]
    g = torch.Generator().manual_seed(3)
    have = torch.randint(rows, 131, (S,), generator=g).tolist()
    new = [rows if s % 3 else 1 for s in range(S)]
    dev = device()
    c["table"] = c["table"].expand(S, -1).contiguous()
    c["lens"] = torch.tensor(have, dtype=torch.int32).to(dev)
    c["starts"] = torch.tensor([0] + new).cumsum(0).int().to(dev)
    c["q"] = _randn((sum(new), 4 * H, D), 9, dtype).to(dev)
    out, at = _np(_attend(c, bits, max_q_len=rows)), 0
    for s in range(S):
        if s < 40 or s % 29 == 0 or s > S - 20:
            ref, mass, size = R.attention(_np(c["q"][at:at + new[s]]), k[:have[s]], v[:have[s]])
            assert np.all(np.abs(out[at:at + new[s]] - ref) <= _bound(ref, mass, size, dtype, bits, D)), s
        at += new[s]
    assert np.isfinite(out).all() and gq.device_status() == 0


def test_attention_of_two_threads_at_once():
    """Calls from two host threads, each on its own stream, give the bits of calls one after another."""
    import threading

    cases = [_case([300, 513, 64], [300, 100, 1], 2, 128, 32, b, torch.bfloat16, 30 + b, Hq=8) for b in (16, 8)]
    want = [_attend(c, b) for c, b in zip(cases, (16, 8))]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got[i] = [_attend(cases[i], (16, 8)[i]) for _ in range(20)]
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20 and all(torch.equal(o, want[i]) for o in got[i])


def test_attention_padding_rows_and_empty():
    D, bits = 64, 8
    c = _case([50, 30], [2, 1], 2, D, 16, bits, torch.bfloat16, 5, pad_rows=4, Hq=4)
    out = torch.full((7, 4, D), 3.25, dtype=torch.bfloat16, device=device())
    assert _attend(c, bits, out=out) is out
    assert torch.all(out[3:] == 3.25)
    _check_all(c, out, [2, 1], torch.bfloat16, bits, D)
    e = gq.paged_attention(c["q"][:0], c["cache"], c["table"], c["lens"], c["starts"], bits)
    assert e.shape == (0, 4, D)
    n = gq.paged_attention(c["q"], c["cache"], c["table"][:0], c["lens"][:0], c["starts"][:1], bits, out=out.clone())
    assert torch.equal(n, out)
    # lengths and pages outside the table and the cache stay inside it
    wild = gq.paged_attention(c["q"], c["cache"], torch.full_like(c["table"], 1 << 30), c["lens"] + (1 << 30), c["starts"],
                              bits)
    torch.cuda.synchronize()
    assert wild.shape == c["q"].shape


@pytest.mark.parametrize("lens", [STEP, CHUNK], ids=["step", "chunk"])
def test_attention_same_bits_again_on_streams_and_in_a_graph(lens):
    have, new = lens
    c = _case(have, new, 2, 128, 64, 8, torch.bfloat16, 21, Hq=8)
    a = _attend(c, 8, max_q_len=max(new))
    side = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [_attend(c, 8, max_q_len=max(new), stream=s) for s in side for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for o in outs)
    out = torch.zeros_like(a)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(a)
    with torch.cuda.graph(g1):
        _attend(c, 8, max_q_len=max(new), out=out)
    with torch.cuda.graph(g2):
        _attend(c, 8, max_q_len=max(new), out=out2)
    for _ in range(3):
        with torch.cuda.stream(side[0]):
            g1.replay()
        with torch.cuda.stream(side[1]):
            g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, out) and torch.equal(a, out2)
    # a replay reads the lengths of its time
    c["lens"].copy_(torch.tensor([max(n, L - 1) for L, n in zip(have, new)], dtype=torch.int32))
    g1.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _attend(c, 8, max_q_len=max(new)))
