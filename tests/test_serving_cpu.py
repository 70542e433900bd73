"""Refusals of the serving operators (C ABI and Python binding), the rotary frequencies (host code)
and pins of the oracle, without a GPU.  Only calls that are rejected, or that have no work, reach the library:
pointers are fake and never read."""

import ctypes
import math

import numpy as np
import pytest
import torch

import post_weight_quantization_layer_b200 as gq
from oracle import serving_ref as R
from post_weight_quantization_layer_b200 import _native
from post_weight_quantization_layer_b200.build import build

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE, ODD = 0x10000, 0x10004


@pytest.fixture(scope="module")
def L():
    build()
    return _native.lib()


def _rotary(L, **kw):
    a = dict(q=FAKE, k=FAKE, dtype=2, tokens=4, heads=8, kv_heads=2, d=128, r=128, inter=0, qt=1024, qh=128, kt=256, kh=128,
             pos=FAKE, freq=FAKE, factor=1.0, qo=2 * FAKE, ko=2 * FAKE, qot=1024, qoh=128, kot=256, koh=128, stream=None)
    a.update(kw)
    return L.gptq_rotary(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(pos=None), INVALID), (dict(freq=None), INVALID),
    (dict(qo=None), INVALID), (dict(ko=None), INVALID), (dict(dtype=0), INVALID), (dict(dtype=9), INVALID),
    (dict(tokens=-1), INVALID), (dict(heads=0), INVALID), (dict(kv_heads=-1), INVALID), (dict(r=0), INVALID),
    (dict(r=7), INVALID), (dict(r=130), INVALID), (dict(d=0), INVALID), (dict(d=132, r=4), UNSUPPORTED),
    (dict(d=520, r=4), UNSUPPORTED), (dict(qt=1028), UNSUPPORTED), (dict(kh=4), UNSUPPORTED), (dict(q=ODD), UNSUPPORTED),
    (dict(ko=ODD), UNSUPPORTED), (dict(qoh=2), UNSUPPORTED), (dict(qo=FAKE, qot=2048), INVALID),
    (dict(ko=FAKE, koh=256), INVALID), (dict(tokens=0), OK), (dict(tokens=0, q=None, qo=None, k=None, ko=None, pos=None), OK)])
def test_rotary_rejections(L, kw, status):
    assert _rotary(L, **kw) == status


def _write(L, **kw):
    a = dict(k=FAKE, v=FAKE, dtype=2, tokens=4, heads=2, d=128, kt=256, kh=128, vt=256, vh=128, kc=FAKE, vc=FAKE, ks=FAKE,
             kz=FAKE, vs=FAKE, vz=FAKE, bits=8, pages=4, page=64, slots=FAKE, stream=None)
    a.update(kw)
    return L.gptq_cache_write(*a.values())


CACHE = [(dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(vz=None), INVALID),
         (dict(bits=2), INVALID), (dict(bits=3), INVALID), (dict(bits=0), INVALID), (dict(pages=0), INVALID),
         (dict(page=0), INVALID), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=512), UNSUPPORTED),
         (dict(pages=1 << 26), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(d=0), INVALID),
         (dict(dtype=0), INVALID), (dict(heads=0), INVALID), (dict(kc=ODD), UNSUPPORTED), (dict(vs=ODD), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(k=None), INVALID), (dict(slots=None), INVALID), (dict(tokens=-1), INVALID), (dict(kt=100), UNSUPPORTED),
    (dict(vh=4), UNSUPPORTED), (dict(v=ODD), UNSUPPORTED), (dict(tokens=0), OK),
    (dict(tokens=0, bits=16, ks=None, kz=None, vs=None, vz=None), OK), (dict(tokens=0, k=None, v=None, slots=None), OK)])
def test_cache_write_rejections(L, kw, status):
    assert _write(L, **kw) == status


def _read(L, **kw):
    a = dict(kc=FAKE, vc=FAKE, ks=FAKE, kz=FAKE, vs=FAKE, vz=FAKE, bits=8, pages=4, page=64, slots=FAKE, count=3, heads=2,
             d=128, dtype=1, k=FAKE, v=FAKE, stream=None)
    a.update(kw)
    return L.gptq_cache_read(*a.values())


@pytest.mark.parametrize("kw,status", CACHE + [(dict(k=None), INVALID), (dict(count=-1), INVALID), (dict(v=ODD), UNSUPPORTED),
                                               (dict(slots=None), INVALID), (dict(count=0), OK)])
def test_cache_read_rejections(L, kw, status):
    assert _read(L, **kw) == status


def _attend(L, **kw):
    a = dict(q=FAKE, dtype=2, tokens=4, q_heads=8, heads=2, d=128, qt=1024, qh=128, kc=FAKE, vc=FAKE, ks=FAKE, kz=FAKE,
             vs=FAKE, vz=FAKE, bits=8, pages=4, page=64, table=FAKE, width=4, lens=FAKE, starts=FAKE, seqs=2, max_q=4,
             causal=1, scale=0.1, out=2 * FAKE, stream=None)
    a.update(kw)
    return L.gptq_paged_attention(*a.values())


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=FAKE), INVALID), (dict(table=None), INVALID), (dict(lens=None), INVALID),
    (dict(starts=None), INVALID), (dict(tokens=-1), INVALID), (dict(seqs=-1), INVALID), (dict(q_heads=0), INVALID),
    (dict(q_heads=9), INVALID), (dict(width=0), INVALID), (dict(max_q=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID),
    (dict(q_heads=130), UNSUPPORTED), (dict(qt=1025), UNSUPPORTED), (dict(q=ODD), UNSUPPORTED), (dict(out=ODD), UNSUPPORTED),
    (dict(seqs=1 << 21), UNSUPPORTED), (dict(width=1 << 25), UNSUPPORTED), (dict(width=1 << 28), UNSUPPORTED), (dict(tokens=0), OK), (dict(seqs=0, table=None, lens=None), OK), (dict(max_q=0), OK)])
def test_attention_rejections(L, kw, status):
    assert _attend(L, **kw) == status


@pytest.mark.parametrize("r", [64, 128, 20, 6])
@pytest.mark.parametrize("scaling,factor,original", [(None, 1.0, 0), ("linear", 4.0, 0), ("ntk", 8.0, 0), ("yarn", 32.0, 4096),
                                                     ("yarn", 1.0, 128)])
def test_rotary_frequencies(L, r, scaling, factor, original):
    f, a = gq.rotary_frequencies(r, 10000.0, scaling, factor, original, device="cpu")
    ref, ra = R.rotary_frequencies(r, 10000.0, scaling, factor, original)
    assert f.dtype == torch.float64 and np.allclose(f.numpy(), ref, rtol=1e-14) and abs(a - ra) <= 2.0 ** -24 * ra
    if scaling == "ntk":  # the slowest pair is slowed by the factor, the fastest kept
        plain, _ = R.rotary_frequencies(r)
        assert f[0] == 1.0 and abs(f[-1] * factor / plain[-1] - 1) < 1e-12


@pytest.mark.parametrize("kw", [dict(base=1.0), dict(base=math.inf), dict(scaling="linear", factor=0.5),
                                dict(scaling="linear", factor=math.nan), dict(scaling="yarn", factor=2.0),
                                dict(scaling="yarn", factor=2.0, original_len=64, beta_fast=1.0, beta_slow=1.0),
                                dict(scaling="other")])
def test_rotary_frequencies_rejections(L, kw):
    with pytest.raises((ValueError, gq.GPTQError)):
        gq.rotary_frequencies(64, device="cpu", **kw)
    with pytest.raises(ValueError):
        gq.rotary_frequencies(7, device="cpu")
    with pytest.raises(gq.GPTQError):
        gq.rotary_frequencies(2, scaling="ntk", factor=2.0, device="cpu")


def test_oracle_quantizer_keeps_the_nearest_code():
    """Against a search over all codes, and the scale's ends."""
    rng = np.random.default_rng(0)
    for bits in (4, 8):
        x = rng.normal(size=(40, 64)) * np.exp(rng.normal(size=(40, 1)) * 3)
        x = x.astype(np.float16).astype(np.float64)
        c, s, z = R.quantize_vectors(x, bits)
        every = s[:, None, None].astype(np.float64) * (np.arange(2 ** bits)[None, None] - z[:, None, None].astype(np.float64))
        best = np.abs(x[..., None] - every).min(-1)
        got = np.abs(x - s[:, None].astype(np.float64) * (c.astype(np.float64) - z[:, None]))
        assert np.all(got <= best + 1e-12 * np.abs(x))
        assert np.array_equal(R.unpack_vector_codes(R.pack_vector_codes(c, bits), bits), c)


def test_oracle_quantizer_by_hand():
    """Worked cases: no value, one sign, both signs with ties, not finite."""
    x = np.array([[0.0, 0, 0, 0], [15, 0, 7.5, 6.5], [-15, 0, -7.5, -1], [-5, 10, 0.5, 1.5], [math.inf, 1, 2, 3],
                  [math.nan, 1, 2, 3], [3e38, -3e38, 0, 1]])
    c, s, z = R.quantize_vectors(x, 4)
    two = np.float32(2.0) / np.float32(15.0)  # no value: from -1 to 1, the zero near 7.5
    assert s[0] == two and z[0] == round(1.0 / float(two)) and np.all(c[0] == z[0])
    assert s[1] == 1 and z[1] == 0 and c[1].tolist() == [15, 0, 8, 6]        # 7.5 -> 8, 6.5 -> 6: half to even
    assert s[2] == 1 and z[2] == 15 and c[2].tolist() == [0, 15, 7, 14]      # 15 - 8
    assert s[3] == 1 and z[3] == 5 and c[3].tolist() == [0, 15, 5, 7]        # 0.5 -> 0, 1.5 -> 2
    assert np.all(np.isnan(s[4:])) and not c[4:].any() and not z[4:].any()   # the last: its range is past float32
    assert R.pack_vector_codes(c[1:2], 4).tolist() == [[15, 8 | 6 << 4]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation(interleaved):
    """Position 0 changes nothing, lengths stay, products depend on the distance alone, the rest of the head stays;
    the first pair's angle is the position."""
    rng = np.random.default_rng(1)
    f, _ = R.rotary_frequencies(16)
    x, y = rng.normal(size=(2, 5, 3, 24))
    pos = np.array([0, 1, 7, 100, 4000])
    a, b = R.rotary(x, pos, f, 1.0, interleaved), R.rotary(y, pos + 3, f, 1.0, interleaved)
    assert np.array_equal(a[0], x[0]) and np.array_equal(a[..., 16:], x[..., 16:])
    assert np.allclose(np.linalg.norm(a, axis=-1), np.linalg.norm(x, axis=-1), rtol=1e-13)
    a2, b2 = R.rotary(x, pos + 50, f, 1.0, interleaved), R.rotary(y, pos + 53, f, 1.0, interleaved)
    assert np.allclose((a * b).sum(-1), (a2 * b2).sum(-1), rtol=0, atol=1e-10)
    e = np.zeros((1, 1, 16))
    e[..., 0] = 1.0
    turned = R.rotary(e, [2], f, 1.0, interleaved)[0, 0]
    assert math.isclose(turned[0], math.cos(2.0)) and math.isclose(turned[1 if interleaved else 8], math.sin(2.0))


def test_oracle_attention():
    """Equal keys: the mean of what each row sees; one key: its value; a chunk at a time is the whole prompt; rows
    before the sequence's start see nothing."""
    rng = np.random.default_rng(2)
    q, v = rng.normal(size=(6, 4, 8)), rng.normal(size=(6, 2, 8))
    out = R.attention(q, np.ones((6, 2, 8)), v)[0]
    mean = np.cumsum(v, 0) / np.arange(1, 7)[:, None, None]
    assert np.allclose(out, np.repeat(mean, 2, 1), atol=1e-13)
    k = rng.normal(size=(6, 2, 8))
    whole = R.attention(q, k, v)[0]
    assert np.allclose(whole[0], np.repeat(v[0], 2, 0), atol=1e-15)
    parts = [R.attention(q[i:j], k[:j], v[:j])[0] for i, j in ((0, 1), (1, 4), (4, 6))]
    assert np.allclose(np.concatenate(parts), whole, atol=1e-14)
    few = R.attention(q, k[:2], v[:2])[0]
    assert not few[:4].any() and np.allclose(few[4], np.repeat(v[0], 2, 0), atol=1e-15)
    full = R.attention(q, k, v, causal=False)[0]
    assert np.allclose(full[5], whole[5], atol=1e-15) and not np.allclose(full[0], whole[0])


# ------------------------------------------------------------------ the binding's own checks
BF = torch.bfloat16


def _cpu_cache(bits=8, D=64, P=16):
    return gq.new_cache(3, 2, D, P, bits, BF, device="cpu")


def test_binding_rejections(L):
    x = torch.zeros(5, 4, 64, dtype=BF)
    kv = torch.zeros(5, 2, 64, dtype=BF)
    i5 = torch.zeros(5, dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    table, lens, starts = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    bad = [
        lambda: gq.rotary(x[0], None, i5, f), lambda: gq.rotary(x.float(), None, i5, f),
        lambda: gq.rotary(x, kv.half(), i5, f), lambda: gq.rotary(x, kv[:3], i5, f), lambda: gq.rotary(x, kv[..., :32], i5, f),
        lambda: gq.rotary(x, kv, i5.long(), f), lambda: gq.rotary(x, kv, i5[:4], f), lambda: gq.rotary(x, kv, i5, f.float()),
        lambda: gq.rotary(x.transpose(1, 2), None, i5, f), lambda: gq.rotary(x, kv, i5, f),  # CPU tensors
        lambda: gq.cache_write(kv, kv.half(), _cpu_cache(), i5, 8), lambda: gq.cache_write(kv, kv[:4], _cpu_cache(), i5, 8),
        lambda: gq.cache_write(kv, kv, _cpu_cache(), i5.long(), 8), lambda: gq.cache_write(kv, kv, _cpu_cache(), i5, 5),
        lambda: gq.cache_write(kv, kv, _cpu_cache(16), i5, 8), lambda: gq.cache_write(kv, kv, _cpu_cache(8), i5, 16),
        lambda: gq.cache_write(kv, kv, _cpu_cache(8), i5, 4), lambda: gq.cache_write(x, x, _cpu_cache(), i5, 8),
        lambda: gq.cache_write(kv, kv, {"k": kv}, i5, 8), lambda: gq.cache_write(kv, kv, None, i5, 8),
        lambda: gq.cache_write(kv.half(), kv.half(), _cpu_cache(16), i5, 16),
        lambda: gq.cache_write(kv, kv, dict(_cpu_cache(), v_zeros=i5), i5, 8),
        lambda: gq.cache_read(_cpu_cache(), i5.float(), 8), lambda: gq.cache_read(_cpu_cache(), i5, 8, torch.float32),
        lambda: gq.cache_read(_cpu_cache(16), i5, 16, torch.float16), lambda: gq.cache_read(_cpu_cache(), i5, 8),
        lambda: gq.paged_attention(torch.zeros(5, 3, 64, dtype=BF), _cpu_cache(), table, lens, starts, 8),
        lambda: gq.paged_attention(x, _cpu_cache(), table[0], lens, starts, 8),
        lambda: gq.paged_attention(x, _cpu_cache(), table, lens, lens, 8),
        lambda: gq.paged_attention(x, _cpu_cache(), table.long(), lens, starts, 8),
        lambda: gq.paged_attention(x, _cpu_cache(D=128), table, lens, starts, 8),
        lambda: gq.new_cache(1, 1, 64, bits=3, device="cpu"), lambda: gq.new_cache(1, 1, 64, dtype=torch.float32, device="cpu"),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")


def test_step_batch():
    from post_weight_quantization_layer_b200 import serving

    b = serving.step_batch([[5, 2], [7], []], [15, 3, 0], [2, 1, 0], 16, device="cpu", width=3)
    assert b.positions.tolist() == [15, 16, 3] and b.slots.tolist() == [95, 32, 115]
    assert b.page_table.tolist() == [[5, 2, 0], [7, 0, 0], [0, 0, 0]]
    assert b.kv_lens.tolist() == [17, 4, 0] and b.q_starts.tolist() == [0, 2, 3, 3] and b.max_q_len == 2
    assert all(t.dtype == torch.int32 for t in (b.positions, b.slots, b.page_table, b.kv_lens, b.q_starts))
    for bad in (([[5]], [15], [2]), ([[5]], [-1], [1]), ([[5]], [0], [1, 1])):
        with pytest.raises(ValueError):
            serving.step_batch(*bad, 16, device="cpu")
    with pytest.raises(ValueError):
        serving.step_batch([[5, 2]], [0], [1], 16, device="cpu", width=1)
    empty = serving.step_batch([], [], [], 16, device="cpu")
    assert empty.page_table.shape == (0, 1) and empty.q_starts.tolist() == [0] and empty.max_q_len == 0
