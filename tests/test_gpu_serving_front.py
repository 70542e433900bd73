"""The serving wrappers' way into the library: the native front, and the Python path that takes over where it does
not."""

import pytest
import torch

import post_weight_quantization_layer_b200 as gq
from tests.gpu_util import device

pytestmark = pytest.mark.gpu


def _call():
    """Arguments of a small attention call over an 8-bit cache, and of its cache calls."""
    dev = device()
    g = torch.Generator().manual_seed(1)
    cache = gq.new_cache(4, 2, 64, 16, 8)
    kv = torch.randn(40, 2, 64, generator=g).bfloat16().to(dev)
    slots = torch.arange(40, dtype=torch.int32, device=dev)
    gq.cache_write(kv, kv, cache, slots, 8)
    q = torch.randn(3, 4, 64, generator=g).bfloat16().to(dev)
    ints = [torch.tensor(x, dtype=torch.int32, device=dev) for x in ([[0, 1, 2]], [40], [0, 3])]
    return cache, kv, slots, q, ints


@pytest.mark.parametrize("bits", [2 ** 63, 2 ** 64 + 8, -2 ** 70, 5])
def test_bits_of_any_size_are_refused_as_such(bits):
    cache, kv, slots, q, ints = _call()
    for call in (lambda: gq.cache_write(kv, kv, cache, slots, bits), lambda: gq.cache_read(cache, slots, bits),
                 lambda: gq.paged_attention(q, cache, *ints, bits=bits)):
        with pytest.raises(ValueError, match="bits must be"):
            call()


def test_max_q_len_of_any_size():
    cache, kv, slots, q, ints = _call()
    want = gq.paged_attention(q, cache, *ints, bits=8)
    for most in (3, 40, 2 ** 62, 2 ** 63, 2 ** 64, 2 ** 80):
        assert torch.equal(gq.paged_attention(q, cache, *ints, bits=8, max_q_len=most), want)
        assert torch.equal(gq.paged_attention(q, cache, *ints, bits=8, max_q_len=most, out=torch.empty_like(q)), want)
    for most in (-1, -2 ** 64, 1.5):
        with pytest.raises(ValueError, match="max_q_len"):
            gq.paged_attention(q, cache, *ints, bits=8, max_q_len=most)
