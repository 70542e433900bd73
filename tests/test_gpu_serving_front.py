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


SLOW = """
#include <unistd.h>
extern "C" {
int gptq_rotary() { usleep(400000); return 0; }
int gptq_cache_write() { usleep(400000); return 0; }
int gptq_cache_read() { usleep(400000); return 0; }
int gptq_paged_attention() { usleep(400000); return 0; }
}
"""


def test_threads_call_at_once(tmp_path):
    """A second copy of the front, on a library whose calls take 0.4 s: those of four threads overlap."""
    import importlib.util
    import shutil
    import subprocess
    import threading
    import time

    from post_weight_quantization_layer_b200 import _native

    (tmp_path / "slow.cpp").write_text(SLOW)
    subprocess.run(["g++", "-shared", "-fPIC", str(tmp_path / "slow.cpp"), "-o", str(tmp_path / "slow.so")], check=True)
    copy = shutil.copy(_native.BINDING_PATH, tmp_path / "_binding.so")
    spec = importlib.util.spec_from_file_location("_binding", copy)
    front = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(front)
    front.open(str(tmp_path / "slow.so"))
    cache, kv, slots, q, ints = _call()
    six = [cache[n] for n in ("k", "v", "k_scales", "k_zeros", "v_scales", "v_zeros")]
    f, _ = gq.rotary_frequencies(64)
    calls = [lambda: front.rotary(kv, None, slots, f, 1.0, False), lambda: front.cache_write(kv, kv, *six, slots, 8),
             lambda: front.cache_read(*six, slots, 8, False),
             lambda: front.paged_attention(q, *six, *ints, 8, None, True, None)]
    got = [None] * 4

    def work(i):
        got[i] = calls[i]()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    start = time.monotonic()
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert time.monotonic() - start < 0.9  # one after another: 1.6
    assert all(r is not None for r in got)


def test_the_same_without_the_front(monkeypatch):
    """Every call through ctypes gives the bits of the native front."""
    from post_weight_quantization_layer_b200 import _native

    cache, kv, slots, q, ints = _call()
    pos, (f, a) = slots % 7, gq.rotary_frequencies(64)

    def run():
        fresh = gq.new_cache(4, 2, 64, 16, 8)
        gq.cache_write(kv, kv, fresh, slots, 8)
        return [*gq.rotary(kv, kv[:, :1], pos, f, a), *gq.cache_read(fresh, slots, 8), *fresh.values(),
                gq.paged_attention(q, fresh, *ints, bits=8)]

    want = run()
    monkeypatch.setattr(_native, "_front", _native._NoFront)
    got = run()
    assert len(want) == len(got) and all(torch.equal(x, y) for x, y in zip(want, got))
