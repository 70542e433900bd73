"""A quantized layer answering over a paged cache: prompts in chunks, then single tokens, the run that the
serving operators are for.

Every step's rotary, cache and attention are held to the float64 oracle on the step's own inputs (the
bounds of test_gpu_serving: each operator's roundings, nothing carried over from step to step), with the
oracle keeping the history of what the cache holds of every sequence; the pieces around them are the
library's own calls on the same inputs, which give the same bits again.
"""

import numpy as np
import pytest
import torch

import oracle as O
import post_weight_quantization_layer_b200 as gq
from oracle import serving_ref as R
from post_weight_quantization_layer_b200 import api, serving, synth
from tests.gpu_util import device
from tests.test_gpu_serving import _bound, _np, _rotary_check

pytestmark = pytest.mark.gpu

HIDDEN, INTER, D = 256, 384, 64


def _checkpoint(n_out, n_in, seed):
    codes, zeros, scales, g_idx = synth.checkpoint_parts(n_out, n_in, 4, 64, seed, False, (0.004, 0.02))
    S16, qz = O.export_tensors(scales.float().numpy(), zeros.numpy(), 4)
    dev = device()
    return {"qweight": torch.from_numpy(O.pack(codes.numpy(), 4)).to(dev), "qzeros": torch.from_numpy(qz).to(dev),
            "scales": torch.from_numpy(S16).to(dev), "g_idx": g_idx.to(dev)}


def _layer(heads, kv_heads, dtype, cache_bits):
    shapes = {"q": (heads * D, HIDDEN), "k": (kv_heads * D, HIDDEN), "v": (kv_heads * D, HIDDEN), "o": (HIDDEN, heads * D),
              "gate": (INTER, HIDDEN), "up": (INTER, HIDDEN), "down": (HIDDEN, INTER)}
    g = torch.Generator().manual_seed(4)
    gam = tuple((1 + 0.1 * torch.randn(HIDDEN, generator=g)).to(dtype).to(device()) for _ in range(2))
    f, a = gq.rotary_frequencies(D, scaling="yarn", factor=4.0, original_len=64)
    return serving.ServedLayer({n: _checkpoint(*s, i) for i, (n, s) in enumerate(shapes.items())}, gam, heads, kv_heads, f, a,
                               cache_bits=cache_bits)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("heads,kv_heads,cache_bits,page", [(4, 4, 16, 16), (4, 2, 8, 32), (8, 1, 4, 16)])
def test_chunks_then_single_tokens(dtype, heads, kv_heads, cache_bits, page):
    layer = _layer(heads, kv_heads, dtype, cache_bits)
    cache = gq.new_cache(24, kv_heads, D, page, cache_bits, dtype)
    g = torch.Generator().manual_seed(9)
    order = torch.randperm(24, generator=g).tolist()
    pages = [order[:8], order[8:15], order[15:24]]
    steps = [[70, 33, 0], [40, 1, 100], [1, 1, 1], [0, 1, 1], [3, 2, 1]]  # new tokens per sequence
    have, past = [0, 0, 0], [(np.zeros((0, kv_heads, D)),) * 2 for _ in range(3)]
    for new in steps:
        batch = serving.step_batch(pages, have, new, page, width=10)
        T = sum(new)
        h = (torch.randn(T, HIDDEN, generator=g)).to(dtype).to(device())
        seen = {}
        out = serving.decoder_layer_step(h, layer, cache, batch, seen=seen)
        assert out.shape == h.shape and torch.isfinite(out.float()).all()
        pos = batch.positions
        for name in ("q", "k"):
            _rotary_check(seen[name], seen[name + "0"], pos, layer.inv_freq, layer.attention_factor, False, dtype)
        at = 0
        for s, n in enumerate(new):
            kv = []
            for x, old in zip((seen["k"], seen["v"]), past[s]):
                x = _np(x[at:at + n])
                if cache_bits < 16 and n:
                    x = R.vector_values(*R.quantize_vectors(x, cache_bits))
                kv.append(np.concatenate([old, x]))
            past[s] = tuple(kv)
            if n:
                ref, mass, size = R.attention(_np(seen["q"][at:at + n]), *kv)
                got = _np(seen["a"].view(T, heads, D)[at:at + n])
                assert np.all(np.abs(got - ref) <= _bound(ref, mass, size, dtype, cache_bits, D))
            at += n
            have[s] += n
        ck = layer.checkpoints
        assert torch.equal(seen["x"], api.rmsnorm(h, layer.gammas[0]))
        assert torch.equal(seen["h1"], api.add(h, api.quantized_linear(seen["a"], ck["o"])))
        assert torch.equal(out, api.add(seen["h1"], api.quantized_linear(seen["m"], ck["down"])))
    assert gq.device_status() == 0


def test_a_step_replays_from_a_graph():
    """A captured single-token step, replayed while its index tensors move on, answers as the calls do."""
    dtype, heads, kv_heads, page = torch.bfloat16, 4, 2, 16
    layer = _layer(heads, kv_heads, dtype, 8)
    dev = device()
    g = torch.Generator().manual_seed(1)
    prompt, hs = torch.randn(20, HIDDEN, generator=g).to(dtype).to(dev), torch.randn(4, 1, HIDDEN, generator=g).to(dtype).to(dev)

    def run(replay):
        cache = gq.new_cache(3, kv_heads, D, page, 8, dtype)
        serving.decoder_layer_step(prompt, layer, cache, serving.step_batch([[2, 0]], [0], [20], page), )
        outs, graph, h, batch = [], None, torch.empty(1, HIDDEN, dtype=dtype, device=dev), None
        for i in range(4):
            b = serving.step_batch([[2, 0]], [20 + i], [1], page)
            if not replay:
                outs.append(serving.decoder_layer_step(hs[i], layer, cache, b))
                continue
            h.copy_(hs[i])
            if graph is None:
                batch, graph = b, torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    out = serving.decoder_layer_step(h, layer, cache, batch)
            for name in ("positions", "slots", "page_table", "kv_lens", "q_starts"):
                getattr(batch, name).copy_(getattr(b, name))
            graph.replay()
            outs.append(out.clone())
        torch.cuda.synchronize()
        return outs

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)
