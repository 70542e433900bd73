"""Answer with a quantized decoder layer: one step of a batch over a paged key/value cache.

A step brings new tokens of several sequences (the whole prompt, a chunk of it, or one token each, mixed
as they come) through the layer that ``sequential.py`` quantizes: rmsnorm, the q, k and v linears on their
checkpoints, rotary positions, the new keys and values written to the cache, attention over everything the
cache holds of each sequence, the o linear, and the gated MLP.  Heads may share keys and values (kv_heads <
heads).  Every step runs in the native library; this module lays out the batch's index tensors and
sequences the calls.
"""

from __future__ import annotations

from dataclasses import dataclass

import torch

from . import api, kvcache


@dataclass
class StepBatch:
    """Index tensors of one step (int32, on the device)."""

    positions: torch.Tensor   # [tokens] position of each new token in its sequence
    slots: torch.Tensor       # [tokens] cache slot that it goes to
    page_table: torch.Tensor  # [seqs, width]
    kv_lens: torch.Tensor     # [seqs] keys of each sequence, the new tokens included
    q_starts: torch.Tensor    # [seqs + 1] first row of each sequence
    max_q_len: int


def step_batch(pages, have, new, page_size, device=None, width=None) -> StepBatch:
    """The index tensors of a step in which sequence s, with have[s] tokens in the cache, brings new[s] more.

    pages: per sequence the list of its pages, enough for have[s] + new[s] tokens; width: of the page table
    (default: the longest list)."""
    if not (len(pages) == len(have) == len(new)):
        raise ValueError("pages, have and new need one entry per sequence")
    for s, (p, a, n) in enumerate(zip(pages, have, new)):
        if a < 0 or n < 0 or len(p) * page_size < a + n:
            raise ValueError(f"sequence {s}: {len(p)} pages of {page_size} do not hold {a} + {n} tokens")
    width = max([1, *(len(p) for p in pages)]) if width is None else width
    if width < 1 or any(len(p) > width for p in pages):
        raise ValueError("width is less than 1 or than a sequence's number of pages")
    positions, slots, starts = [], [], [0]
    for p, a, n in zip(pages, have, new):
        positions += range(a, a + n)
        slots += [p[i // page_size] * page_size + i % page_size for i in range(a, a + n)]
        starts.append(starts[-1] + n)
    device = device if device is not None else torch.device("cuda", torch.cuda.current_device())

    def ints(x):
        return torch.tensor(x, dtype=torch.int32).to(device)

    return StepBatch(ints(positions), ints(slots), ints([list(p) + [0] * (width - len(p)) for p in pages]).view(-1, width),
                     ints([a + n for a, n in zip(have, new)]), ints(starts), max([0, *new]))


@dataclass
class ServedLayer:
    """A quantized decoder layer as it answers."""

    checkpoints: dict            # {q, k, v, o, gate, up, down: checkpoint tensors (export.export_layer)}
    gammas: tuple                # (attention-norm weight, MLP-norm weight)
    heads: int
    kv_heads: int
    inv_freq: torch.Tensor       # kvcache.rotary_frequencies
    attention_factor: float = 1.0
    interleaved: bool = False
    bits: int = 4                # of the weights
    cache_bits: int = 16
    eps: float = 1e-5


def decoder_layer_step(h, layer: ServedLayer, cache, batch: StepBatch, stream=None, seen=None):
    """New tokens' hidden states h [tokens, hidden] through the layer; the cache (kvcache.new_cache) takes
    their keys and values.  seen: optional dict that receives the intermediate activations.  Returns the
    layer's output [tokens, hidden]; a step without tokens has none and leaves the cache as it is."""
    T, H, HK = h.shape[0], layer.heads, layer.kv_heads
    if T == 0:
        return torch.empty_like(h)
    stream = stream or torch.cuda.current_stream()

    def lin(x, name):
        return api.quantized_linear(x, layer.checkpoints[name], layer.bits, stream=stream)

    with torch.cuda.stream(stream):
        x = api.rmsnorm(h, layer.gammas[0], layer.eps, stream=stream)
        q, k, v = lin(x, "q").view(T, H, -1), lin(x, "k").view(T, HK, -1), lin(x, "v").view(T, HK, -1)
        if seen is not None:
            seen.update(x=x, q0=q.clone(), k0=k.clone(), v=v)
        kvcache.rotary(q, k, batch.positions, layer.inv_freq, layer.attention_factor, layer.interleaved, out=(q, k),
                       stream=stream)
        kvcache.cache_write(k, v, cache, batch.slots, layer.cache_bits, stream=stream)
        a = kvcache.paged_attention(q, cache, batch.page_table, batch.kv_lens, batch.q_starts, layer.cache_bits,
                                    batch.max_q_len, stream=stream).view(T, -1)
        h1 = api.add(h, lin(a, "o"), stream=stream)
        y = api.rmsnorm(h1, layer.gammas[1], layer.eps, stream=stream)
        m = api.silu_mul(lin(y, "gate"), lin(y, "up"), stream=stream)
        out = api.add(h1, lin(m, "down"), stream=stream)
        if seen is not None:
            seen.update(q=q, k=k, a=a, h1=h1, y=y, m=m)
    return out
