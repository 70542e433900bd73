"""Cases of the operators that serve a quantized layer from a key/value cache, with their plain forms.

rotary     rotary positions on the queries and keys of a step's tokens
write      keys and values stored into a paged cache (16, 8 or 4 bits) and read back as the values they stand for
read       stored keys and values of a list of slots
attention  a chunk of new tokens of each sequence over its paged cache

Head shapes are those of the configurations of this repository: 12 heads of 64 (OPT-125m), 32 heads of 128
(Llama-2-7B) and 64 heads of 128 over 8 key/value heads (Llama-2-70B).
"""

import math

import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16}


def listed():
    return [
        # one step of 8 users of a 7B-shaped layer: latency
        {"name": "rotary_step", "op": "rotary", "tokens": 8, "heads": 32, "kv_heads": 32, "head_dim": 128,
         "rotary_dim": 128, "interleaved": False, "factor": 1.0, "far": 4096, "dtype": "bfloat16"},
        # a ragged chunk, part of the head, neighbouring pairs, halves
        {"name": "rotary_part", "op": "rotary", "tokens": 1111, "heads": 12, "kv_heads": 12, "head_dim": 64,
         "rotary_dim": 32, "interleaved": True, "factor": 1.0, "far": 2048, "dtype": "float16"},
        # a long prompt of a 70B-shaped layer with frequencies scaled for 32 times its length
        {"name": "rotary_prompt", "op": "rotary", "tokens": 16384, "heads": 64, "kv_heads": 8, "head_dim": 128,
         "rotary_dim": 128, "interleaved": False, "factor": 32.0, "far": 131072, "dtype": "bfloat16"},
        # one token of each of 64 users into 8-bit pages
        {"name": "write_step_8", "op": "write", "tokens": 64, "kv_heads": 8, "head_dim": 128, "page": 64, "bits": 8,
         "dtype": "bfloat16"},
        # a long prompt of a 7B-shaped layer into 4-bit pages
        {"name": "write_prompt_4", "op": "write", "tokens": 8192, "kv_heads": 32, "head_dim": 128, "page": 32,
         "bits": 4, "dtype": "bfloat16"},
        # a cached prefix taken out of 8-bit pages
        {"name": "read_prefix_8", "op": "read", "tokens": 5003, "kv_heads": 32, "head_dim": 128, "page": 16,
         "bits": 8, "dtype": "float16"},
        # the next token of one user, 7B-shaped, unquantized cache: latency
        {"name": "decode_one", "op": "attention", "seqs": 1, "ctx": 2500, "chunk": 1, "heads": 32, "kv_heads": 32,
         "head_dim": 128, "page": 64, "bits": 16, "dtype": "bfloat16", "ragged": False, "causal": True},
        # the next token of 64 users of all lengths, 70B-shaped, 8-bit cache
        {"name": "decode_many_8", "op": "attention", "seqs": 64, "ctx": 8192, "chunk": 1, "heads": 64, "kv_heads": 8,
         "head_dim": 128, "page": 64, "bits": 8, "dtype": "bfloat16", "ragged": True, "causal": True},
        # the next token of four users with very long contexts, 4-bit cache
        {"name": "decode_long_4", "op": "attention", "seqs": 4, "ctx": 131072, "chunk": 1, "heads": 64, "kv_heads": 8,
         "head_dim": 128, "page": 128, "bits": 4, "dtype": "bfloat16", "ragged": False, "causal": True},
        # prompts of a 7B-shaped layer, their own keys and no others
        {"name": "prompt_16", "op": "attention", "seqs": 4, "ctx": 2048, "chunk": 2048, "heads": 32, "kv_heads": 32,
         "head_dim": 128, "page": 64, "bits": 16, "dtype": "bfloat16", "ragged": False, "causal": True},
        # a chunk of a long prompt, 70B-shaped, over what earlier chunks cached in 8 bits
        {"name": "chunk_long_8", "op": "attention", "seqs": 1, "ctx": 16384, "chunk": 1024, "heads": 64,
         "kv_heads": 8, "head_dim": 128, "page": 32, "bits": 8, "dtype": "bfloat16", "ragged": False, "causal": True},
        # a mixed step: chunks of all sizes and single tokens together, heads of 64, halves
        {"name": "mixed_step_16", "op": "attention", "seqs": 24, "ctx": 3900, "chunk": 300, "heads": 12,
         "kv_heads": 12, "head_dim": 64, "page": 16, "bits": 16, "dtype": "float16", "ragged": True, "causal": True},
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rotary", "write", "read", "attention", "attention", "attention"])
    heads, kv_heads, d = rng.choice([(12, 12, 64), (32, 32, 128), (64, 8, 128), (24, 8, 64), (20, 4, 128), (16, 1, 128)])
    dtype = rng.choice(["bfloat16", "bfloat16", "float16"])
    if op == "rotary":
        return {"op": op, "tokens": spread(1, 16384), "heads": heads, "kv_heads": kv_heads, "head_dim": d,
                "rotary_dim": rng.choice([d, d, d // 2, d // 4, 20]), "interleaved": rng.random() < 0.5,
                "factor": rng.choice([1.0, 1.0, 4.0, 32.0]), "far": spread(512, 1000000), "dtype": dtype}
    page = rng.choice([16, 32, 64, 128])
    bits = rng.choice([16, 8, 4])
    if op != "attention":
        return {"op": op, "tokens": spread(1, 8192), "kv_heads": kv_heads, "head_dim": d, "page": page, "bits": bits,
                "dtype": dtype}
    if rng.random() < 0.5:  # single tokens and short guesses
        seqs = spread(1, 64)
        chunk = rng.choice([1, 1, 1, 2, 4])
        ctx = spread(1 + chunk, min(131072, 4 * 131072 * 8 // (seqs * kv_heads * 2)))
    else:
        seqs = spread(1, 16)
        chunk = spread(5, 2048)
        ctx = chunk + spread(1, 16384)
        most = 64 * 1024 * 12000  # scores of the plain form
        while seqs * heads * chunk * ctx > most:
            seqs, chunk = max(1, seqs // 2), chunk if seqs > 1 else chunk // 2
            ctx = max(chunk, ctx)
    return {"op": op, "seqs": seqs, "ctx": ctx, "chunk": chunk, "heads": heads, "kv_heads": kv_heads, "head_dim": d,
            "page": page, "bits": bits, "dtype": dtype, "ragged": rng.random() < 0.5, "causal": rng.random() < 0.85}


def lengths(case):
    """Keys and new tokens of each sequence."""
    S, ctx, chunk = case["seqs"], case["ctx"], case["chunk"]
    if not case["ragged"]:
        return [ctx] * S, [chunk] * S
    new = [max(1, chunk // (1, 2, 300, 5, 3)[s % 5]) for s in range(S)]
    return [max(new[s], ctx - (ctx * s * 7 // 8) // S) for s in range(S)], new


def work(case):
    op, d = case["op"], case["head_dim"]
    if op == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"])
        return {"bytes": 4 * n * d + 4 * case["tokens"] + 4 * case["rotary_dim"], "flops": 3 * n * case["rotary_dim"]}
    vector = d * case["bits"] // 8 + (5 if case["bits"] < 16 else 0)  # codes, scale, zero point
    if op in ("write", "read"):
        n = 2 * case["tokens"] * case["kv_heads"]
        both = 2 if op == "write" else 1  # written, and read back
        return {"bytes": n * both * (2 * d + vector) + 4 * case["tokens"], "flops": 4 * both * n * d}
    have, new = lengths(case)
    pairs = sum(n * (L - n) + n * (n + 1) // 2 if case["causal"] else n * L for L, n in zip(have, new))
    return {"bytes": 4 * sum(new) * case["heads"] * d + sum(have) * case["kv_heads"] * 2 * vector
            + 4 * sum(-(-L // case["page"]) for L in have) + 8 * len(have),
            "flops": 4 * d * case["heads"] * pairs}


# ------------------------------------------------------------------ inputs
def frequencies(r, factor, base=10000.0, original=4096, fast=32.0, slow=1.0):
    """Angle per position of each pair, and the factor on the rotated values.  factor 1: base^(-2i/r); above, the pairs
    that turn less than `slow` times within the original length are slowed by `factor`, those that turn more than `fast`
    times are kept, and between the two the share falls linearly."""
    i = torch.arange(r // 2, dtype=torch.float64)
    f = base ** (-2.0 * i / r)
    if factor == 1.0:
        return f, 1.0
    at = [r * math.log(original / (2 * math.pi * t)) / (2 * math.log(base)) for t in (fast, slow)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
    keep = 1.0 - ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
    return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


def quantize(x, bits):
    """Codes, scale and zero point of each vector of the last dimension: the nearest code, decided in 64 bits."""
    most = 2 ** bits - 1
    x = x.double()
    lo, hi = x.amin(-1).clamp(max=0.0), x.amax(-1).clamp(min=0.0)
    none = (lo == 0) & (hi == 0)
    lo, hi = torch.where(none, -1.0, lo), torch.where(none, 1.0, hi)
    s = ((hi - lo).float().double() / most).float()
    z = torch.round(-lo / s.double()).clamp(0, most)
    c = (torch.round(x / s.double()[..., None]) + z[..., None]).clamp(0, most)
    return c.to(torch.uint8), s, z.to(torch.uint8)


def pack(c, bits):
    return c if bits == 8 else c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(c, bits):
    return c if bits == 8 else torch.stack((c & 15, c >> 4), -1).flatten(-2)


def filled_cache(case, pages, g):
    """Pages of keys (with a few heavy channels, as rotated keys have) and values, quantized where the case says so."""
    H, P, d, bits = case["kv_heads"], case["page"], case["head_dim"], case["bits"]
    dev, cache = "cuda", {}
    heavy = 1.0 + 3.0 * (torch.rand(H, 1, d, generator=g, device=dev) < 0.05)
    for side in ("k", "v"):
        x = torch.randn(pages, H, P, d, generator=g, device=dev)
        x = (x * heavy if side == "k" else x).to(DTYPES[case["dtype"]])
        if bits == 16:
            cache[side] = x
        else:
            parts = [quantize(p, bits) for p in x.split(max(1, (1 << 27) // (H * P * d)))]
            cache[side] = torch.cat([pack(p[0], bits) for p in parts])
            cache[side + "_scales"] = torch.cat([p[1] for p in parts])
            cache[side + "_zeros"] = torch.cat([p[2] for p in parts])
    return cache


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dtype, dev, d = DTYPES[case["dtype"]], "cuda", case["head_dim"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    if case["op"] == "rotary":
        T, Hq, Hk = case["tokens"], case["heads"], case["kv_heads"]
        f, a = frequencies(case["rotary_dim"], case["factor"])
        qkv = normal(T, Hq + 2 * Hk, d)  # of one projection: queries and keys are views of it
        first = torch.randint(0, max(1, case["far"] - T) + 1, (1,), generator=g, device=dev)
        at = first + torch.arange(T, device=dev) if T > 64 else torch.randint(0, case["far"], (T,), generator=g, device=dev)
        return {"case": case, "q": qkv[:, :Hq], "k": qkv[:, Hq:Hq + Hk], "positions": at.int(), "f": f.to(dev), "a": a}
    P = case["page"]
    if case["op"] in ("write", "read"):
        T = case["tokens"]
        pages = -(-T // P) + 3
        slots = (torch.randperm(pages, generator=g, device=dev)[:, None] * P + torch.arange(P, device=dev)).flatten()
        if T <= 64:  # tokens of as many users: anywhere
            slots = slots[torch.randperm(slots.numel(), generator=g, device=dev)]
        state = {"case": case, "cache": filled_cache(case, pages, g), "slots": slots[:T].int().contiguous()}
        if case["op"] == "write":
            state["k"], state["v"] = normal(T, case["kv_heads"], d), normal(T, case["kv_heads"], d)
        return state
    have, new = lengths(case)
    need = [-(-L // P) for L in have]
    pages = sum(need) + 5
    order = torch.randperm(pages, generator=g, device=dev)
    table = torch.zeros(len(have), max(need), dtype=torch.int32, device=dev)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = torch.tensor([0] + new).cumsum(0).int().to(dev)
    return {"case": case, "cache": filled_cache(case, pages, g), "q": normal(sum(new), case["heads"], d), "table": table,
            "kv_lens": torch.tensor(have, dtype=torch.int32).to(dev), "q_starts": starts, "longest": max(new)}


# ------------------------------------------------------------------ one pass
def run(state):
    return run_own(state) if own else run_plain(state)


def run_own(state):
    import post_weight_quantization_layer_b200 as gq

    case = state["case"]
    op = case["op"]
    if op == "rotary":
        return gq.rotary(state["q"], state["k"], state["positions"], state["f"], attention_factor=state["a"],
                         interleaved=case["interleaved"])
    if op == "attention":
        return gq.paged_attention(state["q"], state["cache"], state["table"], state["kv_lens"], state["q_starts"],
                                  bits=case["bits"], max_q_len=state["longest"], causal=case["causal"])
    if op == "write":
        gq.cache_write(state["k"], state["v"], state["cache"], state["slots"], bits=case["bits"])
    k, v = gq.cache_read(state["cache"], state["slots"], bits=case["bits"], dtype=DTYPES[case["dtype"]])
    if op == "read" or case["bits"] == 16:
        return k, v
    return k, v, state["cache"]["k_scales"], state["cache"]["v_scales"], state["cache"]["k_zeros"], state["cache"]["v_zeros"]


def run_plain(state):
    case, op = state["case"], state["case"]["op"]
    if op == "rotary":
        angle = state["positions"].double()[:, None, None] * state["f"]
        cos, sin = (angle.cos() * state["a"]).float(), (angle.sin() * state["a"]).float()
        return tuple(rotate_plain(x, cos, sin, case) for x in (state["q"], state["k"]))
    if op == "attention":
        return attention_plain(state)
    cache, bits = state["cache"], case["bits"]
    slots = state["slots"].long()
    page, at = slots // case["page"], slots % case["page"]
    if op == "write":
        store_plain(cache, "k", state["k"], page, at, bits)
        store_plain(cache, "v", state["v"], page, at, bits)
    k, v = (values_plain(cache, side, (page, slice(None), at), bits).to(DTYPES[case["dtype"]]) for side in ("k", "v"))
    if op == "read" or bits == 16:
        return k, v
    return k, v, cache["k_scales"], cache["v_scales"], cache["k_zeros"], cache["v_zeros"]


def rotate_plain(x, cos, sin, case):
    r = case["rotary_dim"]
    y = x.float().clone()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., :r // 2], y[..., r // 2:r])
    turned = a * cos - b * sin, b * cos + a * sin
    a.copy_(turned[0])
    b.copy_(turned[1])
    return y.to(x.dtype)


def store_plain(cache, side, x, page, at, bits):
    if bits == 16:
        cache[side][page, :, at] = x
        return
    c, s, z = quantize(x, bits)
    cache[side][page, :, at] = pack(c, bits)
    cache[side + "_scales"][page, :, at] = s
    cache[side + "_zeros"][page, :, at] = z


def values_plain(cache, side, where, bits):
    x = cache[side][where]
    if bits == 16:
        return x.float()
    s, z = cache[side + "_scales"][where], cache[side + "_zeros"][where]
    return s[..., None] * (unpack(x, bits).float() - z.float()[..., None])


def attention_plain(state):
    case, q = state["case"], state["q"]
    T, Hq, d = q.shape
    H, P, S = case["kv_heads"], case["page"], state["table"].shape[0]
    starts, have = state["q_starts"].long(), state["kv_lens"].long()
    n, token = starts[1:] - starts[:-1], torch.arange(T, device=q.device)
    seq = torch.searchsorted(starts, token, right=True) - 1
    i = token - starts[seq]
    qs = torch.zeros(S, state["longest"], Hq, d, device=q.device)
    qs[seq, i] = q.float()
    qs = qs.view(S, -1, H, Hq // H, d).permute(0, 2, 3, 1, 4).reshape(S, H, -1, d)
    pages = state["table"].long()
    k, v = (values_plain(state["cache"], side, pages, case["bits"]).transpose(1, 2).reshape(S, H, -1, d) for side in ("k", "v"))
    scores = (qs @ k.transpose(-1, -2)).mul_(d ** -0.5).view(S, H, Hq // H, -1, k.shape[2])
    key = torch.arange(k.shape[2], device=q.device)
    last = have[:, None] - 1
    if case["causal"]:
        last = have[:, None] - n[:, None] + torch.arange(state["longest"], device=q.device)
    scores.masked_fill_((key > last[..., None])[:, None, None] | (key >= have[:, None, None])[:, None, None], -math.inf)
    e = scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    o = (e.view(S, H, -1, k.shape[2]) @ v).view(S, H, Hq // H, -1, d) / e.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4).reshape(S, -1, Hq, d)[seq, i].to(q.dtype)


# ------------------------------------------------------------------ from the definitions, in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        r, a = case["rotary_dim"], st["a"]
        turn = torch.polar(torch.full((1,), a, dtype=torch.float64, device="cuda"), st["positions"].double()[:, None] * st["f"])
        out = []
        for x in (st["q"].double(), st["k"].double()):
            part = x[..., :r].unflatten(-1, (r // 2, 2)) if case["interleaved"] else x[..., :r].unflatten(-1, (2, r // 2)).transpose(-1, -2)
            part = torch.view_as_real(torch.view_as_complex(part.contiguous()) * turn[:, None])
            part = part if case["interleaved"] else part.transpose(-1, -2)
            out.append(torch.cat((part.flatten(-2), x[..., r:]), -1))
        return tuple(out)
    cache, bits = st["cache"], case["bits"]
    if case["op"] != "attention":
        return exact_cache(case, st)
    have, new = lengths(case)
    d, group, at, out = case["head_dim"], case["heads"] // case["kv_heads"], 0, []
    for s, (L, n) in enumerate(zip(have, new)):
        ids = st["table"][s, :-(-L // case["page"])].long()
        q = st["q"][at:at + n].double()
        at += n
        rows = torch.empty(n, case["heads"], d, dtype=torch.float64, device="cuda")
        seen = torch.arange(L, device="cuda")[None] <= (torch.arange(n, device="cuda")[:, None] + L - n if case["causal"] else L - 1)
        for h in range(case["kv_heads"]):
            k, v = (exact_values(cache, side, ids, h, bits)[:L] for side in ("k", "v"))
            for j in range(h * group, (h + 1) * group):
                w = torch.softmax(torch.where(seen, q[:, j] @ k.T / math.sqrt(d), -math.inf), -1)
                rows[:, j] = w @ v
        out.append(rows)
    return torch.cat(out)


def exact_values(cache, side, ids, h, bits):
    x = cache[side][ids, h].flatten(0, 1)
    if bits < 16:
        x = unpack(x, bits).double() - cache[side + "_zeros"][ids, h].flatten().double()[:, None]
        x = x * cache[side + "_scales"][ids, h].flatten().double()[:, None]
    return x.double()


def exact_cache(case, st):
    cache, bits, P = st["cache"], case["bits"], case["page"]
    slots = st["slots"].long()
    out, scales, zeros = [], [], []
    for side in ("k", "v"):
        if bits == 16:
            flat = cache[side].transpose(1, 2).flatten(0, 1)
            out.append((st[side] if case["op"] == "write" else flat[slots]).double())
            continue
        s = cache[side + "_scales"].transpose(1, 2).flatten(0, 1)
        z = cache[side + "_zeros"].transpose(1, 2).flatten(0, 1)
        c = unpack(cache[side], bits).transpose(1, 2).flatten(0, 1)[slots].double()
        if case["op"] == "write":
            x, most = st[side].double(), float(2 ** bits - 1)
            lo, hi = torch.minimum(x.min(-1)[0], torch.zeros(1, device="cuda").double()), torch.maximum(x.max(-1)[0], torch.zeros(1, device="cuda").double())
            step = ((hi - lo).float().double() / most).float()  # the scale is stored in 32 bits
            zero = (-lo / step.double()).round()
            s[slots], z[slots] = step, zero.to(torch.uint8)
            c = ((x / step.double()[..., None]).round() + zero[..., None]).clamp(0.0, most)
        out.append(s[slots].double()[..., None] * (c - z[slots].double()[..., None]))
        scales.append(s.unflatten(0, (-1, P)).transpose(1, 2).double())
        zeros.append(None)
    return tuple(out + (scales + zeros if case["op"] == "write" else []))
