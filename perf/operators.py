"""Cases for the sliding-window serving operators: rotary positions with the cache write
(pa_rope_and_cache), one decode step over a window and a few first tokens that stay visible
(pa_decode_window), and a chunk of new tokens over the same (pa_prefill_window).

What they compute.  Token i of sequence s sits at offset i % B of block block_tables[s][i / B].

* rope: the first r elements of every query and key head turn by the angle t * f_j (t the token's
  position, f_j the frequency of pair j, j < r / 2) and are scaled by a magnitude; pairs are (j, j + r / 2)
  or (2j, 2j + 1).  Keys and values go to the token's cache slot (an FP8 cache holds E4M3 codes of x / scale).
* decode: out = softmax_i(scale * q . k_i) v_i over the positions i <= p with i > p - window or i < sinks,
  p the last position of the sequence.
* prefill: the same for each of the last n tokens of a sequence, p the query's own position.

``run`` computes them in elementary torch operations, or through the package where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
K_SCALE, V_SCALE = 0.0123, 0.0117  # dequantisation scales of the FP8 caches


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the position and cache write of a decode step with few sequences: latency
        rope("rope_step_8", "bf16", 8, 8, 64, 8, 128, 128, False, "none", 32, 4096),
        # a full decode batch into an FP8 cache, halves of the head turned
        rope("rope_step_128_fp8", "fp8", 128, 128, 64, 8, 128, 64, False, "linear", 32, 16384),
        # prompts of a chunked prefill, frequencies stretched for a long context
        rope("rope_prompt_9001", "bf16", 9001, 5, 64, 8, 128, 128, False, "yarn", 32, 100000),
        # a long prompt of a model with one key head for each query head and neighbouring pairs
        rope("rope_prompt_24576_f16", "f16", 24576, 12, 32, 32, 128, 128, True, "none", 16, 2048),
        # one user waiting for the next token: latency
        decode("decode_1", "bf16", 1, 64, 8, 128, 32, 4096, 4, 20000, False),
        # a serving batch, contexts of many lengths around a short window
        decode("decode_128_w1024", "bf16", 128, 64, 8, 128, 32, 1024, 4, 16384, False),
        # one key head for each query head, the step's token appended, window ends off the blocks
        decode("decode_64_mha_append", "f16", 64, 32, 32, 128, 16, 2000, 17, 8192, True),
        # a long window over an FP8 cache
        decode("decode_96_fp8", "fp8", 96, 32, 8, 128, 32, 8192, 128, 40000, False),
        # drafted tokens to verify: a few queries a sequence
        prefill("prefill_drafts_8x5", "bf16", 8, 5, 5, 64, 8, 128, 32, 4096, 4, 20000),
        # chunked prefill of many prompts at once, short window
        prefill("prefill_16_w1024", "bf16", 16, 256, 1024, 32, 8, 128, 16, 1024, 4, 8192),
        # one long prompt, long window
        prefill("prefill_4096_f16", "f16", 1, 4096, 4096, 32, 8, 128, 16, 4096, 64, 12288),
        # short chunks over an FP8 cache
        prefill("prefill_4x61_fp8", "fp8", 4, 61, 61, 32, 8, 128, 32, 2048, 4, 9000),
    ]


def rope(name, dtype, tokens, seqs, q_heads, kv_heads, head_size, rotary_dim, interleaved, scaling, block_size, start):
    return {"name": name, "op": "rope", "dtype": dtype, "tokens": tokens, "seqs": seqs, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_size": head_size, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "scaling": scaling, "block_size": block_size, "start": start, "spread": 1}


def decode(name, dtype, seqs, q_heads, kv_heads, head_size, block_size, window, sinks, max_len, append):
    return {"name": name, "op": "decode", "dtype": dtype, "seqs": seqs, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_size": head_size, "block_size": block_size, "window": window, "sinks": sinks, "max_len": max_len,
            "append": append, "spread": 2}


def prefill(name, dtype, seqs, min_chunk, max_chunk, q_heads, kv_heads, head_size, block_size, window, sinks, max_prefix):
    return {"name": name, "op": "prefill", "dtype": dtype, "seqs": seqs, "min_chunk": min_chunk, "max_chunk": max_chunk,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_size": head_size, "block_size": block_size,
            "window": window, "sinks": sinks, "max_prefix": max_prefix, "spread": 3}


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "decode", "prefill"])
    dtype = rng.choice(["bf16", "bf16", "f16", "fp8", "f32"])
    head_size = 128 if dtype == "fp8" else rng.choice([64, 128, 128])
    q_heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (24, 4), (40, 8), (7, 1), (16, 1)])
    block_size = rng.choice([16, 32, 64] if dtype == "fp8" else [8, 16, 32, 64])
    spread = rng.randrange(1 << 20)
    if op == "rope":
        seqs = log_int(rng, 1, 128)
        tokens = seqs if rng.random() < 0.4 else log_int(rng, seqs, 16384)
        rotary = rng.choice([head_size, head_size, head_size // 2, head_size // 4 + 2])
        c = rope("", dtype, tokens, seqs, q_heads, kv_heads, head_size, rotary, rng.random() < 0.5,
                 rng.choice(["none", "linear", "yarn"]), block_size, log_int(rng, 1, 500000))
    elif op == "decode":
        window, seqs = log_int(rng, 17, 8192), log_int(rng, 1, 128)
        limit = (1 << 30) // (2 * kv_heads * head_size * SIZE[dtype] * window)  # at most 1 GiB of keys and values
        c = decode("", dtype, max(1, min(seqs, limit)), q_heads, kv_heads, head_size, block_size, window,
                   rng.choice([0, 1, 4, 64]), log_int(rng, 64, 40000), dtype != "f32" and rng.random() < 0.5)
    else:
        fast = dtype in ("bf16", "f16") and head_size == 128
        window = log_int(rng, 17, 4096)
        hi = log_int(rng, 1, 2048 if fast else 96)
        limit = (1 << 30) // (q_heads * hi * (hi + window + 64))  # scores of the plain form: at most 4 GiB
        c = prefill("", dtype, max(1, min(log_int(rng, 1, 16), limit)), max(1, hi // 3), hi, q_heads, kv_heads, head_size,
                    block_size, window, rng.choice([0, 1, 4, 64]), log_int(rng, 16, 20000))
    del c["name"]
    c["spread"] = spread
    return c


def shapes(case):
    """The lengths of a case's sequences: they go by the case alone, so that every seed does the same work."""
    rng, n = random.Random(case["spread"]), case["seqs"]
    if case["op"] == "rope":
        share, more = divmod(case["tokens"], n)
        return [(share + (s < more), rng.randrange(case["start"])) for s in range(n)]  # (new tokens, position of the first)
    if case["op"] == "decode":
        return [case["max_len"] if n == 1 else log_int(rng, max(1, case["max_len"] // 16), case["max_len"])
                for s in range(n)]
    chunks = [rng.randint(case["min_chunk"], case["max_chunk"]) for s in range(n)]
    return [(c + log_int(rng, max(1, case["max_prefix"] // 8), case["max_prefix"]), c) for c in chunks]  # (length, chunk)


# ---------------------------------------------------------------- inputs
def normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def codes(x, scale):
    """E4M3 codes of x / scale, saturating."""
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def caches(g, case, num_blocks):
    kv, B, D = case["kv_heads"], case["block_size"], case["head_size"]
    k = normal(g, (num_blocks, kv, B, D), torch.float32 if case["dtype"] == "fp8" else TORCH[case["dtype"]])
    v = normal(g, (num_blocks, kv, B, D), torch.float32 if case["dtype"] == "fp8" else TORCH[case["dtype"]])
    if case["dtype"] == "fp8":  # values: a dimension's 16 tokens side by side
        k = codes(k, K_SCALE)
        v = codes(v, V_SCALE).reshape(num_blocks, kv, B // 16, 16, D).transpose(3, 4).contiguous()
    return k, v


def tables_of(g, case, spans, width):
    """Shuffled blocks for the spans of tokens each sequence still holds; -1 where its blocks were released.
    Returns the table and the number of blocks in the pool."""
    B = case["block_size"]
    held = np.zeros((len(spans), width), bool)
    for s, parts in enumerate(spans):
        for lo, hi in parts:
            if hi > lo:
                held[s, lo // B:-(-hi // B)] = True
    total = int(held.sum())
    num_blocks = total + total // 8 + 1
    ids = torch.randperm(num_blocks, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(held).cuda()] = ids
    return table, num_blocks


def frequencies(case):
    """(radians a position for each pair, magnitude) of a rope case, in 64 bits."""
    r = case["rotary_dim"]
    base = 500000.0 if case["scaling"] == "yarn" else 10000.0
    j = torch.arange(r // 2, dtype=torch.float64)
    f = base ** (-2.0 * j / r)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":
        factor, trained, fast, slow = 16.0, 8192.0, 32.0, 1.0
        turn = lambda n: r * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(0, math.floor(turn(fast))), min(r - 1, math.ceil(turn(slow)))
        ramp = ((j - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        return f * (1 - ramp) + f / factor * ramp, 0.1 * math.log(factor) + 1.0
    return f, 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, D, hq, hkv = case["block_size"], case["head_size"], case["q_heads"], case["kv_heads"]
    t = TORCH[case["dtype"]]
    st = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(D)}
    if case["op"] == "rope":
        new = shapes(case)
        # each sequence's blocks from the one that holds its first new token on
        first = [p // B * B for n, p in new]
        spans = [[(0, p - f + n)] if n else [] for (n, p), f in zip(new, first)]
        table, num_blocks = tables_of(g, case, spans, max(-(-(p - f + n) // B) for (n, p), f in zip(new, first)))
        k, v = caches(g, case, num_blocks)
        seq = torch.from_numpy(np.repeat(np.arange(len(new)), [n for n, p in new])).cuda()
        pos = np.concatenate([np.arange(p, p + n) for n, p in new])
        off = torch.from_numpy(pos - np.repeat(first, [n for n, p in new])).cuda()
        slots = table[seq, off // B].to(torch.int64) * B + off % B
        inv_freq, magnitude = frequencies(case)
        T = case["tokens"]
        st.update(k=k, v=v, slots=slots, positions=torch.from_numpy(pos.astype(np.int32)).cuda(),
                  inv_freq=inv_freq.cuda(), magnitude=magnitude, qkv=normal(g, (T, (hq + 2 * hkv) * D), t),
                  q_out=torch.zeros((T, hq, D), dtype=t, device="cuda"))
        return st
    W, S = case["window"], case["sinks"]
    if case["op"] == "decode":
        lens = shapes(case)
        spans = [[(0, min(S, L)), (max(0, L - W), L)] for L in lens]
        st["q"] = normal(g, (len(lens), hq, D), t)
        if case["append"]:
            st["key"], st["value"] = (normal(g, (len(lens), hkv, D), t) for _ in range(2))
    else:
        both = shapes(case)
        lens, chunks = [L for L, n in both], [n for L, n in both]
        spans = [[(0, min(S, L)), (max(0, L - n - W + 1), L)] for L, n in both]
        starts = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        st.update(query_start=torch.from_numpy(starts).cuda(), max_query_len=max(chunks),
                  q=normal(g, (int(starts[-1]), hq, D), t))
    st["tables"], num_blocks = tables_of(g, case, spans, -(-max(lens) // B))
    st["k"], st["v"] = caches(g, case, num_blocks)
    st["max_len"] = max(lens)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["out"] = torch.zeros_like(st["q"])
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"rope": own_rope, "decode": own_decode, "prefill": own_prefill}[op](st)
    return {"rope": plain_rope, "decode": plain_decode, "prefill": plain_prefill}[op](st)


def split(st):
    """Query, key and value of a fused projection, as views."""
    c = st["case"]
    D, hq, hkv = c["head_size"], c["q_heads"], c["kv_heads"]
    x = st["qkv"].view(-1, hq + 2 * hkv, D)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def held(x):
    """An FP8 cache as the values its codes stand for (to the cache's scale)."""
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def own_rope(st):
    import paged_kv_cache_32_gb300 as pa
    q, key, value = split(st)
    fp8 = st["case"]["dtype"] == "fp8"
    pa.pa_rope_and_cache(st["q_out"], st["k"], st["v"], q, key, value, st["positions"], st["slots"], st["inv_freq"],
                         interleaved=st["case"]["interleaved"], magnitude=st["magnitude"], err_flag=st["err"],
                         k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
    return st["q_out"], held(st["k"]), held(st["v"])


def own_decode(st):
    import paged_kv_cache_32_gb300 as pa
    c = st["case"]
    fp8 = c["dtype"] == "fp8"
    pa.pa_decode_window(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["scale"], c["window"],
                        num_sinks=c["sinks"], key=st.get("key"), value=st.get("value"), err_flag=st["err"],
                        k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
    return (st["out"], held(st["k"]), held(st["v"])) if c["append"] else st["out"]


def own_prefill(st):
    import paged_kv_cache_32_gb300 as pa
    c = st["case"]
    fp8 = c["dtype"] == "fp8"
    pa.pa_prefill_window(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["query_start"],
                         st["max_query_len"], st["scale"], c["window"], num_sinks=c["sinks"], err_flag=st["err"],
                         k_scale=K_SCALE if fp8 else None, v_scale=V_SCALE if fp8 else None)
    return st["out"]


def turn(x, cos, sin, r, interleaved):
    """The first r elements of each head of x turned, in 32 bits; cos and sin [tokens, 1, r / 2]."""
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, v = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    u.copy_(a * cos - b * sin)
    v.copy_(b * cos + a * sin)
    return y


def store(c, k_cache, v_cache, key, value, slots):
    """Key and value rows (32 bits) into their slots."""
    block, off = slots // c["block_size"], slots % c["block_size"]
    if c["dtype"] == "fp8":
        k_cache[block, :, off] = codes(key, K_SCALE)
        v_cache[block, :, off // 16, :, off % 16] = codes(value, V_SCALE)
    else:
        k_cache[block, :, off] = key.to(k_cache.dtype)
        v_cache[block, :, off] = value.to(v_cache.dtype)


def plain_rope(st):
    c = st["case"]
    q, key, value = split(st)
    angle = st["positions"].double()[:, None, None] * st["inv_freq"]
    cos, sin = (torch.cos(angle) * st["magnitude"]).float(), (torch.sin(angle) * st["magnitude"]).float()
    st["q_out"].copy_(turn(q, cos, sin, c["rotary_dim"], c["interleaved"]))
    store(c, st["k"], st["v"], turn(key, cos, sin, c["rotary_dim"], c["interleaved"]), value.float(), st["slots"])
    return st["q_out"], held(st["k"]), held(st["v"])


def rows(c, cache, table, pos, scale, values):
    """Rows [sequence, kv head, position, D] of the tokens at pos [sequence, position] in 32 bits."""
    block = torch.gather(table, 1, pos // c["block_size"]).long().clamp_(min=0)
    off = pos % c["block_size"]
    if c["dtype"] != "fp8":
        return cache[block, :, off].float().transpose(1, 2)
    x = cache[block, :, off // 16, :, off % 16] if values else cache[block, :, off]
    return x.view(torch.float8_e4m3fn).float().transpose(1, 2) * scale


def attend(q, k, v, seen, scale):
    """softmax(scale * q k^T) v over the seen keys: q [n, kv head, rows, D], seen [n, 1, rows, keys]."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.matmul(s, v).div_(total.clamp_(min=1e-30))


def plain_decode(st):
    c = st["case"]
    n, hq, hkv, D, W, S = c["seqs"], c["q_heads"], c["kv_heads"], c["head_size"], c["window"], c["sinks"]
    last = st["lens"].long()[:, None] - 1
    if c["append"]:
        block = torch.gather(st["tables"], 1, last // c["block_size"]).long()
        slots = (block * c["block_size"] + last % c["block_size"])[:, 0]
        store(c, st["k"], st["v"], st["key"].float(), st["value"].float(), slots)
    W = min(W, st["max_len"])
    near = last - W + 1 + torch.arange(W, device="cuda")
    sink = torch.arange(S, device="cuda").expand(n, S)
    pos = torch.cat([sink, near], 1)
    seen = torch.cat([(sink <= last - W) & (sink <= last), near >= 0], 1)[:, None, None]
    pos = pos.clamp(min=0).minimum(last)
    k = rows(c, st["k"], st["tables"], pos, K_SCALE, False)
    v = rows(c, st["v"], st["tables"], pos, V_SCALE, True)
    out = attend(st["q"].float().view(n, hkv, hq // hkv, D), k, v, seen, st["scale"])
    st["out"].copy_(out.reshape(n, hq, D))
    return (st["out"], held(st["k"]), held(st["v"])) if c["append"] else st["out"]


def plain_prefill(st):
    c = st["case"]
    n, hq, hkv, D, W, S = c["seqs"], c["q_heads"], c["kv_heads"], c["head_size"], c["window"], c["sinks"]
    G, m = hq // hkv, st["max_query_len"]
    starts, L = st["query_start"].long(), st["lens"].long()[:, None]
    chunk = (starts[1:] - starts[:-1])[:, None]
    j = torch.arange(m, device="cuda")
    inside = j < chunk
    at = (starts[:-1, None] + j).clamp(max=st["q"].shape[0] - 1)
    qpos = (L - chunk + j).minimum(L - 1)
    span = min(m + W - 1, st["max_len"])
    near = L - span + torch.arange(span, device="cuda")
    sink = torch.arange(S, device="cuda").expand(n, S)
    pos = torch.cat([sink, near], 1)
    alive = torch.cat([(sink < L - span), near >= 0], 1)
    seen = (pos[:, None] <= qpos[..., None]) & ((pos[:, None] > qpos[..., None] - W) | (pos[:, None] < S))
    seen = (seen & alive[:, None])[:, None, :, None].expand(n, 1, m, G, -1).reshape(n, 1, m * G, -1)
    pos = pos.clamp(min=0).minimum(L - 1)
    k = rows(c, st["k"], st["tables"], pos, K_SCALE, False)
    v = rows(c, st["v"], st["tables"], pos, V_SCALE, True)
    q = st["q"][at].float().view(n, m, hkv, G, D).transpose(1, 2).reshape(n, hkv, m * G, D)
    out = attend(q, k, v, seen, st["scale"]).view(n, hkv, m, G, D).transpose(1, 2).reshape(n, m, hq, D)
    st["out"][at[inside]] = out[inside].to(st["out"].dtype)
    return st["out"]


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    D, hq, hkv, e = case["head_size"], case["q_heads"], case["kv_heads"], SIZE[case["dtype"]]
    eq = max(2, e)  # queries, outputs and new rows of an FP8 cache are fp16
    if case["op"] == "rope":
        T = case["tokens"]
        return {"bytes": T * D * (2 * hq * eq + 2 * hkv * (eq + e)) + T * 12 + case["rotary_dim"] * 4,
                "flops": 6.0 * T * (hq + hkv) * (case["rotary_dim"] // 2)}
    W, S = case["window"], case["sinks"]
    if case["op"] == "decode":
        lens = shapes(case)
        seen = sum(min(L, W) + min(S, max(0, L - W)) for L in lens)
        moved = 2 * len(lens) * hq * D * eq + (2 * len(lens) * hkv * D * eq if case["append"] else 0)
        held_blocks = sum(-(-L // case["block_size"]) - max(0, L - W) // case["block_size"] for L in lens)
        return {"bytes": 2 * seen * hkv * D * e + moved + 4 * (held_blocks + len(lens)), "flops": 4.0 * seen * hq * D}
    both = shapes(case)
    pairs = keys = 0
    for L, n in both:
        p = np.arange(L - n, L)
        pairs += int((np.minimum(p + 1, W) + np.minimum(S, np.maximum(0, p + 1 - W))).sum())
        lo = max(0, L - n - W + 1)
        keys += L - lo + min(S, lo)
    return {"bytes": 2 * keys * hkv * D * e + 2 * sum(n for L, n in both) * hq * D * eq, "flops": 4.0 * pairs * hq * D}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    """Sequence by sequence (token by token for the cache), every position compared with the definition's bounds."""
    st = prepare(case, seed)
    B, D, hq, hkv = case["block_size"], case["head_size"], case["q_heads"], case["kv_heads"]
    fp8 = case["dtype"] == "fp8"

    def real(cache):
        return cache.view(torch.float8_e4m3fn).double() if fp8 else cache.double()

    def put(kc, vc, key, value, slots):  # unrounded rows, an FP8 cache's in units of its scale
        key = (key / float(np.float32(K_SCALE))).clamp(-448, 448) if fp8 else key
        value = (value / float(np.float32(V_SCALE))).clamp(-448, 448) if fp8 else value
        b, o = slots.div(B, rounding_mode="floor"), slots.remainder(B)
        for h in range(hkv):
            kc[b, h, o] = key[:, h]
            if fp8:
                vc[b, h, o.div(16, rounding_mode="floor"), :, o.remainder(16)] = value[:, h]
            else:
                vc[b, h, o] = value[:, h]
        return kc, vc

    if case["op"] == "rope":
        r, x = case["rotary_dim"], st["qkv"].double().view(case["tokens"], hq + 2 * hkv, D)
        turned = x.clone()
        theta = torch.outer(st["positions"].double(), st["inv_freq"])
        for j in range(r // 2):
            i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + r // 2)
            c, s = theta[:, j].cos()[:, None] * st["magnitude"], theta[:, j].sin()[:, None] * st["magnitude"]
            turned[:, :, i0] = c * x[:, :, i0] - s * x[:, :, i1]
            turned[:, :, i1] = s * x[:, :, i0] + c * x[:, :, i1]
        kc, vc = put(real(st["k"]), real(st["v"]), turned[:, hq:hq + hkv], x[:, hq + hkv:], st["slots"])
        return turned[:, :hq].contiguous(), kc, vc
    kc, vc = real(st["k"]), real(st["v"])
    lens, table, W, S, G = st["lens"].tolist(), st["tables"], case["window"], case["sinks"], hq // hkv
    if case["op"] == "decode":
        starts = list(range(len(lens) + 1))
        if case["append"]:
            slots = torch.stack([table[s, (L - 1) // B].long() * B + (L - 1) % B for s, L in enumerate(lens)])
            kc, vc = put(kc, vc, st["key"].double(), st["value"].double(), slots)
    else:
        starts = st["query_start"].tolist()
    q, out = st["q"].double(), torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    k_unit, v_unit = (float(np.float32(K_SCALE)), float(np.float32(V_SCALE))) if fp8 else (1.0, 1.0)
    for s, L in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        i = torch.arange(L, device="cuda")
        p = torch.arange(L - (b - a), L, device="cuda")
        mask = (i[None] <= p[:, None]) & ((i[None] > p[:, None] - W) | (i[None] < S))
        i = i[mask.any(0)]
        mask = mask[:, i]
        blk, off = table[s, i // B].long(), i % B
        for h in range(hkv):
            kk = kc[blk, h, off] * k_unit
            vv = (vc[blk, h, off // 16, :, off % 16] if fp8 else vc[blk, h, off]) * v_unit
            for u in range(h * G, (h + 1) * G):
                w = (q[a:b, u] @ kk.T) * st["scale"]
                out[a:b, u] = torch.softmax(w.masked_fill(~mask, -math.inf), 1) @ vv
    return (out, kc, vc) if case["op"] == "decode" and case["append"] else out
