"""Cases for serving over a cache held in 4 bits: its write and read (pa_reshape_and_cache_fp4, pa_read_cache_fp4), one
decode step (pa_decode_fp4) and a chunk of new tokens (pa_prefill_fp4) over it, block tables and slot maps kept on the GPU
(pa_tables_trim, pa_tables_extend), and rotary positions with several axes (pa_rope_axes_and_cache).

What they compute.  Token i of sequence s sits at offset i % B of block block_tables[s][i / B].

* 4-bit rows: every 16 neighbouring elements x share a scale, s = e4m3(max |x| / (6 unit)); an element is held as the
  e2m1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to x * (1 / (s unit)), ties to even, and stands
  for e2m1 * s * unit.  All steps are single fp32 operations.  Of each (block, head), 16 tokens lie in 1152 bytes:
  [16][64] bytes of two elements (the first in the low half), then [16][8] scales.
* decode: out = softmax_i(scale * q . k_i) v_i over the positions i <= p with i > p - window or i < sinks, p the last
  position of the sequence (no window: all).
* prefill: the same for each of the last n tokens of a sequence, p the query's own position.
* tables: requests keep their first `keep` tokens (rejected drafts, finished requests), the blocks past them go back on
  the stack of free blocks; then every request gets `new` tokens with their slots, positions and fresh blocks.
* rope: the first r elements of every query and key head turn by the angle t * f_j; t is the token's position along the
  axis that pair j belongs to (time, height, width).  Keys and values go to the token's cache slot.

``run`` computes them in elementary torch operations, or through the package where ``own`` is true.
"""
import math
import random

import numpy as np
import torch

own = False

TORCH = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2, "fp8": 1}
K_UNIT, V_UNIT = 0.0025, 0.0028  # units of the 4-bit caches: scales of up to 448 reach 6.7 and 7.5
K_SCALE, V_SCALE = 0.0123, 0.0117  # dequantisation scales of the FP8 caches
D = 128  # head size of the 4-bit caches
TILE, CODES = 1152, 1024  # bytes of 16 tokens of a head, of their elements
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the cache write of a decode step: latency
        write("fp4_write_step_64", "bf16", 64, 8, 32),
        # the cache write of a batch of prompts
        write("fp4_write_prompt_20001", "f16", 20001, 8, 16),
        # one user waiting for the next token of a long context: latency
        decode("fp4_decode_1", "bf16", 1, 64, 8, 32, 0, 0, 20000, False),
        # a serving batch, contexts of many lengths
        decode("fp4_decode_96", "f16", 96, 64, 8, 32, 0, 0, 16384, False),
        # one key head for each query head, the step's token appended, a window over each context's end
        decode("fp4_decode_64_mha_append", "bf16", 64, 32, 32, 16, 4000, 17, 8192, True),
        # drafted tokens to verify: a few queries a sequence
        prefill("fp4_drafts_16x5", "bf16", 16, 5, 5, 64, 8, 32, 0, 0, 20000),
        # one long prompt's chunk
        prefill("fp4_prompt_2048", "f16", 1, 2048, 2048, 32, 8, 16, 0, 0, 8192),
        # chunked prefill of several prompts at once
        prefill("fp4_prompts_8", "bf16", 8, 200, 900, 32, 8, 64, 1500, 4, 4096),
        # a decode step after the verification of drafts, few requests: latency
        tables("tables_drafts_64", 64, 5, 0, 0, 16, 16384),
        # a large batch: most requests decode, some are done and make room for prompts
        tables("tables_prompts_2000", 2000, 5, 60, 20000, 32, 40000),
        # the position and cache write of a decode step
        rope("axes_step_48", "bf16", 48, 0, 64, 8, 128, 128, False, 32),
        # prompts with images: patches of one time, many heights and widths
        rope("axes_images_16000", "f16", 16000, 900, 32, 8, 128, 128, False, 16),
    ]


def write(name, dtype, tokens, kv_heads, block_size):
    return {"name": name, "op": "write", "dtype": dtype, "tokens": tokens, "kv_heads": kv_heads, "block_size": block_size,
            "spread": 4}


def decode(name, dtype, seqs, q_heads, kv_heads, block_size, window, sinks, max_len, append):
    return {"name": name, "op": "decode", "dtype": dtype, "seqs": seqs, "q_heads": q_heads, "kv_heads": kv_heads,
            "block_size": block_size, "window": window, "sinks": sinks, "max_len": max_len, "append": append, "spread": 5}


def prefill(name, dtype, seqs, min_chunk, max_chunk, q_heads, kv_heads, block_size, window, sinks, max_prefix):
    return {"name": name, "op": "prefill", "dtype": dtype, "seqs": seqs, "min_chunk": min_chunk, "max_chunk": max_chunk,
            "q_heads": q_heads, "kv_heads": kv_heads, "block_size": block_size, "window": window, "sinks": sinks,
            "max_prefix": max_prefix, "spread": 6}


def tables(name, seqs, drafts, prompts, max_prompt, block_size, max_len):
    return {"name": name, "op": "tables", "seqs": seqs, "drafts": drafts, "prompts": prompts, "max_prompt": max_prompt,
            "block_size": block_size, "max_len": max_len, "spread": 7}


def rope(name, dtype, tokens, patches, q_heads, kv_heads, head_size, rotary_dim, interleaved, block_size):
    """patches: of an image; 0: text alone, whose positions are the same along every axis."""
    return {"name": name, "op": "rope", "dtype": dtype, "tokens": tokens, "patches": patches, "q_heads": q_heads,
            "kv_heads": kv_heads, "head_size": head_size, "rotary_dim": rotary_dim, "interleaved": interleaved,
            "block_size": block_size, "spread": 8}


def log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "prefill", "tables", "rope"])
    dtype = rng.choice(["f16", "bf16"])
    q_heads, kv_heads = rng.choice([(64, 8), (32, 8), (32, 32), (24, 4), (40, 8), (7, 1), (16, 1)])
    block_size = rng.choice([16, 32, 48, 64, 128])
    window, sinks = rng.choice([(0, 0), (0, 0), (log_int(rng, 17, 8192), rng.choice([0, 1, 4, 64]))])
    spread = rng.randrange(1 << 20)
    if op == "write":
        c = write("", dtype, log_int(rng, 1, 16384), kv_heads, block_size)
    elif op == "decode":
        max_len, seqs = log_int(rng, 64, 40000), log_int(rng, 1, 128)
        limit = (3 << 28) // (144 * kv_heads * min(max_len, (window or max_len) + sinks))  # 768 MiB of keys and values
        c = decode("", dtype, max(1, min(seqs, limit)), q_heads, kv_heads, block_size, window, sinks, max_len,
                   rng.random() < 0.4)
    elif op == "prefill":
        hi, prefix = log_int(rng, 1, 2048), log_int(rng, 16, 16000)
        limit = (1 << 31) // (q_heads * hi * (hi + min(prefix, (window or prefix) + sinks)))
        c = prefill("", dtype, max(1, min(log_int(rng, 1, 16), limit)), max(1, hi // 3), hi, q_heads, kv_heads, block_size,
                    window, sinks, prefix)
    elif op == "tables":
        seqs = log_int(rng, 1, 2000)
        c = tables("", seqs, rng.choice([1, 3, 5, 9]), rng.randrange(min(seqs, 50) + 1), log_int(rng, 16, 20000),
                   rng.choice([8, 16, 24, 32, 64]), log_int(rng, 64, 40000))
    else:
        dtype = rng.choice(["bf16", "f16", "fp8", "f32"])
        head_size = 128 if dtype == "fp8" else rng.choice([64, 128, 128])
        rotary = rng.choice([head_size, head_size, head_size // 2, head_size // 4 + 2])
        tokens = log_int(rng, 1, 12000)
        c = rope("", dtype, tokens, rng.choice([0, log_int(rng, 4, 2000)]), q_heads, kv_heads, head_size, rotary,
                 rng.random() < 0.5, rng.choice([16, 32, 64]))
    del c["name"]
    c["spread"] = spread
    return c


def shapes(case):
    """The lengths of a case's sequences: they go by the case alone, so that every seed does the same work."""
    rng = random.Random(case["spread"])
    if case["op"] == "decode":
        n = case["seqs"]
        return [case["max_len"] if n == 1 else log_int(rng, max(1, case["max_len"] // 16), case["max_len"])
                for s in range(n)]
    if case["op"] == "prefill":
        chunks = [rng.randint(case["min_chunk"], case["max_chunk"]) for s in range(case["seqs"])]
        return [(c + log_int(rng, max(1, case["max_prefix"] // 8), case["max_prefix"]), c) for c in chunks]  # (length, chunk)
    # (length, tokens kept) of each request
    n, got = case["seqs"], []
    fresh = set(rng.sample(range(n), case["prompts"]))
    for s in range(n):
        if s in fresh:
            got.append((log_int(rng, max(1, case["max_prompt"] // 16), case["max_prompt"]), 0))
        else:
            L = log_int(rng, max(case["drafts"], case["max_len"] // 16), case["max_len"])
            got.append((L, max(0, L - rng.randint(1, case["drafts"]))))
    return got


# ---------------------------------------------------------------- 4-bit rows
def quantise(x, unit):
    """Elements and scales, [..., 64] and [..., 8] bytes, of rows x [..., 128] in 32 bits; unit: a number on the device."""
    g = x.unflatten(-1, (8, 16))
    s = (g.abs().amax(-1) / (unit * 6.0)).clamp_(max=448.0).to(torch.float8_e4m3fn)
    t = s.float() * unit
    y = g * torch.where(t > 0, 1.0 / t, torch.zeros_like(t))[..., None]
    a = y.abs()
    code = torch.zeros_like(a, dtype=torch.uint8)
    for at, with_tie in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= at) if with_tie else (a > at)
    code += (torch.signbit(y) & (t > 0)[..., None]).to(torch.uint8) * 8
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), s.view(torch.uint8)


def parts(cache):
    """A cache's elements [blocks, heads, B / 16, 16, 64] and scales [blocks, heads, B / 16, 16, 8], as views."""
    return cache[..., :CODES].unflatten(-1, (16, 64)), cache[..., CODES:].unflatten(-1, (16, 8))


def values(codes, scales, unit):
    """The numbers that elements and scales stand for, in 32 bits."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    x = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return x * scales.view(torch.float8_e4m3fn).float().repeat_interleave(16, -1) * unit


def held_rows(cache, block, off, unit):
    """Rows of the tokens at offset off of the blocks, [..., heads, 128]."""
    codes, scales = parts(cache)
    return values(codes[block, :, off // 16, off % 16], scales[block, :, off // 16, off % 16], unit)


def store_rows(cache, block, off, x, unit):
    codes, scales = parts(cache)
    c, s = quantise(x, unit)
    codes[block, :, off // 16, off % 16] = c
    scales[block, :, off // 16, off % 16] = s


# ---------------------------------------------------------------- inputs
def normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def cache_of(g, num_blocks, heads, block_size, unit):
    """A pool of quantised normal rows."""
    cache = torch.empty((num_blocks, heads, block_size // 16, TILE), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (heads * block_size * D))
    codes, scales = parts(cache)
    for b in range(0, num_blocks, step):
        x = torch.randn((min(step, num_blocks - b), heads, block_size // 16, 16, D), generator=g, device="cuda")
        codes[b:b + step], scales[b:b + step] = quantise(x, unit)
    return cache


def tables_of(g, block_size, spans, width):
    """Shuffled blocks for the spans of tokens each sequence still holds; -1 where its blocks were released.
    Returns the table and the number of blocks in the pool."""
    held = np.zeros((len(spans), width), bool)
    for s, ranges in enumerate(spans):
        for lo, hi in ranges:
            if hi > lo:
                held[s, lo // block_size:-(-hi // block_size)] = True
    total = int(held.sum())
    num_blocks = total + total // 8 + 1
    ids = torch.randperm(num_blocks, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full(held.shape, -1, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(held).cuda()] = ids
    return table, num_blocks


def frequencies(r):
    return 1000000.0 ** (-2.0 * torch.arange(r // 2, dtype=torch.float64) / r)


def axes_of(r):
    """The axis of each rotary pair: a quarter of the pairs for time, the rest shared by height and width."""
    t = r // 8
    h = (r // 2 - t) // 2
    return [0] * t + [1] * h + [2] * (r // 2 - t - h)


def positions_of(case):
    """Positions [3, tokens]: text, and images of `patches` patches (half as many rows as columns) between."""
    rng, n, got = random.Random(case["spread"]), case["tokens"], []
    if not case["patches"]:
        at = [rng.randrange(100000) for _ in range(n)] if n <= 64 else range(n)
        return np.tile(np.asarray(at, np.int32), (3, 1))
    at = 0
    while len(got) < n:
        text = rng.randint(5, 200)
        got += [(at + i,) * 3 for i in range(text)]
        at += text
        h = max(1, int(math.sqrt(case["patches"] / 2)))
        w = max(1, case["patches"] // h)
        got += [(at, at + y, at + x) for y in range(h) for x in range(w)]
        at += max(h, w)
    return np.ascontiguousarray(np.asarray(got[:n], np.int32).T)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st = {"case": case, "err": torch.zeros(1, dtype=torch.int32, device="cuda"), "scale": 1.0 / math.sqrt(D),
          "k_unit": torch.tensor(K_UNIT, device="cuda"), "v_unit": torch.tensor(V_UNIT, device="cuda")}
    return {"write": prepare_write, "decode": prepare_attention, "prefill": prepare_attention, "tables": prepare_tables,
            "rope": prepare_rope}[case["op"]](case, st, g)


def prepare_write(case, st, g):
    T, B, hkv, t = case["tokens"], case["block_size"], case["kv_heads"], TORCH[case["dtype"]]
    num_blocks = -(-T // B) + T // (8 * B) + 1
    st["k"], st["v"] = cache_of(g, num_blocks, hkv, B, st["k_unit"]), cache_of(g, num_blocks, hkv, B, st["v_unit"])
    if T <= 256:  # a step: tokens of sequences of their own
        st["slots"] = torch.randperm(num_blocks * B, generator=g, device="cuda")[:T]
    else:
        table = torch.randperm(num_blocks, generator=g, device="cuda")
        i = torch.arange(T, device="cuda")
        st["slots"] = table[i // B] * B + i % B
    st["key"], st["value"] = normal(g, (T, hkv, D), t), normal(g, (T, hkv, D), t)
    st["key_held"], st["value_held"] = torch.zeros_like(st["key"]), torch.zeros_like(st["value"])
    return st


def prepare_attention(case, st, g):
    B, hq, hkv, t = case["block_size"], case["q_heads"], case["kv_heads"], TORCH[case["dtype"]]
    W, S = case["window"] or 1 << 30, case["sinks"]
    if case["op"] == "decode":
        lens = shapes(case)
        spans = [[(0, min(S, L)), (max(0, L - W), L)] for L in lens]
        st["q"] = normal(g, (len(lens), hq, D), t)
        if case["append"]:
            st["key"], st["value"] = (normal(g, (len(lens), hkv, D), t) for _ in range(2))
            st["key_held"], st["value_held"] = torch.zeros_like(st["key"]), torch.zeros_like(st["value"])
    else:
        both = shapes(case)
        lens, chunks = [L for L, n in both], [n for L, n in both]
        spans = [[(0, min(S, L)), (max(0, L - n - W + 1), L)] for L, n in both]
        starts = np.concatenate([[0], np.cumsum(chunks)]).astype(np.int32)
        st.update(query_start=torch.from_numpy(starts).cuda(), max_query_len=max(chunks),
                  q=normal(g, (int(starts[-1]), hq, D), t))
    st["tables"], num_blocks = tables_of(g, B, spans, -(-max(lens) // B))
    st["k"], st["v"] = cache_of(g, num_blocks, hkv, B, st["k_unit"]), cache_of(g, num_blocks, hkv, B, st["v_unit"])
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    st["out"] = torch.zeros_like(st["q"])
    if case["op"] == "decode" and case["append"]:
        last = st["lens"].long() - 1
        st["slots"] = st["tables"].long().gather(1, (last // B)[:, None])[:, 0] * B + last % B
    return st


def prepare_tables(case, st, g):
    both, B = shapes(case), case["block_size"]
    lens = np.array([L for L, keep in both], np.int32)
    held = -(-lens // B)
    width = int(held.max()) + 1
    total = int(held.sum())
    num_blocks = total + total // 8 + 1
    ids = torch.randperm(num_blocks, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(both), width), -1, dtype=torch.int32, device="cuda")
    table[torch.from_numpy(np.arange(width)[None] < held[:, None]).cuda()] = ids[:total]
    free = torch.full((num_blocks,), -1, dtype=torch.int32, device="cuda")
    free[:num_blocks - total] = ids[total:]
    keep = torch.tensor([k for L, k in both], dtype=torch.int32, device="cuda")
    lens = torch.from_numpy(lens).cuda()
    rows = int(sum(L - k for L, k in both))
    st.update(table=table, lens=lens, held=torch.from_numpy(held.astype(np.int32)).cuda(), free=free,
              num_free=torch.tensor([num_blocks - total], dtype=torch.int32, device="cuda"), keep=keep, new=lens - keep,
              slots=torch.zeros(rows + rows // 16, dtype=torch.int64, device="cuda"),
              positions=torch.zeros(rows + rows // 16, dtype=torch.int32, device="cuda"),
              query_start=torch.zeros(len(both) + 1, dtype=torch.int32, device="cuda"))
    return st


def prepare_rope(case, st, g):
    B, d, hq, hkv, T, t = (case[k] for k in ("block_size", "head_size", "q_heads", "kv_heads", "tokens", "dtype"))
    num_blocks = -(-T // B) + T // (8 * B) + 1
    shape, t, fp8 = (num_blocks, hkv, B, d), TORCH[t], t == "fp8"
    st["k"] = torch.zeros(shape, dtype=torch.uint8 if fp8 else t, device="cuda")
    st["v"] = torch.zeros((num_blocks, hkv, B // 16, d, 16) if fp8 else shape, dtype=st["k"].dtype, device="cuda")
    table = torch.randperm(num_blocks, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    st.update(slots=table[i // B] * B + i % B, positions=torch.from_numpy(positions_of(case)).cuda(),
              inv_freq=frequencies(case["rotary_dim"]).cuda(), axes=axes_of(case["rotary_dim"]),
              axis=torch.tensor(axes_of(case["rotary_dim"]), device="cuda"),
              qkv=normal(g, (T, (hq + 2 * hkv) * d), t), q_out=torch.zeros((T, hq, d), dtype=t, device="cuda"))
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return {"write": own_write, "decode": own_decode, "prefill": own_prefill, "tables": own_tables,
                "rope": own_rope}[op](st)
    return {"write": plain_write, "decode": plain_decode, "prefill": plain_prefill, "tables": plain_tables,
            "rope": plain_rope}[op](st)


def own_write(st):
    import paged_kv_cache_32_gb300 as pa
    pa.pa_reshape_and_cache_fp4(st["k"], st["v"], st["key"], st["value"], st["slots"], K_UNIT, V_UNIT, err_flag=st["err"])
    pa.pa_read_cache_fp4(st["key_held"], st["value_held"], st["k"], st["v"], st["slots"], K_UNIT, V_UNIT,
                         err_flag=st["err"])
    return st["key_held"], st["value_held"]


def own_decode(st):
    import paged_kv_cache_32_gb300 as pa
    c = st["case"]
    pa.pa_decode_fp4(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["scale"], K_UNIT, V_UNIT,
                     window=c["window"] or None, num_sinks=c["sinks"], key=st.get("key"), value=st.get("value"),
                     err_flag=st["err"])
    if not c["append"]:
        return st["out"]
    pa.pa_read_cache_fp4(st["key_held"], st["value_held"], st["k"], st["v"], st["slots"], K_UNIT, V_UNIT,
                         err_flag=st["err"])
    return st["out"], st["key_held"], st["value_held"]


def own_prefill(st):
    import paged_kv_cache_32_gb300 as pa
    c = st["case"]
    pa.pa_prefill_fp4(st["out"], st["q"], st["k"], st["v"], st["tables"], st["lens"], st["query_start"],
                      st["max_query_len"], st["scale"], K_UNIT, V_UNIT, window=c["window"] or None, num_sinks=c["sinks"],
                      err_flag=st["err"])
    return st["out"]


def own_tables(st):
    import paged_kv_cache_32_gb300 as pa
    B = st["case"]["block_size"]
    pa.pa_tables_trim(st["table"], st["lens"], st["held"], st["free"], st["num_free"], st["keep"], B, err_flag=st["err"])
    pa.pa_tables_extend(st["table"], st["lens"], st["held"], st["free"], st["num_free"], st["new"], st["slots"],
                        st["positions"], st["query_start"], B, err_flag=st["err"])
    return [st[k] for k in ("table", "lens", "held", "free", "num_free", "slots", "positions", "query_start")]


def own_rope(st):
    import paged_kv_cache_32_gb300 as pa
    c = st["case"]
    q, key, value = split(st)
    scales = dict(k_scale=K_SCALE, v_scale=V_SCALE) if c["dtype"] == "fp8" else {}
    pa.pa_rope_axes_and_cache(st["q_out"], st["k"], st["v"], q, key, value, st["positions"], st["slots"], st["inv_freq"],
                              st["axes"], interleaved=c["interleaved"], err_flag=st["err"], **scales)
    return st["q_out"], as_values(st["k"]), as_values(st["v"])


def plain_write(st):
    B = st["case"]["block_size"]
    block, off = st["slots"] // B, st["slots"] % B
    for name, cache, unit in (("key", "k", "k_unit"), ("value", "v", "v_unit")):
        store_rows(st[cache], block, off, st[name].float(), st[unit])
        st[name + "_held"].copy_(held_rows(st[cache], block, off, st[unit]))
    return st["key_held"], st["value_held"]


def attend(q, k, v, seen, scale):
    """softmax(scale * q k^T) v over the seen keys: q [n, kv head, rows, D], seen [n, 1, rows, keys]."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    s = s.sub_(s.amax(-1, keepdim=True).clamp_(min=-3e38)).exp_()
    total = s.sum(-1, keepdim=True)
    return torch.matmul(s, v).div_(total.clamp_(min=1e-30))


def plain_decode(st):
    c = st["case"]
    hq, hkv, B, S = c["q_heads"], c["kv_heads"], c["block_size"], c["sinks"]
    if c["append"]:
        block, off = st["slots"] // B, st["slots"] % B
        for name, cache, unit in (("key", "k", "k_unit"), ("value", "v", "v_unit")):
            store_rows(st[cache], block, off, st[name].float(), st[unit])
            st[name + "_held"].copy_(held_rows(st[cache], block, off, st[unit]))
    lens = shapes(c)
    s = 0
    while s < len(lens):  # as many sequences at once as half a GiB of keys holds
        e, most = s, 0
        while e < len(lens) and (e == s or (e + 1 - s) * max(most, lens[e]) * hkv * D * 4 <= 1 << 29):
            most = max(most, lens[e])
            e += 1
        W = min(c["window"] or most, most)
        last = st["lens"][s:e].long()[:, None] - 1
        near = last - W + 1 + torch.arange(W, device="cuda")
        sink = torch.arange(S, device="cuda").expand(e - s, S)
        pos = torch.cat([sink, near], 1)
        seen = torch.cat([(sink <= last - W) & (sink <= last), near >= 0], 1)[:, None, None]
        pos = pos.clamp(min=0).minimum(last)
        block = torch.gather(st["tables"][s:e], 1, pos // B).long().clamp_(min=0)
        k = held_rows(st["k"], block, pos % B, st["k_unit"]).transpose(1, 2)
        v = held_rows(st["v"], block, pos % B, st["v_unit"]).transpose(1, 2)
        out = attend(st["q"][s:e].float().view(e - s, hkv, hq // hkv, D), k, v, seen, st["scale"])
        st["out"][s:e] = out.reshape(e - s, hq, D).to(st["out"].dtype)
        s = e
    return (st["out"], st["key_held"], st["value_held"]) if c["append"] else st["out"]


def plain_prefill(st):
    c = st["case"]
    hq, hkv, B, S = c["q_heads"], c["kv_heads"], c["block_size"], c["sinks"]
    G, a = hq // hkv, 0
    for s, (L, n) in enumerate(shapes(c)):
        W = c["window"] or L
        lo = max(0, L - n - W + 1)
        pos = torch.arange(L, device="cuda")
        pos = torch.cat([pos[:min(S, lo)], pos[lo:]])
        p = torch.arange(L - n, L, device="cuda")[:, None]
        seen = (pos <= p) & ((pos > p - W) | (pos < S))
        block = st["tables"][s][pos // B].long()
        k = held_rows(st["k"], block, pos % B, st["k_unit"]).transpose(0, 1)[None]
        v = held_rows(st["v"], block, pos % B, st["v_unit"]).transpose(0, 1)[None]
        q = st["q"][a:a + n].float().view(n, hkv, G, D).transpose(0, 1).reshape(1, hkv, n * G, D)
        seen = seen[:, None].expand(n, G, -1).reshape(1, 1, n * G, -1)
        out = attend(q, k, v, seen, st["scale"])[0].view(hkv, n, G, D).transpose(0, 1)
        st["out"][a:a + n] = out.reshape(n, hq, D).to(st["out"].dtype)
        a += n
    return st["out"]


def plain_tables(st):
    B, table, lens, held, free = st["case"]["block_size"], st["table"], st["lens"], st["held"], st["free"]
    width, cols = table.shape[1], torch.arange(table.shape[1], device="cuda")
    rows = torch.arange(st["slots"].numel(), device="cuda")
    # ---- trim: the blocks past the kept tokens, the first request's first one on top of the stack
    kept = (st["keep"] + B - 1) // B
    gone = held - kept
    before = torch.cumsum(gone, 0) - gone
    total = gone.sum()
    out = (cols >= kept[:, None]) & (cols < held[:, None])
    at = st["num_free"] + total - 1 - (before[:, None] + cols - kept[:, None])
    sink = torch.cat([free, free[:1]])  # (one place more, for the blocks that stay)
    sink[torch.where(out, at, free.numel()).long()] = table
    free.copy_(sink[:-1])
    table.masked_fill_(out, -1)
    lens.copy_(st["keep"])
    held.copy_(kept)
    st["num_free"].add_(total)
    # ---- extend
    new = st["new"]
    want = torch.maximum((lens + new + B - 1) // B, held)
    need = want - held
    before = torch.cumsum(need, 0) - need
    got = (cols >= held[:, None]) & (cols < want[:, None])
    at = (st["num_free"] - 1 - (before[:, None] + cols - held[:, None])).clamp(0, free.numel() - 1).long()
    table.copy_(torch.where(got, free[at], table))
    end = torch.cumsum(new, 0)
    st["query_start"][1:] = end
    s = torch.searchsorted(end, rows, right=True)
    real = s < new.numel()
    s = s.clamp(max=new.numel() - 1)
    pos = (lens[s] + rows - (end[s] - new[s])).long()
    block = table.flatten()[(s * width + pos // B).clamp(max=table.numel() - 1)].long()
    st["slots"].copy_(torch.where(real, block * B + pos % B, -1))
    st["positions"].copy_(torch.where(real, pos, 0))
    lens.add_(new)
    held.copy_(want)
    st["num_free"].sub_(need.sum())
    return [st[k] for k in ("table", "lens", "held", "free", "num_free", "slots", "positions", "query_start")]


def split(st):
    """Query, key and value of a fused projection, as views."""
    c = st["case"]
    hq, hkv = c["q_heads"], c["kv_heads"]
    x = st["qkv"].view(-1, hq + 2 * hkv, c["head_size"])
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]


def as_values(x):
    """An FP8 cache as the values its codes stand for (to the cache's scale)."""
    return x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x


def e4m3(x, scale):
    """E4M3 codes of x / scale, saturating."""
    return (x / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def turn(x, cos, sin, r, interleaved):
    """The first r elements of each head of x turned, in 32 bits; cos and sin [tokens, 1, r / 2]."""
    x = x.float()
    y = x.clone()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    u, v = (y[..., 0:r:2], y[..., 1:r:2]) if interleaved else (y[..., :r // 2], y[..., r // 2:r])
    u.copy_(a * cos - b * sin)
    v.copy_(b * cos + a * sin)
    return y


def plain_rope(st):
    c = st["case"]
    q, key, value = split(st)
    r, B, inter = c["rotary_dim"], c["block_size"], c["interleaved"]
    angle = (st["positions"][st["axis"]].T.double() * st["inv_freq"])[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    st["q_out"].copy_(turn(q, cos, sin, r, inter))
    key, block, off = turn(key, cos, sin, r, inter), st["slots"] // B, st["slots"] % B
    if c["dtype"] == "fp8":
        st["k"][block, :, off] = e4m3(key, K_SCALE)
        st["v"][block, :, off // 16, :, off % 16] = e4m3(value.float(), V_SCALE)
    else:
        st["k"][block, :, off] = key.to(st["k"].dtype)
        st["v"][block, :, off] = value
    return st["q_out"], as_values(st["k"]), as_values(st["v"])


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "write":  # the rows read, written in 4 bits, read back
        rows = case["tokens"] * case["kv_heads"] * 2
        return {"bytes": rows * (2 * D * 2 + 2 * 72) + 16 * case["tokens"], "flops": 6.0 * rows * D}
    if case["op"] == "tables":
        both, B = shapes(case), case["block_size"]
        new = sum(L - k for L, k in both)
        moved = sum(-(-L // B) - -(-k // B) for L, k in both)
        # lengths, blocks held, kept, new; the blocks' entries both ways; of each new token its block, slot and position
        return {"bytes": 8 * 4 * len(both) + moved * 4 * 4 + new * (8 + 4) + 4 * sum(-(-(L - k) // B) for L, k in both),
                "flops": 4.0 * new}
    hq, hkv = case["q_heads"], case["kv_heads"]
    if case["op"] == "rope":
        d, T, e = case["head_size"], case["tokens"], SIZE[case["dtype"]]
        eq = max(2, e)
        return {"bytes": T * d * (2 * hq * eq + 2 * hkv * (eq + e)) + T * 20 + case["rotary_dim"] * 4,
                "flops": 6.0 * T * (hq + hkv) * (case["rotary_dim"] // 2)}
    W, S = case["window"] or 1 << 30, case["sinks"]
    if case["op"] == "decode":
        lens = shapes(case)
        seen = sum(min(L, W) + min(S, max(0, L - W)) for L in lens)
        rows = len(lens) * hkv * 2  # appended: read, written, read back
        moved = 2 * len(lens) * hq * D * 2 + (rows * (2 * D * 2 + 2 * 72) if case["append"] else 0)
        blocks = sum(-(-L // case["block_size"]) - max(0, L - W) // case["block_size"] for L in lens)
        return {"bytes": 144 * seen * hkv + moved + 4 * (blocks + len(lens)), "flops": 4.0 * seen * hq * D}
    both = shapes(case)
    pairs = keys = 0
    for L, n in both:
        p = np.arange(L - n, L)
        pairs += int((np.minimum(p + 1, W) + np.minimum(S, np.maximum(0, p + 1 - W))).sum())
        lo = max(0, L - n - W + 1)
        keys += L - lo + min(S, lo)
    return {"bytes": 144 * keys * hkv + 2 * sum(n for L, n in both) * hq * D * 2, "flops": 4.0 * pairs * hq * D}


# ---------------------------------------------------------------- the definition in 64 bits
def nearest(y):
    """The e2m1 numbers nearest to y, ties to the even one (64 bits)."""
    steps = torch.tensor(E2M1, dtype=torch.float64, device=y.device)
    far = (y.abs()[..., None] - steps).abs()
    best = far.amin(-1, keepdim=True)
    # among the (at most two) nearest the one with an even place
    order = torch.arange(8, device=y.device)
    rank = torch.where(far == best, order % 2 * 8 + order, 99).amin(-1)
    return steps[rank % 8] * torch.where(y < 0, -1.0, 1.0)


def single(x):
    """Rounded to 32 bits, as a 64-bit number (a quotient or product of two 32-bit numbers is rounded right this way)."""
    return x.float().double()


def exact_rows(x, unit):
    """What rows x stand for once held in 4 bits."""
    unit = float(np.float32(unit))
    six = float(np.float32(np.float32(unit) * np.float32(6.0)))
    got = []
    for part in x.double().split(2048):
        g = part.unflatten(-1, (8, 16))
        s = single(g.abs().amax(-1) / six).clamp(max=448.0).float().to(torch.float8_e4m3fn).double()
        t = single(s * unit)
        y = single(g * single(1.0 / t.clamp(min=1e-30))[..., None])
        got.append((torch.where(t[..., None] > 0, nearest(y), 0.0) * s[..., None] * unit).flatten(-2))
    return torch.cat(got)


def exact_held(cache, block, off, unit):
    """Rows [tokens, heads, 128] from the bytes of a cache, in 64 bits."""
    rows = cache[block, :, off.div(16, rounding_mode="floor")]
    r, i = off.remainder(16), torch.arange(len(off), device="cuda")
    codes = rows[..., :CODES].reshape(*rows.shape[:2], 16, 64).transpose(1, 2)[i, r]
    scale = rows[..., CODES:].reshape(*rows.shape[:2], 16, 8).transpose(1, 2)[i, r]
    x = torch.empty((*codes.shape[:2], 128), dtype=torch.float64, device="cuda")
    for half in (0, 1):
        nibble = codes.long().bitwise_right_shift(4 * half).bitwise_and(15)
        e, m = nibble.bitwise_right_shift(1).bitwise_and(3), nibble.bitwise_and(1)
        mag = torch.where(e > 0, (1.0 + 0.5 * m) * 2.0 ** (e - 1).double(), 0.5 * m)
        x[..., half::2] = torch.where(nibble > 7, -mag, mag)
    return (x.view(*x.shape[:2], 8, 16) * scale.contiguous().view(torch.float8_e4m3fn).double()[..., None]).view(x.shape) * float(
        np.float32(unit))


def exact(case, seed):
    """Sequence by sequence, every position compared with the definition's bounds; tables in plain loops."""
    st = prepare(case, seed)
    if case["op"] == "write":
        return exact_rows(st["key"], K_UNIT), exact_rows(st["value"], V_UNIT)
    if case["op"] == "tables":
        return exact_tables(case, st)
    if case["op"] == "rope":
        return exact_rope(case, st)
    hq, hkv, B = case["q_heads"], case["kv_heads"], case["block_size"]
    lens, G, W, S = st["lens"].tolist(), hq // hkv, case["window"] or 1 << 30, case["sinks"]
    append = case["op"] == "decode" and case["append"]
    starts = st["query_start"].tolist() if case["op"] == "prefill" else list(range(len(lens) + 1))
    if append:
        new_k, new_v = exact_rows(st["key"], K_UNIT), exact_rows(st["value"], V_UNIT)
    q, out = st["q"].double(), torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for s, L in enumerate(lens):
        a, b = starts[s], starts[s + 1]
        i, p = torch.arange(L, device="cuda"), torch.arange(L - (b - a), L, device="cuda")
        mask = (i[None] <= p[:, None]) & ((i[None] > p[:, None] - W) | (i[None] < S))
        i = i[mask.any(0)]
        mask = mask[:, i]
        blk = st["tables"][s, i // B].long()
        k, v = exact_held(st["k"], blk, i % B, K_UNIT), exact_held(st["v"], blk, i % B, V_UNIT)
        if append:
            k[-1], v[-1] = new_k[s], new_v[s]
        for u in range(hq):
            w = (q[a:b, u] @ k[:, u // G].T) * st["scale"]
            out[a:b, u] = torch.softmax(w.masked_fill(~mask, -math.inf), 1) @ v[:, u // G]
    return (out, new_k, new_v) if append else out


def exact_tables(case, st):
    B = case["block_size"]
    table, lens, held, free, keep, new = (st[k].cpu().numpy().copy() for k in ("table", "lens", "held", "free", "keep", "new"))
    top = int(st["num_free"].item())
    gone = []
    for s in range(len(lens)):
        first = -(-int(keep[s]) // B)
        gone += [int(x) for x in table[s, first:held[s]]]
        table[s, first:held[s]] = -1
        lens[s], held[s] = keep[s], first
    free[top:top + len(gone)] = gone[::-1]
    top += len(gone)
    slots, pos = np.full(st["slots"].numel(), -1, np.int64), np.zeros(st["slots"].numel(), np.int32)
    start = np.zeros(len(lens) + 1, np.int32)
    for s in range(len(lens)):
        while held[s] * B < lens[s] + new[s]:
            top -= 1
            table[s, held[s]] = free[top]
            held[s] += 1
        i = np.arange(lens[s], lens[s] + new[s])
        start[s + 1] = start[s] + new[s]
        slots[start[s]:start[s + 1]] = table[s, i // B].astype(np.int64) * B + i % B
        pos[start[s]:start[s + 1]] = i
        lens[s] += new[s]
    return [torch.from_numpy(x) for x in (table, lens, held, free, np.array([top], np.int32), slots, pos, start)]


def exact_rope(case, st):
    B, d, hq, hkv = case["block_size"], case["head_size"], case["q_heads"], case["kv_heads"]
    r, fp8, x = case["rotary_dim"], case["dtype"] == "fp8", st["qkv"].double().view(case["tokens"], hq + 2 * hkv, d)
    turned = x.clone()
    for j in range(r // 2):
        theta = st["positions"][st["axes"][j]].double() * st["inv_freq"][j]
        i0, i1 = (2 * j, 2 * j + 1) if case["interleaved"] else (j, j + r // 2)
        c, s = theta.cos()[:, None], theta.sin()[:, None]
        turned[:, :, i0] = c * x[:, :, i0] - s * x[:, :, i1]
        turned[:, :, i1] = s * x[:, :, i0] + c * x[:, :, i1]
    key, value = turned[:, hq:hq + hkv], x[:, hq + hkv:]
    kc, vc = (as_values(st[n]).double() for n in ("k", "v"))
    if fp8:
        key = (key / float(np.float32(K_SCALE))).clamp(-448, 448)
        value = (value / float(np.float32(V_SCALE))).clamp(-448, 448)
    b, o = st["slots"].div(B, rounding_mode="floor"), st["slots"].remainder(B)
    for h in range(hkv):
        kc[b, h, o] = key[:, h]
        if fp8:
            vc[b, h, o.div(16, rounding_mode="floor"), :, o.remainder(16)] = value[:, h]
        else:
            vc[b, h, o] = value[:, h]
    return turned[:, :hq].contiguous(), kc, vc
