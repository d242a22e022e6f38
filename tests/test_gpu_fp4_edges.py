"""Caches held in 4 bits: calls and values at the edges of what they take (needs a GB300)."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


def test_copy_blocks_without_a_descriptor(pa):
    """Whole blocks, codes and scales, and no other byte."""
    import torch
    k, v = (torch.randint(0, 256, (6, 3, 3, 1152), dtype=torch.uint8, device="cuda") for _ in range(2))
    want = k.clone(), v.clone()
    for t in want:
        t[4], t[1] = t[0], t[5]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks(k, v, torch.tensor([[0, 4], [5, 1]], dtype=torch.int32, device="cuda"), err_flag=err)
    assert int(err.item()) == 0 and torch.equal(k, want[0]) and torch.equal(v, want[1])


def lagging_cache(pa, length, low, unit):
    """One sequence's blocks of 16 in bf16: keys +-6 (the first `low` tokens the negative ones), every value the largest
    number that a cache of this unit holds.  The scores of queries of ones rise by 7.9 binary orders behind the low tokens,
    which the running maximum of what starts at the low ones does not follow."""
    import torch
    key = torch.full((length, 1, 128), 6.0, dtype=torch.bfloat16, device="cuda")
    key[:low] = -6.0
    value = torch.full_like(key, 2688.0 * unit)
    k, v = (pa.fp4_cache(length // 16, 1, 16) for _ in range(2))
    pa.pa_reshape_and_cache_fp4(k, v, key, value, torch.arange(length, device="cuda"), 1.0, unit)
    return k, v, 7.9 / (2 * 128 * 6 * 1.4426950408889634)


@pytest.mark.parametrize("power", [100, -100])
@pytest.mark.parametrize("form,length", [("clusters", 4000), ("even", 40000), ("tiles", 4096)])
def test_value_unit_at_its_ends(pa, form, length, power):
    """Values that the rows' type holds come out as they are, however large or small the unit and whatever a row has added
    up before the division: every value is the same number, a weighted mean of it within 2^-11 for the rounding of the
    weights, and half a step of bf16."""
    import torch
    unit, seqs = 2.0 ** power, 160
    k, v, scale = lagging_cache(pa, length, 192, unit)
    table = torch.arange(length // 16, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if form == "tiles":
        q = torch.ones(300, 8, 128, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        start = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
        pa.pa_prefill_fp4(out, q, k, v, table[:1].contiguous(), lens[:1], start, 300, scale, 1.0, unit, err_flag=err)
    else:
        q = torch.ones(seqs, 8, 128, dtype=torch.bfloat16, device="cuda")
        out = torch.zeros_like(q)
        need = pa.pa_decode_fp4_workspace_size(seqs, 8, length // 16, pa.fp4_cache_desc(k))
        assert need > 0
        kw = dict(alibi_slopes=torch.zeros(8, device="cuda")) if form == "clusters" else {}  # (ALiBi: always in clusters)
        pa.pa_decode_fp4(out, q, k, v, table, lens, scale, 1.0, unit, err_flag=err, **kw)
    assert int(err.item()) == 0
    want = 2688.0 * unit
    far = (out.double() / want - 1).abs().max().item()
    assert far <= 2.0 ** -11 + 2.0 ** -8, far


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("form", ["clusters", "even", "tiles", "split tiles"])
def test_many_small_weights_beside_a_large_one(pa, rows, form):
    """The first token takes nearly everything, and 2^20 others of 2^-25.5 each have a share of 2 % between them: their
    values are 1, the first one's 0.  Off by at most 2^-11 for the weights' rounding, half a step of the rows' type, and
    what fp32 sums lose: 16 weights of 2^-25.5 at a time against a sum of 1 to 2^-23 of it lose up to 0.36 of their share
    of the sum (0.36 * 2 % of the result), and against their own sum, of values times weights, up to 2^-7 of it."""
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16
    length, unit = 1 << 20, 1.0 / 6
    # block 0 holds the first token and 15 others, block 1 others only; a sequence is block 0, then block 1 over and over
    key = torch.full((32, 1, 128), -6.0, dtype=t, device="cuda")
    value = torch.ones_like(key)
    key[0], value[0] = 6.0, 0.0
    k, v = (pa.fp4_cache(2, 1, 16) for _ in range(2))
    pa.pa_reshape_and_cache_fp4(k, v, key, value, torch.arange(32, device="cuda"), 1.0, unit)
    scale = 25.5 / (2 * 128 * 6 * 1.4426950408889634)
    seqs = 160 if form in ("clusters", "even") else 1
    table = torch.ones(seqs, length // 16, dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if seqs > 1:
        q = torch.ones(seqs, 8, 128, dtype=t, device="cuda")
        out, seen = torch.zeros_like(q), torch.full((seqs,), float(length), dtype=torch.float64)
        kw = dict(alibi_slopes=torch.zeros(8, device="cuda")) if form == "clusters" else {}  # (ALiBi: always in clusters)
        pa.pa_decode_fp4(out, q, k, v, table, lens, scale, 1.0, unit, err_flag=err, **kw)
    else:
        n = 1200 if form == "split tiles" else 1200 * 16
        q = torch.ones(n, 8, 128, dtype=t, device="cuda")
        out, seen = torch.zeros_like(q), torch.arange(length - n + 1, length + 1, dtype=torch.float64)
        start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        pa.pa_prefill_fp4(out, q, k, v, table, lens, start, n, scale, 1.0, unit, err_flag=err)
    assert int(err.item()) == 0
    w = (seen - 1) * 2.0 ** -25.5
    want = (w / (1 + w))[:, None, None]
    far = ((out.cpu().double() - want).abs() / (2.0 ** -11 * 1.25 + want * (2.0 ** -8 + 2.0 ** -6))).max().item()
    assert far <= 1, far


FIRST_CALL = """
import torch
import paged_kv_cache_32_gb300 as pa
for rows in (torch.float16, torch.bfloat16):
    k = torch.randint(0, 112, (2600, 1, 1, 1152), device="cuda", dtype=torch.uint8)
    table = torch.arange(2600, device="cuda", dtype=torch.int32)[None]
    lens = torch.tensor([40000], device="cuda", dtype=torch.int32)
    slots = torch.arange(200, device="cuda")
    inv, _ = pa.pa_rope_frequencies(128, device="cuda")
    def chunk(n):
        q = torch.ones(n, 8, 128, device="cuda", dtype=rows)
        start = torch.tensor([0, n], device="cuda", dtype=torch.int32)
        return lambda o: pa.pa_prefill_fp4(o, q, k, k, table, lens, start, n, 0.01, 0.01, 0.01), torch.zeros_like(q)
    def decode(**kw):
        q = torch.ones(1, 8, 128, device="cuda", dtype=rows)
        return lambda o: pa.pa_decode_fp4(o, q, k, k, table, lens, 0.01, 0.01, 0.01, **kw), torch.zeros_like(q)
    def write(rotary):
        x = torch.ones(200, 6, 128, device="cuda", dtype=rows)
        pos = torch.arange(200, device="cuda", dtype=torch.int32)[None].contiguous()
        c = pa.fp4_cache(20, 1, 16)
        return lambda o: pa.pa_rope_axes_and_cache(o, c, c.clone(), x[:, :4], x[:, 4:5], x[:, 5:], pos, slots,
                                                   inv[:rotary // 2].contiguous(), bytes(rotary // 2), k_scale=0.1,
                                                   v_scale=0.1), x[:, :4].clone()
    for call, out in (decode(), decode(window=9000), chunk(1), chunk(40), chunk(3000), write(128), write(34)):
        again = torch.zeros_like(out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(out)
        graph.replay()
        call(again)
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.count_nonzero(out) > 0
print("same")
"""


def test_first_call_captured():
    """A process whose first call of each kernel is captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_pool_past_32_bits(pa, rows):
    """The last blocks of caches of 5.9 GB: every call gives what it gives over the first blocks of small ones."""
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16
    nb, hkv, B, used = 40000, 8, 256, 24
    assert nb * hkv * B // 16 * 1152 > 2 ** 32
    big = [torch.zeros((nb, hkv, B // 16, 1152), dtype=torch.uint8, device="cuda") for _ in range(2)]
    small = [pa.fp4_cache(used, hkv, B) for _ in range(2)]
    shift = nb - used
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(used * B, 4 * hkv, 128, generator=g, device="cuda").to(t)
    slots = torch.randperm(used * B, generator=g, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    key, value, back = x[:, :hkv], x[:, hkv:2 * hkv], torch.zeros(2, 2, used * B, hkv, 128, dtype=t, device="cuda")

    def same():
        assert int(err.item()) == 0
        assert all(torch.equal(b[shift:], s) for b, s in zip(big, small))

    for i, (c, at) in enumerate(((small, slots), (big, slots + shift * B))):
        pa.pa_reshape_and_cache_fp4(*c, key, value, at, 0.0025, 0.0031, err_flag=err)
        pa.pa_read_cache_fp4(*back[i], *c, at, 0.0025, 0.0031, err_flag=err)
    same()
    assert torch.equal(back[0], back[1]) and bool((back[0] != 0).any())
    pos = torch.arange(3 * used * B, dtype=torch.int32, device="cuda").view(3, -1)
    q_out = torch.zeros(2, used * B, 2 * hkv, 128, dtype=t, device="cuda")
    for rotary in (128, 34):
        inv, _ = pa.pa_rope_frequencies(rotary, device="cuda")
        for i, (c, at) in enumerate(((small, slots), (big, slots + shift * B))):
            pa.pa_rope_axes_and_cache(q_out[i], *c, x[:, 2 * hkv:], key, value, pos, at, inv,
                                      bytes(j % 3 for j in range(rotary // 2)), err_flag=err, k_scale=0.0025, v_scale=0.0031)
        same()
        assert torch.equal(q_out[0], q_out[1])
    table = torch.randperm(used, generator=g, device="cuda").to(torch.int32).view(2, 12)
    lens = torch.tensor([12 * B, 2000], dtype=torch.int32, device="cuda")
    wide = torch.cat([table, torch.full((2, 140), -1, dtype=torch.int32, device="cuda")], 1)
    for n, tab in ((1, table), (1, wide), (3, table), (700, table)):
        outs = []
        for c, add in ((small, 0), (big, shift)):
            q = q_out[0, :2 * n].contiguous()
            out, at = torch.zeros_like(q), torch.where(tab >= 0, tab + add, tab)
            if n == 1:
                new = [x[:2, j * hkv:(j + 1) * hkv].contiguous() for j in (2, 3)]
                pa.pa_decode_fp4(out, q, *c, at, lens, 0.09, 0.0025, 0.0031, key=new[0], value=new[1], err_flag=err)
            else:
                start = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
                pa.pa_prefill_fp4(out, q, *c, at, lens, start, n, 0.09, 0.0025, 0.0031, err_flag=err)
            outs.append(out)
        same()
        assert torch.equal(*outs) and bool((outs[0] != 0).any())
    pairs = torch.tensor([[0, 5], [used - 1, 7]], dtype=torch.int32, device="cuda")
    pa.pa_copy_blocks(*small, pairs, err_flag=err)
    pa.pa_copy_blocks(*big, pairs + shift, err_flag=err)
    same()
    assert not any(bool(b[:shift].any()) for b in big)


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_chunk_in_buffers_of_a_capacity(pa, rows):
    """Single tokens in buffers that could hold prompts, as a captured graph's do: rows past the last are left alone."""
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16
    seqs, length, capacity = 120, 300, 60000
    k, v = (torch.randint(0, 112, (seqs * 19, 2, 1, 1152), device="cuda", dtype=torch.uint8) for _ in range(2))
    table = torch.arange(seqs * 19, device="cuda", dtype=torch.int32).view(seqs, 19)
    lens = torch.full((seqs,), length, dtype=torch.int32, device="cuda")
    q = torch.randn(capacity, 16, 128, device="cuda").to(t)
    for n in (seqs, 90):
        start = torch.arange(n + 1, device="cuda", dtype=torch.int32)
        outs = []
        for rows_of, most in ((capacity, capacity), (n, 1)):
            out = torch.full((rows_of, 16, 128), 123.0, dtype=t, device="cuda")
            err = torch.zeros(1, dtype=torch.int32, device="cuda")
            pa.pa_prefill_fp4(out, q[:rows_of], k, v, table[:n].contiguous(), lens[:n], start, most, 0.01, 0.01, 0.01,
                              err_flag=err)
            assert int(err.item()) == 0
            outs.append(out.double())
        # (the two may run on different kernels: each weight rounded once, by 2^-11; the output, by half a step)
        step = 2.0 ** -11 if rows == "f16" else 2.0 ** -8
        top = 2688 * 0.01
        assert bool(((outs[0][:n] - outs[1]).abs() <= 2 * (2.0 ** -11 * top + step * outs[1].abs() + 2.0 ** -14 * top)).all())
        assert bool((outs[0][n:] == 123.0).all())


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_step_from_pinned_memory(pa, rows, long):
    """The step's small arrays in pinned host memory: the bytes and bits of device arrays (long: slabs dealt out evenly)."""
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16

    def pinned(x):
        return torch.empty(x.shape, dtype=x.dtype).pin_memory().copy_(x.cpu())

    g = torch.Generator(device="cuda").manual_seed(1)
    n, hq, hkv, B, nb = 5, 12, 2, 32, 300
    x = torch.randn(n, hq + 2 * hkv, 128, generator=g, device="cuda").to(t)
    table = torch.randperm(nb, generator=g, device="cuda").to(torch.int32).view(n, nb // n)
    if long:
        table = torch.cat([table, torch.full((n, 1000), -1, dtype=torch.int32, device="cuda")], 1).contiguous()
    lens = torch.tensor([1, 700, 33, 1920, 0], dtype=torch.int32, device="cuda")
    pos = torch.stack([lens, lens // 2, lens // 3])
    slots = torch.arange(n, device="cuda") * 7 + 3
    inv, _ = pa.pa_rope_frequencies(128, device="cuda")
    held = torch.randint(0, 112, (2, nb, hkv, B // 16, 1152), generator=g, device="cuda", dtype=torch.uint8)
    got = []
    for move in (lambda a: a, pinned):
        k, v = held.clone()
        q, key, value, tab, ln, po, sl, fr = (move(a.contiguous()) for a in (x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], table,
                                                                         lens, pos, slots, inv))
        q_out, out = move(torch.zeros_like(x[:, :hq])), move(torch.zeros_like(x[:, :hq]))
        back = [move(torch.zeros_like(x[:, :hkv])) for _ in range(2)]
        err = torch.zeros(1, dtype=torch.int32, device="cuda")
        pa.pa_rope_axes_and_cache(q_out, k, v, q, key, value, po, sl, fr, bytes(j % 3 for j in range(64)), err_flag=err,
                                  k_scale=0.0025, v_scale=0.0031)
        pa.pa_reshape_and_cache_fp4(k, v, key, value, move(slots + 1), 0.0025, 0.0031, err_flag=err)
        pa.pa_decode_fp4(out, q_out, k, v, tab, ln, 0.01, 0.01, 0.01, key=key, value=value, err_flag=err)
        pa.pa_read_cache_fp4(*back, k, v, sl, 0.0025, 0.0031, err_flag=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        got.append([a.cpu() for a in (q_out, out, *back, k, v)])
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(*got)) and bool((got[0][1][1] != 0).any())
