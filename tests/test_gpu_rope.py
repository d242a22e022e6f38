"""Rotary positions with the cache write, against fp64 or better (needs a GB300).

Bound per element, derived: y = c x_a -+ s x_b in fp32 from c, s that are within 2^-22 of magnitude * cos, sin (an
angle fraction off by 2^-24 of a half turn, pi 2^-24 radians; sincospif within 2 ulp, 2^-23; the product with the
magnitude 2^-24), two products and a sum off by 2^-24 each: at most (|x_a| + |x_b|) * magnitude * 2^-21, plus the
rounding to the output type, finfo.eps / 2 of |y|.  The angle's fraction comes from f / 2 pi in 64 bits: its
relative error of 2^-52 moves an angle by |position| f 2^-52.
"""
import numpy as np
import pytest

import oracle as O
import workloads as W
from harness import to_numpy_storage, to_torch
from window_ref import CODE_VALUES, K_SCALE, V_SCALE

pytestmark = pytest.mark.gpu

HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


def turned(x, pos, inv_freq, magnitude, interleaved):
    """(y, bound on |got - y| before the output's rounding) for x [tokens, heads, D] in fp64."""
    r = 2 * len(inv_freq)
    ang = pos.astype(np.longdouble)[:, None] * inv_freq.astype(np.longdouble)[None]
    ang = np.remainder(ang, 2 * PI).astype(np.float64)
    c, s = np.cos(ang)[:, None] * magnitude, np.sin(ang)[:, None] * magnitude
    a = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    b = a + 1 if interleaved else a + r // 2
    y, e = x.copy(), np.zeros_like(x)
    y[..., a] = c * x[..., a] - s * x[..., b]
    y[..., b] = c * x[..., b] + s * x[..., a]
    size = (np.abs(x[..., a]) + np.abs(x[..., b])) * magnitude
    off = size * (2.0 ** -21 + (np.abs(pos.astype(np.float64))[:, None] * np.abs(inv_freq) * 2.0 ** -52)[:, None])
    e[..., a] = off
    e[..., b] = off
    return y, e


PI = np.longdouble("3.14159265358979323846264338327950288")


class Rope:
    def __init__(self, pa, dtype, tokens, hq, hkv, d, block_size, rotary, interleaved, *, seed=0, positions=None,
                 method=0, fused=True, padding=(), magnitude=None, base=10000.0):
        import torch
        rng = np.random.default_rng(seed)
        self.pa, self.dtype, self.hq, self.hkv, self.d, self.B = pa, dtype, hq, hkv, d, block_size
        self.t = "f16" if dtype == "fp8" else dtype
        self.interleaved = interleaved
        x = W.to_storage(rng.standard_normal((tokens, hq + 2 * hkv, d)), self.t)
        self.x = O.to_f64(x, self.t)
        dev = to_torch(x, self.t)
        if not fused:
            self.q, self.key, self.value = (t.contiguous() for t in (dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]))
        else:
            self.q, self.key, self.value = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
        self.num_blocks = -(-tokens // block_size) + 2
        shape = (self.num_blocks, hkv, block_size, d)
        if dtype == "fp8":
            self.k = torch.full(shape, 0x55, dtype=torch.uint8, device="cuda")
            self.v = torch.full((self.num_blocks, hkv, block_size // 16, d, 16), 0x55, dtype=torch.uint8, device="cuda")
        else:
            self.k = torch.full(shape, 7.0, dtype=dev.dtype, device="cuda")
            self.v = torch.full(shape, 7.0, dtype=dev.dtype, device="cuda")
        self.slots = rng.permutation(self.num_blocks * block_size)[:tokens].astype(np.int64)
        self.slots[list(padding)] = -1
        self.pos = (rng.integers(0, 200000, tokens) if positions is None else np.resize(positions, tokens)).astype(np.int32)
        self.inv, mag = pa.pa_rope_frequencies(rotary, base, method, factor=8.0, original_max_position=4096.0)
        self.mag = mag if magnitude is None else magnitude
        self.q_out = torch.full((tokens, hq, d), 9.0, dtype=dev.dtype, device="cuda")
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, **kw):
        import torch
        self.pa.pa_rope_and_cache(self.q_out if self.hq else None, self.k, self.v, self.q if self.hq else None, self.key,
                                  self.value, torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.slots).cuda(),
                                  self.inv.cuda(), interleaved=self.interleaved, magnitude=self.mag, err_flag=self.err,
                                  k_scale=K_SCALE if self.dtype == "fp8" else None,
                                  v_scale=V_SCALE if self.dtype == "fp8" else None, **kw)

    def check(self, q_rows=None):
        """Queries, keys and values of every token with a slot; everything else as it was."""
        assert int(self.err.item()) == 0
        hq, hkv, B = self.hq, self.hkv, self.B
        y, e = turned(self.x, self.pos, self.inv.numpy(), self.mag, self.interleaved)
        live = self.slots >= 0
        q = O.to_f64(to_numpy_storage(self.q_out if q_rows is None else q_rows, self.t), self.t)
        step = HALF_STEP[self.t]
        tiny = 2.0 ** -25 if self.t == "f16" else 0.0  # half of fp16's smallest step
        if hq:
            assert np.all(np.abs(q - y[:, :hq])[live] <= (step * np.abs(y[:, :hq]) * (1 + 2 ** -8) + e[:, :hq] + tiny)[live])
            if q_rows is None:
                assert np.all(q[~live] == 9.0)
        blk, off = self.slots[live] // B, self.slots[live] % B
        ky, ke, vy = y[live, hq:hq + hkv], e[live, hq:hq + hkv], self.x[live, hq + hkv:]
        if self.dtype == "fp8":
            k, v = self.k.cpu().numpy(), self.v.cpu().numpy()
            got = CODE_VALUES[k[blk, :, off]]
            want = np.clip(ky / np.float64(np.float32(K_SCALE)), -448, 448)
            spacing = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(want), 2.0 ** -9))), -6) - 3)
            # half a step, the fp32 result's error, its division's rounding
            lim = spacing / 2 + ke / K_SCALE + np.abs(want) * 2.0 ** -22
            assert np.all(np.abs(got - want) <= lim)
            code = np.asarray(O.quantize_e4m3((vy.astype(np.float32) / np.float32(V_SCALE)).astype(np.float64)),
                              np.uint8).reshape(vy.shape)
            assert np.array_equal(v[blk, :, off // 16, :, off % 16], code)
            k[blk, :, off] = 0x55
            v[blk, :, off // 16, :, off % 16] = 0x55
            assert np.all(k == 0x55) and np.all(v == 0x55)
        else:
            k = O.to_f64(to_numpy_storage(self.k, self.t), self.t)
            v = O.to_f64(to_numpy_storage(self.v, self.t), self.t)
            assert np.all(np.abs(k[blk, :, off] - ky) <= step * np.abs(ky) * (1 + 2 ** -8) + ke + tiny)
            assert np.array_equal(v[blk, :, off], vy)
            k[blk, :, off] = 7.0
            v[blk, :, off] = 7.0
            assert np.all(k == 7.0) and np.all(v == 7.0)


@pytest.mark.parametrize("dtype,d,block_size", [("f32", 64, 5), ("f32", 128, 16), ("f16", 128, 8), ("f16", 64, 16),
                                                ("bf16", 128, 32), ("bf16", 64, 8), ("fp8", 128, 16), ("fp8", 128, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [2, 6, 18, 20, 24, 32, 48, 64, 128])
def test_rope(pa, dtype, d, block_size, interleaved, rotary):
    if rotary > d:
        rotary = d - 2
    for tokens, hq, hkv in ((1, 7, 1), (3, 8, 2), (67, 4, 4), (500, 12, 2)):
        r = Rope(pa, dtype, tokens, hq, hkv, d, block_size, rotary, interleaved, seed=tokens + rotary)
        r.run()
        r.check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "fp8"])
@pytest.mark.parametrize("method", [0, 1, 2, 3, 4])
def test_rope_scalings_and_far_positions(pa, dtype, method):
    pos = np.array([0, 1, -1, 4095, 4096, 131071, 1048575, 16777217, 2 ** 31 - 1, -2 ** 31], np.int64).astype(np.int32)
    r = Rope(pa, dtype, 40, 8, 2, 128, 16, 128, False, seed=method, positions=pos, method=method, base=500000.0)
    r.run()
    r.check()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_rope_prompt(pa, dtype):
    """A long prompt (several units a thread), dense inputs and views of a fused projection, few heads."""
    for tokens, hq, hkv, fused in ((3001, 16, 2, True), (3001, 16, 2, False), (9000, 1, 1, True), (9000, 0, 1, True)):
        r = Rope(pa, dtype, tokens, hq, hkv, 128, 16, 128, False, seed=tokens, fused=fused)
        r.run()
        r.check()


@pytest.mark.parametrize("dtype", ["f16", "fp8"])
def test_rope_prompt_runs_of_slots(pa, dtype):
    """Tokens of prompts in order: slots run on inside blocks that start and end anywhere."""
    import torch
    r = Rope(pa, dtype, 1000, 8, 2, 128, 32, 64, True, seed=3)
    lens, at, n = [1, 15, 16, 17, 100, 333, 18, 500], 0, 0
    for i, L in enumerate(lens):
        first = 5 * i % 16
        slots = np.arange(n * 32 + first, n * 32 + first + L)
        r.slots[at:at + L] = slots
        at, n = at + L, n + -(-(first + L) // 32)
    assert at == 1000
    r.num_blocks = n
    r.k, r.v = r.k[:1].repeat(n, 1, 1, 1), r.v[:1].repeat(n, *([1] * (r.v.dim() - 1)))
    r.run()
    r.check()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,hq,tokens", [("fp8", 8, 200), ("fp8", 8, 1000), ("fp8", 58, 2600), ("bf16", 60, 2600),
                                             ("f32", 60, 2700), ("f16", 73, 2500)])
def test_rope_prompts_with_holes(pa, dtype, hq, tokens):
    """Prompts over shuffled blocks, with padding and slots outside the pool between and inside them; enough tokens
    that groups of several are cut into parts."""
    B = 32
    r = Rope(pa, dtype, tokens, hq, 2, 128, B, 128, tokens % 200 == 0, seed=tokens + hq)
    rng = np.random.default_rng(tokens)
    r.num_blocks = tokens // B + 64
    r.k, r.v = r.k[:1].repeat(r.num_blocks, 1, 1, 1), r.v[:1].repeat(r.num_blocks, *([1] * (r.v.dim() - 1)))
    blocks, at, free = rng.permutation(r.num_blocks), 0, 0
    while at < tokens:
        length = min(int(rng.choice([1, 3, 16, 31, 47, 200])), tokens - at)
        first = int(rng.integers(0, B)) if free + 8 < len(blocks) - (tokens - at) // B else 0
        for _ in range(length):
            if at == tokens or free == len(blocks):
                break
            r.slots[at] = blocks[free] * B + first
            at, first = at + 1, first + 1
            if first == B:
                first, free = 0, free + 1
        free += first > 0
        if free >= len(blocks):
            break
    r.slots[at:] = -1
    assert at > tokens // 2
    live = r.slots[r.slots >= 0]
    assert len(np.unique(live)) == len(live)
    holes = rng.choice(tokens, tokens // 12, replace=False)
    r.slots[holes] = -1
    bad = rng.choice(at, 9, replace=False)
    good = r.slots.copy()
    r.slots[bad[:6]], r.slots[bad[6:]] = r.num_blocks * B, 2 ** 62
    r.run()
    assert int(r.err.item()) == 2
    r.err.zero_()
    r.slots = good
    r.slots[bad] = -1
    r.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_rope_in_place_and_padding(pa, dtype):
    r = Rope(pa, dtype, 37, 8, 2, 128, 16, 96, False, seed=4, padding=(0, 5, 36))
    before = r.q.clone()
    r.run()
    r.check()
    r.q_out = r.q  # a view of the fused projection, in place
    r.run()
    live = r.slots >= 0
    assert np.array_equal(to_numpy_storage(r.q[~live], r.t), to_numpy_storage(before[~live], r.t))
    r.check(q_rows=r.q)


def test_rope_bad_slot_is_reported_and_skipped(pa):
    r = Rope(pa, "bf16", 10, 4, 2, 128, 16, 128, False, seed=4)
    good = r.slots.copy()
    r.slots[3] = r.num_blocks * 16
    r.slots[7] = 2 ** 62
    r.run()
    assert int(r.err.item()) == 2
    r.err.zero_()
    r.slots = good
    r.slots[[3, 7]] = -1
    r.check()


def test_rope_then_window_step(pa):
    """The path as it is used: prompt chunks, then decode steps, each rope + cache write followed by attention;
    the whole against fp64 on the rounded keys."""
    import torch
    rng = np.random.default_rng(0)
    hq, hkv, d, B, window, sinks = 8, 2, 128, 16, 48, 4
    bm = pa_block_manager(64, B)
    seqs, chunks = [1, 2, 3], [70, 5, 33]
    k = torch.zeros((64, hkv, B, d), dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    inv, mag = pa.pa_rope_frequencies(d, 10000.0, pa.PA_ROPE_LINEAR, factor=2.0, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    keys, values = {s: [] for s in seqs}, {s: [] for s in seqs}

    def step(counts, first):
        """New tokens of each sequence (counts), from position first[s]; returns nothing, checks the outputs."""
        T = sum(counts)
        qkv = torch.from_numpy(rng.standard_normal((T, hq + 2 * hkv, d)).astype(np.float32)).to("cuda", torch.bfloat16)
        tables, lens = bm.build_tables(seqs)
        pos = np.concatenate([np.arange(f, f + c) for f, c in zip(first, counts)]).astype(np.int32)
        row = np.repeat(np.arange(len(seqs)), counts)
        slots = tables[row, pos // B].astype(np.int64) * B + pos % B
        q = torch.empty((T, hq, d), dtype=torch.bfloat16, device="cuda")
        pa.pa_rope_and_cache(q, k, v, qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:],
                             torch.from_numpy(pos).cuda(), torch.from_numpy(slots).cuda(), inv, err_flag=err)
        out = torch.empty_like(q)
        t, n = torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()
        if max(counts) == 1:
            pa.pa_decode_window(out, q, k, v, t, n, d ** -0.5, window, num_sinks=sinks, err_flag=err)
        else:
            start = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device="cuda")
            pa.pa_prefill_window(out, q, k, v, t, n, start, max(counts), d ** -0.5, window, num_sinks=sinks, err_flag=err)
        assert int(err.item()) == 0
        x = qkv.double().cpu().numpy()
        y, _ = turned(x[:, :hq + hkv], pos, inv.cpu().numpy(), mag, False)
        for i, s in enumerate(row):
            keys[seqs[s]].append(y[i, hq:])
            values[seqs[s]].append(x[i, hq + hkv:])
        got = out.double().cpu().numpy()
        for i, s in enumerate(row):
            p = pos[i]
            see = np.array([j for j in range(p + 1) if j > p - window or j < sinks])
            kk = np.repeat(np.stack([keys[seqs[s]][j] for j in see]), hq // hkv, 1)
            vv = np.repeat(np.stack([values[seqs[s]][j] for j in see]), hq // hkv, 1)
            sc = np.einsum("hd,thd->ht", y[i, :hq], kk) * d ** -0.5
            w = np.exp(sc - sc.max(1, keepdims=True))
            want = np.einsum("ht,thd->hd", w / w.sum(1, keepdims=True), vv)
            # q and k are rounded to bf16 (2^-8 of an element each): a score moves by at most
            # 2 * 2^-8 * sum |q k| d^-1/2 (measured here below 12), a weight by e^x - 1 of that, the output by
            # twice max|v| of it; plus the output's own half step
            ds = 2.0 ** -7 * (np.einsum("hd,thd->ht", np.abs(y[i, :hq]), np.abs(kk)) * d ** -0.5).max()
            lim = 2 * np.expm1(ds) * np.abs(vv).max() + 2.0 ** -8 * np.abs(want) + 2.0 ** -12
            assert np.all(np.abs(got[i] - want) <= lim)

    for s, c in zip(seqs, chunks):
        bm.allocate(s, c)
    step(chunks, [0, 0, 0])
    at = list(chunks)
    for _ in range(20):
        bm.append_slots(seqs)
        step([1, 1, 1], at)
        at = [a + 1 for a in at]


def pa_block_manager(n, b):
    from paged_kv_cache_32_gb300.block_manager import BlockManager
    return BlockManager(n, b, shuffle_seed=5)


def test_rope_graph_replay(pa):
    import torch
    r = Rope(pa, "bf16", 24, 8, 2, 128, 16, 128, False, seed=1)
    pos, slots, inv = torch.from_numpy(r.pos).cuda(), torch.from_numpy(r.slots).cuda(), r.inv.cuda()

    def call():
        pa.pa_rope_and_cache(r.q_out, r.k, r.v, r.q, r.key, r.value, pos, slots, inv, magnitude=r.mag, err_flag=r.err)

    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    r.pos = (r.pos + 12345).astype(np.int32)
    pos.copy_(torch.from_numpy(r.pos))
    g.replay()
    torch.cuda.synchronize()
    r.check()


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_rope_pinned_host_arrays(pa, dtype):
    """The step's rows, positions and slots in pinned host memory."""
    import torch
    r = Rope(pa, dtype, 21, 8, 2, 128, 16, 64, False, seed=6, fused=False)
    r.q, r.key, r.value, r.q_out = (t.cpu().pin_memory() for t in (r.q, r.key, r.value, r.q_out))
    r.run()
    torch.cuda.synchronize()
    r.check()


def test_rope_refuses_wrong_tensors(pa):
    import torch
    r = Rope(pa, "bf16", 5, 8, 2, 128, 16, 128, False, seed=6)
    good = dict(q_out=r.q_out, k_cache=r.k, v_cache=r.v, q=r.q, key=r.key, value=r.value,
                positions=torch.from_numpy(r.pos).cuda(), slot_mapping=torch.from_numpy(r.slots).cuda(),
                inv_freq=r.inv.cuda())
    for kw, error in ((dict(q=r.q.half()), TypeError), (dict(positions=good["positions"].long()), TypeError),
                      (dict(slot_mapping=good["slot_mapping"].int()), TypeError),
                      (dict(inv_freq=good["inv_freq"].float()), TypeError), (dict(inv_freq=r.inv), ValueError),
                      (dict(q=None), ValueError), (dict(key=r.key.cpu()), ValueError), (dict(value=r.value[:4]), ValueError),
                      (dict(key=r.key.transpose(0, 1)), ValueError), (dict(key=r.key[..., ::2]), ValueError),
                      (dict(q=r.q[:, ::2], q_out=r.q_out[:, ::2]), ValueError),
                      (dict(positions=good["positions"][:3]), ValueError),
                      (dict(k_cache=r.k[0]), ValueError),
                      (dict(q_out=r.key.expand(-1, -1, -1), q=r.q[:, :2]), pa.PaError)):  # q_out on the keys
        with pytest.raises(error):
            pa.pa_rope_and_cache(**{**good, **kw})
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,num_blocks", [("bf16", 140000), ("fp8", 270000)])
def test_rope_large_pool(pa, dtype, num_blocks):
    """Slots past 2^31 elements (2^32 bytes) of the caches: the last blocks take what a small pool takes."""
    import torch
    r = Rope(pa, dtype, 100, 8, 8, 128, 16, 128, False, seed=2)
    t = Rope(pa, dtype, 100, 8, 8, 128, 16, 128, False, seed=2)
    r.run()
    small, shift = t.num_blocks, num_blocks - t.num_blocks
    first = t.k[:1], t.v[:1]
    t.k = torch.zeros((num_blocks, *t.k.shape[1:]), dtype=t.k.dtype, device="cuda")
    t.v = torch.zeros((num_blocks, *t.v.shape[1:]), dtype=t.v.dtype, device="cuda")
    t.k[shift:], t.v[shift:] = first[0], first[1]
    t.slots = t.slots + shift * 16
    t.run()
    assert int(t.err.item()) == 0
    assert torch.equal(t.k[shift:], r.k) and torch.equal(t.v[shift:], r.v) and torch.equal(t.q_out, r.q_out)
    assert torch.count_nonzero(t.k[:small]) == 0 and torch.count_nonzero(t.v[:small]) == 0
    del t
    torch.cuda.empty_cache()
