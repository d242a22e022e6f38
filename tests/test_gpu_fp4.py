"""Caches held in 4 bits: write, read, decode steps and chunks, against 64 bits (needs a GB300).

Written bytes are compared with the definition's (every step of it is one fp32 operation).  Attention, per element: keys
and values enter exactly, the weights p_i as fp16 numbers p_i (1 + d_i), |d_i| <= 2^-11, and their sum is that of the
rounded ones, so the result moves by sum w_i d_i (v_i - out), at most 2^-11 max|v|: 2.7e-3 for |v| < 5.5 (normals, whose
groups' largest elements are rounded by up to 1/16).  Rounding it to the output's type adds half a step, which for bf16 is
as much as 2^-9 below 1 (so that over bf16 rows harness.bound's 3e-3 does not hold both: 2.7e-3 + 2^-9 = 4.6e-3); fp32
scores, exponentials and sums add less than 2^-14.
Everything that no query sees has NaN scales, and the
table's entries for blocks without a visible token lie outside the pool.
"""
import numpy as np
import pytest

import oracle as O
import workloads as W
from fp4_ref import K_UNIT, NAN_SCALE, V_UNIT, Fp4Case, pack, quantise, unpack, values
from harness import out_f64, to_numpy_storage, to_torch

pytestmark = pytest.mark.gpu

SENTINEL = 123.0
BIG = None


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


class Step:
    def __init__(self, w: Fp4Case):
        import torch
        self.w = w
        self.k, self.v = torch.from_numpy(w.k_cache).cuda(), torch.from_numpy(w.v_cache).cuda()
        self.q = to_torch(w.q, w.qdt)
        self.table = torch.from_numpy(w.table).cuda()
        self.lens = torch.tensor(w.lens, dtype=torch.int32, device="cuda")
        self.start = torch.from_numpy(w.query_start()).cuda()
        self.nk = to_torch(w.new_key, w.qdt) if w.new_key is not None else None
        self.nv = to_torch(w.new_value, w.qdt) if w.new_value is not None else None
        self.out = torch.full_like(self.q, SENTINEL)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def decode(self, **kw):
        import paged_kv_cache_32_gb300 as pa
        w = self.w
        pa.pa_decode_fp4(self.out, self.q, self.k, self.v, self.table, self.lens, w.scale, K_UNIT, V_UNIT,
                         window=None if w.window >= 2 ** 30 else w.window, num_sinks=w.sinks, key=self.nk, value=self.nv,
                         err_flag=self.err, **kw)
        return self.out

    def prefill(self, max_query_len=None, **kw):
        import paged_kv_cache_32_gb300 as pa
        w = self.w
        pa.pa_prefill_fp4(self.out, self.q, self.k, self.v, self.table, self.lens, self.start,
                          max(w.chunks) if max_query_len is None else max_query_len, w.scale, K_UNIT, V_UNIT,
                          window=None if w.window >= 2 ** 30 else w.window, num_sinks=w.sinks, err_flag=self.err, **kw)
        return self.out


def case(rows, lens, chunks, hq, hkv, block_size, window, sinks, **kw):
    return Fp4Case(rows, lens, chunks, hq, hkv, block_size, 2 ** 31 - 1 if window is None else window, sinks, **kw)


MANTISSA = {"f16": 10, "bf16": 7}


def limit(ref, rows):
    """See above."""
    moved = 5.5 * 2.0 ** -11 + 2.0 ** -14
    e = np.floor(np.log2(np.maximum(np.abs(ref) + moved, 2.0 ** -14)))
    return moved + 2.0 ** (e - MANTISSA[rows] - 1)


def within_bound(got, ref, rows):
    err = np.abs(got - ref)
    ratio = err / limit(ref, rows)
    return bool(np.all(ratio <= 1.0)), float(err.max(initial=0)), float(ratio.max(initial=0))


def check(step, ref, what=""):
    assert int(step.err.item()) == 0, f"{what}: error flag {int(step.err.item())}"
    got = out_f64(step.out)
    assert not np.isnan(got).any(), f"{what}: NaN in the output"
    ok, err, ratio = within_bound(got, ref, step.w.qdt)
    assert ok, f"{what}: max abs err {err}, worst err/bound {ratio}"


# ---------------------------------------------------------------- write and read
def edge_rows(rng, tokens, heads):
    """Normals of many sizes, and rows where the quantisation can go wrong."""
    x = rng.standard_normal((tokens, heads, 128)) * 2.0 ** rng.integers(-12, 3, (tokens, heads, 1))
    flat = x.reshape(-1, 128)
    special = [np.zeros(128), -np.zeros(128), np.full(128, 6.7), np.full(128, -1e4), np.full(128, 1e-7),
               np.where(np.arange(128) % 16 == 3, 5.0, 0.0),          # one element of each group
               np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 16) * K_UNIT * 32,  # ties of a power-of-two scale
               -np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 16) * V_UNIT * 32,
               np.where(np.arange(128) % 32 == 0, np.inf, 1.0), np.linspace(-3, 3, 128)]
    for i, row in enumerate(special[:len(flat)]):
        flat[i] = row
    return x


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("tokens,heads,block_size", [(1, 1, 16), (7, 3, 48), (200, 8, 32), (1000, 2, 256), (64, 5, 16)])
def test_write_and_read(pa, rows, tokens, heads, block_size):
    """The bytes of every slot, others as they were; then the rows that they stand for."""
    import torch
    rng = np.random.default_rng(tokens)
    nb = -(-tokens // block_size) + 2
    with np.errstate(over="ignore"):
        x = [W.to_storage(edge_rows(rng, tokens, heads), rows) for _ in range(2)]
    slots = rng.permutation(nb * block_size)[:tokens].astype(np.int64)
    slots[tokens // 2::9] = -1
    caches = [torch.full((nb, heads, block_size // 16, 1152), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    # views of a fused projection
    fused = torch.zeros((tokens, 2 * heads + 3, 128), dtype=torch.float16 if rows == "f16" else torch.bfloat16, device="cuda")
    fused[:, 1:1 + heads], fused[:, 2 + heads:2 + 2 * heads] = to_torch(x[0], rows), to_torch(x[1], rows)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    at = torch.from_numpy(slots).cuda()
    pa.pa_reshape_and_cache_fp4(*caches, fused[:, 1:1 + heads], fused[:, 2 + heads:2 + 2 * heads], at, K_UNIT, V_UNIT,
                                err_flag=err)
    back = [torch.full((tokens, heads, 128), SENTINEL, dtype=fused.dtype, device="cuda") for _ in range(2)]
    pa.pa_read_cache_fp4(*back, *caches, at, K_UNIT, V_UNIT, err_flag=err)
    assert int(err.item()) == 0
    live = slots >= 0
    blk, off = slots[live] // block_size, slots[live] % block_size
    for cache, src, unit, got in zip(caches, x, (K_UNIT, V_UNIT), back):
        want_c = np.full((nb, heads, block_size, 64), 0x55, np.uint8)
        want_s = np.full((nb, heads, block_size, 8), 0x55, np.uint8)
        c, s = quantise(O.to_f64(src[live], rows), unit)
        want_c[blk, :, off], want_s[blk, :, off] = c, s
        assert np.array_equal(cache.cpu().numpy(), pack(want_c, want_s))
        r = O.to_f64(to_numpy_storage(got, rows), rows)
        assert np.all(r[~live] == SENTINEL)
        # one fp32 product of an exact number and the unit, rounded once
        w32 = (values(c, s, 1.0).astype(np.float32) * np.float32(unit)).astype(np.float64)
        assert np.array_equal(r[live], O.to_f64(W.to_storage(w32, rows), rows))


def test_write_bad_slot_and_copy_blocks(pa):
    import torch
    rng = np.random.default_rng(1)
    key, value = (torch.randn(4, 2, 128, device="cuda", dtype=torch.float16) for _ in range(2))
    k, v = pa.fp4_cache(4, 2, 32), pa.fp4_cache(4, 2, 32)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([5, 4 * 32, 2 ** 40, 33], device="cuda")
    pa.pa_reshape_and_cache_fp4(k, v, key, value, slots, K_UNIT, V_UNIT, err_flag=err)
    assert int(err.item()) == 2
    got = torch.zeros_like(key), torch.zeros_like(value)
    pa.pa_read_cache_fp4(*got, k, v, slots, K_UNIT, V_UNIT)
    assert bool((got[0][1:3] == 0).all()) and bool((got[0][0] != 0).any()) and bool((got[1][3] != 0).any())
    err.zero_()
    pa.pa_copy_blocks(k, v, torch.tensor([[0, 3], [1, 2]], dtype=torch.int32, device="cuda"), err_flag=err,
                      desc=pa.fp4_cache_desc(k))
    assert int(err.item()) == 0 and torch.equal(k[0], k[3]) and torch.equal(v[1], v[2])
    with pytest.raises(pa.PaError):  # an FP8 call over a 4-bit cache
        pa.pa_decode(key, key, k, v, torch.zeros(4, 1, dtype=torch.int32, device="cuda"),
                     torch.ones(4, dtype=torch.int32, device="cuda"), 1.0, desc=pa.fp4_cache_desc(k))


# ---------------------------------------------------------------- decode
LENS = [0, 1, 2, 15, 16, 17, 33, 200, 500, 1031, 1800]


@pytest.mark.parametrize("rows,block_size,hq,hkv", [("f16", 16, 8, 2), ("bf16", 16, 4, 4), ("bf16", 32, 24, 2),
                                                    ("f16", 48, 20, 2), ("bf16", 64, 16, 1), ("f16", 256, 7, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (15, 0), (16, 16), (17, 3), (100, 1), (700, 64), (1500, 900),
                                          (BIG, 0), (300, 2 ** 31 - 1)])
def test_decode(rows, block_size, hq, hkv, window, sinks):
    w = case(rows, LENS, [1] * len(LENS), hq, hkv, block_size, window, sinks, seed=(window or 5) % 97 + sinks % 89)
    s = Step(w)
    s.decode()
    check(s, w.reference(), "decode")


@pytest.mark.parametrize("rows,block_size", [("f16", 16), ("bf16", 32), ("bf16", 48), ("f16", 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 5), (BIG, 0)])
def test_decode_append(pa, rows, block_size, window, sinks):
    """The step's append: the output, the caches bit for bit what the append call writes, nothing else written."""
    import torch
    lens = [1, 2, 16, 17, 300, 0, 1201]
    w = case(rows, lens, [1] * len(lens), 24, 2, block_size, window, sinks, seed=5, append=True)
    s, t = Step(w), Step(w)
    s.decode()
    check(s, w.reference(), "append")
    pos = np.array(lens) - 1
    slots = np.array([w.table[i, p // block_size] * block_size + p % block_size if p >= 0 else -1
                      for i, p in enumerate(pos)], np.int64)
    pa.pa_reshape_and_cache_fp4(t.k, t.v, t.nk, t.nv, torch.from_numpy(slots).cuda(), K_UNIT, V_UNIT, err_flag=t.err)
    assert torch.equal(s.k, t.k) and torch.equal(s.v, t.v)
    t.nk = t.nv = None
    t.decode()  # over the written caches: the same bits
    assert torch.equal(s.out, t.out)


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_decode_many_sequences(rows):
    rng = np.random.default_rng(3)
    for n, hkv, most in ((130, 8, 330), (60, 8, 330), (9, 4, 3000), (40, 2, 2500)):
        lens = [int(x) for x in rng.integers(1, most, n)]
        w = case(rows, lens, [1] * n, 2 * hkv, hkv, 16, 250 if most == 330 else None, 4, seed=n)
        s = Step(w)
        s.decode()
        check(s, w.reference(), f"{n} sequences")


@pytest.mark.parametrize("rows,hkv,append", [("f16", 1, True), ("bf16", 8, False), ("bf16", 4, True), ("f16", 2, False)])
def test_decode_few_long_sequences(rows, hkv, append):
    for lens, window in (([9001], 4200), ([6000], BIG), ([4100, 3], 4096)):
        w = case(rows, lens, [1] * len(lens), hkv * 5, hkv, 16, window, 3, seed=29, append=append)
        s = Step(w)
        s.decode()
        check(s, w.reference(), f"{lens} window {window}")
        import torch
        assert torch.equal(s.out, Step(w).decode())


@pytest.mark.parametrize("rows,hq,hkv,block_size", [("f16", 8, 8, 16), ("bf16", 24, 2, 32), ("bf16", 7, 1, 48)])
def test_decode_workspace(pa, rows, hq, hkv, block_size):
    """Slabs dealt out evenly (no window), empty and bad sequences among them, with a workspace full of NaN and one that a
    captured call keeps; without a workspace the same to rounding."""
    import torch
    rng = np.random.default_rng(hq)
    lens = [0, 5000, 1, 31, 32, 33, 0, 700] + [int(x) for x in rng.integers(1, 900, 30)] + [0]
    # (a table of 40000 tokens: the slabs are dealt out by what it holds)
    w = case(rows, lens, [1] * len(lens), hq, hkv, block_size, BIG, 0, seed=4, slack_blocks=35000 // block_size)
    ref = w.reference()
    ref[[0, 6, -1]] = 0.0
    need = pa.pa_decode_fp4_workspace_size(len(lens), hq, w.width, pa.pa_cache_desc(w.num_blocks, block_size, hkv, 128,
                                                                                    pa.PA_FP4_E2M1))
    assert need > 0
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    s, t = Step(w), Step(w)
    s.decode(workspace=ws)
    check(s, ref, "even")
    assert torch.equal(s.out, Step(w).decode())  # the same bits again
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        t.decode(workspace=ws)
    ws.fill_(0xFF)
    graph.replay()
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0 and torch.equal(s.out, t.out)
    # a bounded wait that runs out is reported, and the workspace is as good as before
    t = Step(w)
    t.decode(workspace=ws, test_flags=pa.PA_DECODE_TEST_EXPIRE_FIRST_WAIT)
    torch.cuda.synchronize()
    assert int(t.err.item()) == 4
    t = Step(w)
    t.decode(workspace=ws)
    assert int(t.err.item()) == 0 and torch.equal(s.out, t.out)
    # a length past the table is reported, the others stay right
    s = Step(w)
    s.lens[3] = 10 ** 6
    s.decode()
    got = out_f64(s.out)
    assert int(s.err.item()) == 5 and np.all(got[3] == SENTINEL)
    ok, err, _ = within_bound(np.delete(got, 3, 0), np.delete(ref, 3, 0), rows)
    assert ok, err
    # the C call without one
    s = Step(w)
    d = pa.fp4_cache_desc(s.k)
    status = pa.lib().pa_decode_fp4(s.out.data_ptr(), s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), None, None,
                                    s.table.data_ptr(), s.lens.data_ptr(), len(lens), hq, w.width, d,
                                    pa.PA_F16 if rows == "f16" else pa.PA_BF16, w.scale, 2 ** 31 - 1, 0, K_UNIT, V_UNIT, None,
                                    0, None, 0, s.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    check(s, ref, "clusters")


@pytest.mark.parametrize("scale", [-0.09, 0.0, 1e-36])
def test_decode_any_scale(scale):
    """Negative scales, and those that leave every token the same weight."""
    for window in (BIG, 50):
        w = case("bf16", [300, 77, 5], [1, 1, 1], 8, 2, 16, window, 0, seed=3)
        w.scale = scale
        s = Step(w)
        s.decode()
        check(s, w.reference(), "scale")


def test_decode_alibi():
    import torch
    slopes = -(2.0 ** -np.arange(1, 13)).astype(np.float32)
    w = case("bf16", [40, 900, 1], [1] * 3, 12, 1, 16, 300, 20, seed=8)
    s = Step(w)
    s.decode(alibi_slopes=torch.from_numpy(slopes).cuda())
    check(s, w.reference(alibi=slopes), "alibi")


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_decode_large_scores(rows):
    w = case(rows, [700, 33, 1500], [1] * 3, 8, 1, 16, 600, 7, seed=12, spread=2.0)
    s = Step(w)
    s.decode()
    check(s, w.reference(), "large scores")


@pytest.mark.parametrize("power", [-120, -30, 30, 100])
def test_decode_bf16_queries_of_any_size(power):
    """Queries far outside fp16's range: the scale brings the scores back."""
    w = case("bf16", [300, 77], [1, 1], 8, 2, 16, BIG, 0, seed=3)
    ref = w.reference()
    w.q = W.to_storage(O.to_f64(w.q, "bf16") * 2.0 ** power, "bf16")
    w.scale *= 2.0 ** -power
    s = Step(w)
    s.decode()
    check(s, ref, "scaled queries")


def test_decode_bad_data(pa):
    """A bad block ID and a length outside the table are reported; the other sequences are right."""
    w = case("bf16", [100, 50, 400, 60], [1] * 4, 8, 2, 16, 64, 4, seed=4)
    ref = w.reference()
    s = Step(w)
    s.table[2, (400 - 64) // 16] = w.num_blocks
    s.decode()
    assert int(s.err.item()) == 1
    ok, err, _ = within_bound(out_f64(s.out)[[0, 1, 3]], ref[[0, 1, 3]], "bf16")
    assert ok, err
    for bad in (w.width * 16 + 1, -3):
        s = Step(w)
        s.lens[1] = bad
        s.decode()
        got = out_f64(s.out)
        assert int(s.err.item()) == 5 and np.all(got[1] == SENTINEL)
        ok, err, _ = within_bound(got[[0, 2, 3]], ref[[0, 2, 3]], "bf16")
        assert ok, err


def test_decode_nan_query_is_a_nan_row():
    w = case("f16", [100, 400], [1] * 2, 8, 2, 16, BIG, 0, seed=4)
    s = Step(w)
    s.q[1, 3, 7] = float("nan")
    s.decode()
    got, ref = out_f64(s.out), w.reference()
    assert np.isnan(got[1, 3]).all()
    got[1, 3] = ref[1, 3]
    assert within_bound(got, ref, "f16")[0]


def test_decode_expired_wait_is_reported(pa):
    import torch
    w = case("f16", [900, 300], [1] * 2, 8, 2, 16, 500, 4, seed=6)
    s = Step(w)
    s.decode(test_flags=pa.PA_DECODE_TEST_EXPIRE_FIRST_WAIT)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 4
    t = Step(w)
    t.decode()
    check(t, w.reference(), "after the expired wait")


# ---------------------------------------------------------------- chunks
CHUNKS = [(1, 1), (5, 5), (133, 130), (3, 0), (0, 0), (500, 1), (700, 77), (1030, 200), (131, 3), (640, 128)]


@pytest.mark.parametrize("rows,block_size,hq,hkv", [("f16", 16, 8, 2), ("bf16", 16, 4, 4), ("bf16", 32, 12, 2),
                                                    ("f16", 48, 6, 1), ("bf16", 64, 16, 1), ("f16", 128, 5, 1),
                                                    ("bf16", 256, 4, 1), ("f16", 80, 8, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (64, 130), (128, 4), (300, 1), (BIG, 0)])
def test_prefill(rows, block_size, hq, hkv, window, sinks):
    lens, chunks = [L for L, c in CHUNKS], [c for L, c in CHUNKS]
    w = case(rows, lens, chunks, hq, hkv, block_size, window, sinks, seed=(window or 3) % 89)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "prefill")


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_prefill_short_chunks(rows):
    lens, chunks = [900, 33, 1200, 9, 64, 4, 700], [5, 1, 3, 9, 2, 4, 0]
    for window, sinks in ((1, 0), (5, 2), (600, 4), (BIG, 0)):
        w = case(rows, lens, chunks, 8, 1, 16, window, sinks, seed=window or 1)
        s = Step(w)
        s.prefill()
        check(s, w.reference(), f"window {window}")


@pytest.mark.parametrize("rows,block_size", [("f16", 16), ("bf16", 32), ("bf16", 48)])
@pytest.mark.parametrize("window,sinks,lens,chunks", [
    (2500, 3, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),
    (BIG, 0, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),
    (4300, 5, [4700, 40], [40, 40]),
    (900, 0, [3000, 1500], [300, 150]),
])
def test_prefill_few_long_items(rows, block_size, window, sinks, lens, chunks):
    import torch
    w = case(rows, lens, chunks, 8, 1, block_size, window, sinks, seed=7)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "few long items")
    assert torch.equal(s.out, Step(w).prefill())


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("seqs,window,sinks", [(24, BIG, 0), (24, 9000, 5), (40, BIG, 0), (40, 8000, 0)])
def test_prefill_unequal_sequences(rows, seqs, window, sinks):
    """More divided items than SMs, of equal and unequal lengths, in a table wide enough for 10000 tokens; the second
    sequence has no queries, the last one is inconsistent."""
    import torch
    rng = np.random.default_rng(seqs)
    chunks = [int(x) for x in rng.integers(1, 25, seqs)]
    lens = [24 + int(x) for x in rng.integers(0, 700, seqs)]
    lens[3:9] = [300] * 6
    lens[seqs - 2] = 1500
    chunks[1], chunks[-1], lens[-1] = 0, 9, 40
    w = case(rows, lens, chunks, 16, 4, 16, window, sinks, seed=seqs)
    ref = w.reference()
    s = Step(w)
    s.table = torch.cat([s.table, torch.full((seqs, 625 - s.table.shape[1]), -3, dtype=torch.int32, device="cuda")], 1)
    s.prefill(max_query_len=24)
    check(s, ref, "unequal sequences")
    bad = Step(w)
    bad.table = s.table
    bad.lens[-1] = 8  # fewer than its queries
    bad.prefill(max_query_len=24)
    assert int(bad.err.item()) == 5 and torch.equal(bad.out[:-9], s.out[:-9])
    assert torch.all(bad.out[-9:] == SENTINEL)


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("seqs,most,window,sinks", [(1, 1300, BIG, 0), (2, 700, 90, 2), (20, 60, BIG, 0), (39, 24, 500, 4),
                                                    (77, 33, BIG, 0), (96, 40, 30, 0), (97, 40, BIG, 0)])
def test_prefill_more_items_than_sms(rows, seqs, most, window, sinks):
    """Whole and partial rounds of items, sequences without queries and one that is inconsistent among them."""
    import torch
    rng = np.random.default_rng(seqs)
    chunks = [most] + [int(x) for x in rng.integers(0, most + 1, seqs - 1)]
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 400, seqs))]
    w = case(rows, lens, chunks, 16, 4, 16, window, sinks, seed=seqs)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "many items")
    assert not torch.any(s.out == SENTINEL)
    start, n = w.query_start(), seqs - 1
    bad = Step(w)
    bad.lens[n] = -1
    bad.prefill()
    assert int(bad.err.item()) == 5 and torch.equal(bad.out[:start[n]], s.out[:start[n]])
    assert torch.all(bad.out[start[n]:] == SENTINEL)


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_prefill_mixed_batch(rows):
    """One prompt among many single tokens (more items in the grid than exist)."""
    rng = np.random.default_rng(2)
    chunks = [1] * 150 + [260] + [1] * 99
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 90, 250))]
    w = case(rows, lens, chunks, 16, 4, 16, BIG, 0, seed=11)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "mixed batch")


@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_prefill_prompt_among_single_tokens(rows):
    """As above, with few enough sequences that their items are dealt out: far more places than items."""
    rng = np.random.default_rng(3)
    chunks = [1] * 60 + [900] + [1] * 35
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 300, 96))]
    w = case(rows, lens, chunks, 16, 4, 32, BIG, 0, seed=12)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "a prompt among single tokens")


def test_prefill_rows_and_bad_chunks():
    """Rows that no chunk owns keep what they held; an inconsistent chunk is reported and skipped."""
    import torch
    w = case("bf16", [300, 200, 90], [140, 60, 7], 8, 2, 16, 100, 4, seed=9)
    ref = w.reference()
    s = Step(w)
    pad = torch.full((50, 8, 128), SENTINEL, dtype=s.q.dtype, device="cuda")
    s.q, s.out = torch.cat([s.q, pad]), torch.cat([s.out, pad])
    s.prefill()
    got = out_f64(s.out)
    assert int(s.err.item()) == 0 and np.all(got[207:] == SENTINEL)
    assert within_bound(got[:207], ref, "bf16")[0]
    for lens, most in (([300, 59, 90], 140), ([300, 5000, 90], 140)):
        s = Step(w)
        s.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s.prefill(max_query_len=most)
        got = out_f64(s.out)
        assert int(s.err.item()) == 5 and np.all(got[140:200] == SENTINEL)
        assert within_bound(np.delete(got, range(140, 200), 0), np.delete(ref, range(140, 200), 0), "bf16")[0]


def test_prefill_bad_block():
    w = case("f16", [300, 200, 90], [140, 60, 7], 8, 2, 16, BIG, 0, seed=9)
    s = Step(w)
    s.table[1, 2] = -5
    s.prefill()
    got, ref = out_f64(s.out), w.reference()
    assert int(s.err.item()) == 1
    assert within_bound(got[:140], ref[:140], "f16")[0] and within_bound(got[200:], ref[200:], "f16")[0]


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("chunk", [3, 200])
def test_prefill_scales_and_nan(rows, chunk):
    """A scale that leaves every visible token the same weight; a NaN query is a NaN row and no other."""
    w = case(rows, [300, 260], [chunk, chunk], 8, 2, 16, 150, 3, seed=3)
    w.scale = 1e-36
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "tiny scale")
    w = case(rows, [300, 260], [chunk, chunk], 8, 2, 16, BIG, 0, seed=5)
    s = Step(w)
    s.q[chunk + 1, 5, 99] = float("nan")
    s.prefill()
    got, ref = out_f64(s.out), w.reference()
    assert int(s.err.item()) == 0 and np.isnan(got[chunk + 1, 5]).all()
    got[chunk + 1, 5] = ref[chunk + 1, 5]
    assert within_bound(got, ref, rows)[0]


@pytest.mark.parametrize("power", [-100, 90])
def test_prefill_bf16_queries_of_any_size(power):
    w = case("bf16", [300, 177], [150, 130], 8, 2, 16, BIG, 0, seed=3)
    ref = w.reference()
    w.q = W.to_storage(O.to_f64(w.q, "bf16") * 2.0 ** power, "bf16")
    w.scale *= 2.0 ** -power
    s = Step(w)
    s.prefill()
    check(s, ref, "scaled queries")


# ---------------------------------------------------------------- streams and graphs
def test_captured_step_on_another_stream(pa):
    """Write and attention captured in a graph on a stream of their own, replayed over changed inputs."""
    import torch
    w = case("bf16", [300, 77, 1500], [1] * 3, 16, 2, 32, BIG, 0, seed=13, append=True)
    s = Step(w)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        s.decode()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.decode()
    torch.cuda.synchronize()
    s.out.fill_(SENTINEL)
    graph.replay()
    torch.cuda.synchronize()
    check(s, w.reference(), "replay")
    first = s.out.clone()
    s.q.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(first, s.out)
