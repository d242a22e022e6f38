"""Decode steps and chunks with a sliding window and first tokens that stay visible, against fp64 (needs a GB300).

Bar: harness.bound per element (1e-5 for fp32; 3e-3, or half an output ulp + 2^-12 where that is more, for fp16 and
bf16, which the FP8 caches' fp16 outputs share: their one-term fp16 weights are off by at most 2^-12 of a weight
each, and their sum is that of the rounded weights, so the output moves by at most 2 * 2^-12 max|v|, 2.5e-3 for
|v| < 5).  Everything that no query sees is NaN, and the table's entries for blocks without a visible token lie
outside the pool, so a read of either shows in the output or in the error flag.
"""
import numpy as np
import pytest

import workloads as W
from harness import out_f64, to_numpy_storage, to_torch, within_bound
from window_ref import K_SCALE, V_SCALE, WindowCase

pytestmark = pytest.mark.gpu

SENTINEL = 123.0
BIG = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


class Step:
    def __init__(self, w: WindowCase, device="cuda"):
        import torch
        self.w = w
        cdt = "f16" if w.dtype == "fp8" else w.dtype
        self.k = torch.from_numpy(w.k_cache).to(device) if w.dtype == "fp8" else to_torch(w.k_cache, cdt, device)
        self.v = torch.from_numpy(w.v_cache).to(device) if w.dtype == "fp8" else to_torch(w.v_cache, cdt, device)
        self.q = to_torch(w.q, w.qdt, device)
        self.table = torch.from_numpy(w.table).to(device)
        self.lens = torch.tensor(w.lens, dtype=torch.int32, device=device)
        self.start = torch.from_numpy(w.query_start()).to(device)
        self.nk = to_torch(w.new_key, w.qdt, device) if w.new_key is not None else None
        self.nv = to_torch(w.new_value, w.qdt, device) if w.new_value is not None else None
        self.out = torch.full_like(self.q, SENTINEL)
        self.err = torch.zeros(1, dtype=torch.int32, device=device)
        self.scales = dict(k_scale=K_SCALE, v_scale=V_SCALE) if w.dtype == "fp8" else {}

    def decode(self, **kw):
        import paged_kv_cache_32_gb300 as pa
        w = self.w
        pa.pa_decode_window(self.out, self.q, self.k, self.v, self.table, self.lens, w.scale, w.window,
                            num_sinks=w.sinks, key=self.nk, value=self.nv, err_flag=self.err, **self.scales, **kw)
        return self.out

    def prefill(self, max_query_len=None, **kw):
        import paged_kv_cache_32_gb300 as pa
        w = self.w
        pa.pa_prefill_window(self.out, self.q, self.k, self.v, self.table, self.lens, self.start,
                             max(w.chunks) if max_query_len is None else max_query_len, w.scale, w.window,
                             num_sinks=w.sinks, err_flag=self.err, **self.scales, **kw)
        return self.out


def check(step, ref, what):
    assert int(step.err.item()) == 0, f"{what}: error flag {int(step.err.item())}"
    got = out_f64(step.out)
    assert not np.isnan(got).any(), f"{what}: NaN in the output"
    ok, err, ratio = within_bound(got, ref, step.w.qdt)
    assert ok, f"{what}: max abs err {err}, worst err/bound {ratio}"


# ---------------------------------------------------------------- decode
LENS = [0, 1, 2, 15, 16, 17, 33, 200, 500, 1031, 1800]
CACHES = [("f32", 64, 5), ("f32", 128, 16), ("f16", 128, 8), ("f16", 64, 8), ("f16", 128, 16), ("bf16", 64, 16),
          ("bf16", 128, 32), ("bf16", 128, 8), ("bf16", 128, 256), ("fp8", 128, 16), ("fp8", 128, 48), ("fp8", 128, 64)]
WINDOWS = [(1, 0), (1, 4), (15, 0), (16, 16), (17, 3), (100, 1), (700, 64), (1500, 900), (BIG, 0), (300, BIG)]


@pytest.mark.parametrize("dtype,d,block_size", CACHES)
@pytest.mark.parametrize("window,sinks", WINDOWS)
def test_decode_window(dtype, d, block_size, window, sinks):
    hq, hkv = {8: (8, 2), 16: (4, 4), 5: (6, 2), 32: (24, 2), 256: (7, 1), 48: (24, 2), 64: (16, 2)}[block_size]
    w = WindowCase(dtype, LENS, [1] * len(LENS), hq, hkv, d, block_size, window, sinks, seed=window % 97 + sinks % 89)
    s = Step(w)
    s.decode()
    ref = w.reference()
    ref[0] = 0.0  # an empty sequence writes zeros
    check(s, ref, "decode")


@pytest.mark.parametrize("dtype,d,block_size", [("f16", 128, 16), ("f16", 64, 8), ("bf16", 128, 32), ("fp8", 128, 16),
                                                ("fp8", 128, 64)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (40, 5), (700, 64)])
def test_decode_window_append(pa, dtype, d, block_size, window, sinks):
    """The step's append: the output, the caches bit for bit what the append call writes, nothing else written."""
    import torch
    lens = [1, 2, 16, 17, 300, 0, 1201]
    w = WindowCase(dtype, lens, [1] * len(lens), 24, 2, d, block_size, window, sinks, seed=5, append=True)
    s, t = Step(w), Step(w)
    s.decode()
    ref = w.reference()
    ref[5] = 0.0
    check(s, ref, "append")
    pos = np.array(lens) - 1
    slots = np.array([w.table[i, p // block_size] * block_size + p % block_size if p >= 0 else -1
                      for i, p in enumerate(pos)], np.int64)
    args = (t.k, t.v, t.nk, t.nv, torch.from_numpy(slots).cuda())
    if dtype == "fp8":
        pa.pa_reshape_and_cache_fp8(*args, K_SCALE, V_SCALE, err_flag=t.err)
    else:
        pa.pa_reshape_and_cache(*args, err_flag=t.err)
    for a, b in ((s.k, t.k), (s.v, t.v)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    t.nk = t.nv = None
    t.decode()  # over the written caches: the same bits
    assert torch.equal(s.out, t.out)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "fp8", "f32"])
def test_decode_window_many_sequences(dtype):
    """Enough items that an item's keys stay with one CTA, or two (the split goes by the size of the grid)."""
    rng = np.random.default_rng(3)
    for n, hkv in ((130, 8), (60, 8)):
        lens = [int(x) for x in rng.integers(1, 330, n)]
        w = WindowCase(dtype, lens, [1] * n, 2 * hkv, hkv, 128, 16, 250, 4, seed=n)
        s = Step(w)
        s.decode()
        check(s, w.reference(), f"{n} sequences")


def test_decode_window_many_long_sequences():
    """fp32: more items than the SMs hold, long enough to be split all the same."""
    rng = np.random.default_rng(5)
    lens = [int(x) for x in rng.integers(1, 2600, 60)]
    w = WindowCase("f32", lens, [1] * 60, 8, 8, 64, 16, 2400, 4, seed=31)
    s = Step(w)
    s.decode()
    check(s, w.reference(), "f32, 480 items")


@pytest.mark.parametrize("dtype,hkv,append", [("f32", 2, False), ("f16", 1, True), ("bf16", 8, False), ("bf16", 4, True),
                                              ("fp8", 8, True), ("fp8", 2, False)])
def test_decode_window_few_long_sequences(dtype, hkv, append):
    """One sequence over thousands of keys: an item's keys go to the largest clusters."""
    for lens, window in (([9001], 4200), ([6000], BIG), ([4100], 4096)):
        w = WindowCase(dtype, lens, [1], hkv * 5, hkv, 128, 16, window, 3, seed=29, append=append)
        s = Step(w)
        ref = w.reference()
        s.decode()
        check(s, ref, f"{dtype} {lens} window {window}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_decode_window_alibi(dtype):
    import torch
    w = WindowCase(dtype, [40, 900, 1], [1] * 3, 12, 1, 128, 16, 300, 20, seed=8)
    slopes = -(2.0 ** -np.arange(1, 13)).astype(np.float32)
    s = Step(w)
    s.decode(alibi_slopes=torch.from_numpy(slopes).cuda())
    ref = w.reference(alibi=slopes)
    if dtype == "f32":
        # Scores here reach 0.5 * 900 = 450, 650 in log2 units, where the fp32 sum of score and bias is rounded by up to
        # 2^-15 and the slope's own rounding (2^-24 of it) moves the bias by 650 * 2^-24: a weight is off by up to
        # ln 2 * (2^-15 + 650 * 2^-24) = 4.8e-5 of itself, the output by twice that times max|v| < 5.
        err = np.max(np.abs(out_f64(s.out) - ref))
        assert int(s.err.item()) == 0 and err <= 2 * 5 * 4.8e-5, err
    else:
        check(s, ref, "alibi")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "fp8"])
def test_decode_window_large_scores(dtype):
    """Scores of hundreds: the running maxima move, far weights vanish."""
    w = WindowCase(dtype, [700, 33, 1500], [1] * 3, 8, 1, 128, 16, 600, 7, seed=12, spread=3.0)
    s = Step(w)
    s.decode()
    # fp32 products of scores s are off by up to 2^-24 * D * |q k| a term: far below the 16-bit bound; for fp32
    # outputs a score of |s| <= 300 (|q| |k| scale = 9 * 128 / 11.3 = 102 typical) is off by up to
    # 2^-23 * 300 = 3.6e-5 from its rounding alone, and the output by twice that times max|v| < 5
    if dtype == "f32":
        got, ref = out_f64(s.out), w.reference()
        assert int(s.err.item()) == 0 and np.max(np.abs(got - ref)) <= 2 * 5 * 300 * 2.0 ** -23
    else:
        check(s, w.reference(), "large scores")


def test_decode_window_whole_context_is_decode(pa):
    """A window past every length gives pa_decode's result."""
    import torch
    lens = [5, 77, 640]
    w = WindowCase("bf16", lens, [1] * 3, 16, 2, 128, 16, 640, 0, seed=2)
    s, t = Step(w), Step(w)
    s.decode()
    # pa_decode reads its last slab whole: nothing but NaN there, as here
    pa.pa_decode(t.out, t.q, t.k, t.v, t.table, t.lens, w.scale, err_flag=t.err)
    a, b = out_f64(s.out), out_f64(t.out)
    assert int(s.err.item()) == 0 and int(t.err.item()) == 0
    assert np.max(np.abs(a - b)) <= 2 * 3e-3
    assert torch.equal(s.out, Step(w).decode())  # and the same bits again


def test_decode_window_bad_data():
    """A bad block ID and a length outside the table are reported; the other sequences are right, and a sequence
    with a bad length is left as it was."""
    import torch
    w = WindowCase("bf16", [100, 50, 400, 60], [1] * 4, 8, 2, 128, 16, 64, 4, seed=4)
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
        assert int(s.err.item()) == 5
        got = out_f64(s.out)
        assert np.all(got[1] == SENTINEL)
        ok, err, _ = within_bound(got[[0, 2, 3]], ref[[0, 2, 3]], "bf16")
        assert ok, err
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", ["f16", "fp8"])
def test_decode_window_expired_wait_is_reported(pa, dtype):
    """A bounded wait that runs out ends the call with a status; the next call is unaffected."""
    import torch
    w = WindowCase(dtype, [900, 300], [1] * 2, 8, 2, 128, 16, 500, 4, seed=6)
    s = Step(w)
    s.decode(test_flags=pa.PA_DECODE_TEST_EXPIRE_FIRST_WAIT)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 4
    t = Step(w)
    t.decode()
    check(t, w.reference(), "after the expired wait")


# ---------------------------------------------------------------- chunks
CHUNK_CACHES = [("f32", 64, 5, 6, 2), ("f32", 128, 16, 3, 3), ("f16", 64, 8, 8, 2), ("f16", 128, 8, 8, 2),
                ("f16", 128, 16, 4, 4), ("f16", 128, 128, 5, 1), ("bf16", 64, 32, 8, 1), ("bf16", 128, 16, 8, 1),
                ("bf16", 128, 32, 12, 2), ("bf16", 128, 64, 16, 1), ("bf16", 128, 96, 4, 2), ("bf16", 128, 256, 4, 1),
                ("fp8", 128, 16, 8, 2), ("fp8", 128, 48, 6, 1), ("fp8", 128, 64, 4, 4)]
CHUNKS = [(1, 1), (5, 5), (133, 130), (3, 0), (0, 0), (500, 1), (700, 77), (1030, 200), (131, 3), (640, 128)]


@pytest.mark.parametrize("dtype,d,block_size,hq,hkv", CHUNK_CACHES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 0), (64, 130), (128, 4), (300, 1), (BIG, 0)])
def test_prefill_window(dtype, d, block_size, hq, hkv, window, sinks):
    lens, chunks = [L for L, c in CHUNKS], [c for L, c in CHUNKS]
    w = WindowCase(dtype, lens, chunks, hq, hkv, d, block_size, window, sinks, seed=window % 89)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "prefill")


@pytest.mark.parametrize("dtype", ["f16", "bf16", "fp8", "f32"])
def test_prefill_window_short_chunks(dtype):
    """Chunks of a few tokens only (drafted tokens to verify): 1 to 9 queries a sequence."""
    lens = [900, 33, 1200, 9, 64, 4, 700]
    chunks = [5, 1, 3, 9, 2, 4, 0]
    for window, sinks in ((1, 0), (5, 2), (600, 4), (2000, 0)):
        w = WindowCase(dtype, lens, chunks, 8, 1, 128, 16, window, sinks, seed=window)
        s = Step(w)
        s.prefill()
        check(s, w.reference(), f"window {window}")


@pytest.mark.parametrize("dtype,block_size,d", [("bf16", 16, 128), ("f16", 64, 128), ("fp8", 32, 128), ("bf16", 8, 128),
                                                ("bf16", 32, 64), ("f16", 16, 64)])
@pytest.mark.parametrize("window,sinks,lens,chunks", [
    (2500, 3, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),   # four CTAs an item
    (1100, 0, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),   # two
    (BIG, 0, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),    # four
    (700, 400, [3100, 2600, 130, 3, 900], [64, 33, 50, 3, 0]),  # two
    (4300, 5, [4700, 40], [40, 40]),                            # eight
    (900, 0, [3000, 1500], [300, 150]),                         # two, more query tiles
])
def test_prefill_window_few_long_items(dtype, block_size, d, window, sinks, lens, chunks):
    """Few items over many keys: the CTAs of a cluster share an item's key tiles and merge their rows; the short
    sequences leave some of them without a tile, a ragged chunk some rows outside it."""
    w = WindowCase(dtype, lens, chunks, 8, 1, d, block_size, window, sinks, seed=window % 97)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "few long items")
    assert torch_equal(s.out, Step(w).prefill())


def torch_equal(a, b):
    import torch
    torch.cuda.synchronize()
    return torch.equal(a, b)


def test_prefill_window_is_prefill_and_decode(pa):
    """A window past every length gives pa_prefill's result, a chunk of one token pa_decode_window's."""
    w = WindowCase("bf16", [700, 260], [200, 129], 8, 2, 128, 16, 800, 0, seed=3)
    s, t = Step(w), Step(w)
    s.prefill()
    pa.pa_prefill(t.out, t.q, t.k, t.v, t.table, t.lens, t.start, 200, w.scale, err_flag=t.err)
    assert int(s.err.item()) == 0 and int(t.err.item()) == 0
    # either side is within half an ulp and 2^-12 of the exact value
    a, b = out_f64(s.out), out_f64(t.out)
    assert np.all(np.abs(a - b) <= np.maximum(np.abs(a), np.abs(b)) * 2.0 ** -7 + 2.0 ** -11)
    w = WindowCase("bf16", [700, 260, 5], [1, 1, 1], 8, 2, 128, 16, 100, 3, seed=3)
    s, t = Step(w), Step(w)
    s.prefill()
    t.decode()
    a, b = out_f64(s.out), out_f64(t.out)
    assert np.all(np.abs(a - b) <= np.maximum(np.abs(a), np.abs(b)) * 2.0 ** -7 + 2.0 ** -11)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_prefill_window_rows_and_bad_chunks(dtype):
    """Rows that no chunk owns keep what they held; an inconsistent chunk is reported and skipped."""
    import torch
    w = WindowCase(dtype, [300, 200, 90], [140, 60, 7], 8, 2, 128, 16, 100, 4, seed=9)
    ref = w.reference()
    s = Step(w)
    pad = torch.full((50, 8, 128), SENTINEL, dtype=s.q.dtype, device="cuda")
    s.q, s.out = torch.cat([s.q, pad]), torch.cat([s.out, pad])
    s.prefill()
    got = out_f64(s.out)
    assert int(s.err.item()) == 0 and np.all(got[207:] == SENTINEL)
    ok, err, _ = within_bound(got[:207], ref, w.qdt)
    assert ok, err
    for lens, most in (([300, 59, 90], 140), ([300, 5000, 90], 140), ([300, 200, 90], 100)):
        s = Step(w)
        s.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        s.prefill(max_query_len=most)
        got = out_f64(s.out)
        assert int(s.err.item()) == 5
        bad = slice(0, 140) if most == 100 else slice(140, 200)
        good = np.ones(207, bool)
        good[bad] = False
        assert np.all(got[bad] == SENTINEL)
        ok, err, _ = within_bound(got[good], ref[good], w.qdt)
        assert ok, err


def test_prefill_window_c_call_with_a_loose_bound(pa):
    """max_query_len may be any bound: the C call takes the largest int32."""
    import ctypes
    import torch
    w = WindowCase("bf16", [300, 200, 90], [140, 60, 7], 24, 2, 128, 16, 100, 4, seed=9)
    s = Step(w)
    desc = pa.cache_desc(s.k)
    status = pa.lib().pa_prefill_window(
        s.out.data_ptr(), s.q.data_ptr(), s.k.data_ptr(), s.v.data_ptr(), s.table.data_ptr(), s.lens.data_ptr(),
        s.start.data_ptr(), 3, s.q.shape[0], 24, s.table.shape[1], 2 ** 31 - 1, ctypes.byref(desc), w.scale, w.window,
        w.sinks, 0.0, 0.0, s.err.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert status == 0
    check(s, w.reference(), "loose bound")


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_prefill_window_bad_block(dtype):
    w = WindowCase(dtype, [300, 200], [140, 60], 8, 2, 128, 16, 100, 4, seed=9)
    ref = w.reference()
    s = Step(w)
    s.table[0, 250 // 16] = w.num_blocks + 5
    s.prefill()
    assert int(s.err.item()) == 1
    ok, err, _ = within_bound(out_f64(s.out)[140:], ref[140:], w.qdt)
    assert ok, err


def test_prefill_window_many_items():
    """More work items than SMs, ragged, several tiles each: state runs on from item to item."""
    rng = np.random.default_rng(1)
    chunks = [int(x) for x in rng.integers(1, 200, 14)]
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 400, 14))]
    for dtype, hq, hkv, bs, d in (("bf16", 32, 8, 16, 128), ("f16", 16, 16, 64, 128), ("fp8", 32, 8, 16, 128),
                                  ("bf16", 32, 8, 16, 64), ("f16", 16, 16, 8, 64)):
        w = WindowCase(dtype, lens, chunks, hq, hkv, d, bs, 150, 10, seed=2)
        s = Step(w)
        s.prefill()
        check(s, w.reference(), dtype)


# ---------------------------------------------------------------- streams, graphs, together
@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
def test_window_graphs_on_two_streams(dtype):
    """Two captured steps replayed at once on two streams give the eager bits, also after inputs change."""
    import torch
    steps = [Step(WindowCase(dtype, [900, 40, 333], [1] * 3, 8, 2, 128, 16, 200, 4, seed=i)) for i in (1, 2)]
    pre = [Step(WindowCase(dtype, [300, 180], [130, 9], 8, 2, 128, 16, 90, 4, seed=i)) for i in (3, 4)]
    graphs, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for s, p in zip(steps, pre):
        s.decode()
        p.prefill()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.decode()
            p.prefill()
        graphs.append(g)
    for s, p in zip(steps, pre):
        s.q.mul_(-0.5)
        p.q.mul_(-0.5)
    want = []
    for s, p in zip(steps, pre):
        want.append((s.decode().clone(), p.prefill().clone()))
        s.out.fill_(SENTINEL)
        p.out.fill_(SENTINEL)
    torch.cuda.synchronize()
    for _ in range(5):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for s, p, (a, b) in zip(steps, pre, want):
        assert int(s.err.item()) == 0 and int(p.err.item()) == 0
        assert torch.equal(s.out, a) and torch.equal(p.out, b)


def test_window_reads_lengths_written_just_before():
    """Lengths, tables and queries written by the kernels right before the call on the same stream."""
    import torch
    w = WindowCase("bf16", [900, 40, 333], [1] * 3, 8, 2, 128, 16, 200, 4, seed=7)
    ref = w.reference()
    s = Step(w)
    lens, table, q = s.lens.clone(), s.table.clone(), s.q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        with torch.cuda.stream(side):
            s.lens.zero_()
            s.table.fill_(-1)
            s.q.zero_()
            s.decode()
            s.lens.copy_(lens)
            s.table.copy_(table)
            s.q.copy_(q)
            s.decode()
    side.synchronize()
    check(s, ref, "right after the writes")


# ---------------------------------------------------------------- arguments
def pinned(t):
    return t.cpu().pin_memory()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_decode_window_pinned_host_arrays(dtype):
    """The step's small arrays in pinned host memory, read and written in place: the same bits."""
    import torch
    w = WindowCase(dtype, [300, 0, 41], [1] * 3, 8, 2, 128, 16, 100, 4, seed=3, append=dtype != "f32")
    s, t = Step(w), Step(w)
    s.decode()
    for name in ("q", "out", "table", "lens"):
        setattr(t, name, pinned(getattr(t, name)))
    if t.nk is not None:
        t.nk, t.nv = pinned(t.nk), pinned(t.nv)
    t.decode()
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0
    assert torch.equal(t.out, s.out.cpu())
    assert torch.equal(t.k.view(torch.uint8), s.k.view(torch.uint8))


def test_window_calls_refuse_wrong_tensors(pa):
    import torch
    w = WindowCase("bf16", [30, 20], [1, 1], 8, 2, 128, 16, 10, 2, seed=3)
    s = Step(w)
    good = dict(out=s.out, q=s.q, k_cache=s.k, v_cache=s.v, block_tables=s.table, seq_lens=s.lens)

    def decode(**kw):
        pa.pa_decode_window(**{**good, **kw}, scale=0.1, window=10)

    def prefill(start=s.start, **kw):
        pa.pa_prefill_window(**{**good, **kw}, query_start=start, max_query_len=1, scale=0.1, window=10)

    for call in (decode, prefill):
        for kw, error in ((dict(q=s.q.half()), TypeError), (dict(out=s.out.float()), TypeError),
                          (dict(block_tables=s.table.long()), TypeError), (dict(seq_lens=s.lens.long()), TypeError),
                          (dict(q=s.q.cpu()), ValueError), (dict(seq_lens=s.lens[:1]), ValueError),
                          (dict(q=s.q[:, :, :64]), ValueError), (dict(q=s.q[:, :4]), ValueError),
                          (dict(v_cache=s.v.half()), ValueError), (dict(v_cache=s.v[:1]), ValueError),
                          (dict(block_tables=s.table[:, ::2]), ValueError), (dict(err_flag=torch.zeros(1)), TypeError),
                          (dict(err_flag=pinned(s.err)), ValueError)):
            with pytest.raises(error):
                call(**kw)
    with pytest.raises(ValueError):  # tensor-map copies move q and out
        prefill(q=pinned(s.q))
    with pytest.raises(ValueError):
        prefill(start=s.start[:2])
    with pytest.raises(ValueError):
        decode(key=s.q[:, :2].contiguous())
    with pytest.raises(ValueError):
        decode(key=s.q, value=s.q)
    with pytest.raises(ValueError):
        decode(alibi_slopes=torch.zeros(3, device="cuda"))
    with pytest.raises(pa.PaError):
        pa.pa_decode_window(**good, scale=0.1, window=0)
    # a descriptor of another pool: more blocks than there are, another type
    right = pa.cache_desc(s.k)
    for field, value in (("num_blocks", right.num_blocks + 1), ("head_size", 64), ("dtype", pa.PA_F16)):
        desc = pa.cache_desc(s.k)
        setattr(desc, field, value)
        for call in (decode, prefill):
            with pytest.raises(ValueError):
                call(desc=desc)
    decode(desc=right)
    torch.cuda.synchronize()


def test_windowless_empty_batches(pa):
    """No sequences, no queries, no table: nothing to do."""
    import torch
    w = WindowCase("bf16", [30, 20], [1, 1], 8, 2, 128, 16, 10, 2, seed=3)
    s = Step(w)
    before = s.out.clone()
    pa.pa_decode_window(s.out[:0], s.q[:0], s.k, s.v, s.table[:0], s.lens[:0], 0.1, 10)
    pa.pa_prefill_window(s.out, s.q, s.k, s.v, s.table, s.lens, torch.zeros_like(s.start), 0, 0.1, 10)
    pa.pa_prefill_window(s.out, s.q, s.k, s.v, s.table, s.lens, torch.zeros_like(s.start), 3, 0.1, 10, err_flag=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0 and torch.equal(s.out, before)
    # a table without columns: only empty sequences fit
    zero = torch.zeros_like(s.lens)
    pa.pa_decode_window(s.out, s.q, s.k, s.v, s.table[:, :0].contiguous(), zero, 0.1, 10, err_flag=s.err)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0 and torch.count_nonzero(s.out) == 0


def in_large_pool(s, num_blocks):
    """The step's blocks as the last ones of a pool of num_blocks (offsets past 32 bits)."""
    import torch
    w, shift = s.w, num_blocks - s.w.num_blocks
    for name in ("k", "v"):
        small = getattr(s, name)
        big = torch.zeros((num_blocks, *small.shape[1:]), dtype=small.dtype, device="cuda")
        big[shift:] = small
        setattr(s, name, big)
    inside = (s.table >= 0) & (s.table < w.num_blocks)
    s.table = torch.where(inside, s.table + shift, torch.full_like(s.table, -1))
    return s


@pytest.mark.parametrize("dtype,num_blocks", [("f32", 70000), ("bf16", 140000), ("fp8", 270000)])
def test_window_large_pool(dtype, num_blocks):
    """Caches of more than 2^31 elements (2^32 bytes): the step, its append, and a chunk, in their last blocks."""
    import torch
    hkv = 16 if dtype == "f32" else 8
    w = WindowCase(dtype, [500, 90, 17], [1] * 3, 2 * hkv, hkv, 128, 16, 60, 4, seed=1, append=dtype != "f32")
    s = in_large_pool(Step(w), num_blocks)
    s.decode()
    check(s, w.reference(), "decode")
    assert torch.count_nonzero(s.k[:1000].view(torch.uint8)) == 0
    del s
    torch.cuda.empty_cache()
    w = WindowCase(dtype, [500, 90], [70, 90], 2 * hkv, hkv, 128, 16, 60, 4, seed=2)
    s = in_large_pool(Step(w), num_blocks)
    s.prefill()
    check(s, w.reference(), "chunk")
    del s
    torch.cuda.empty_cache()


def test_decode_window_longer_than_int32():
    """A window past int32 sees everything, as one of 2^31 - 1 does."""
    w = WindowCase("bf16", [50, 300], [1, 1], 8, 2, 128, 16, BIG, 0, seed=3)
    s = Step(w)
    ref = w.reference()
    w.window = 2 ** 32 + 5
    s.decode()
    check(s, ref, "long window")
