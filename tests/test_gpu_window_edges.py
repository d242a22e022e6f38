"""Windowed attention at its edges: arguments that must not matter, values that must (needs a GB300)."""
import numpy as np
import pytest

from test_gpu_window import Step
from window_ref import WindowCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


# chunks for each kernel that a pa_prefill_window call may come to: rows of eight queries; tiles; tiles whose keys a
# cluster shares
CHUNK_FORMS = {
    "rows": dict(lens=[900, 33], chunks=[1, 2], hq=8, hkv=2, window=300),
    "tiles": dict(lens=[700, 260, 90] * 4, chunks=[200, 129, 77] * 4, hq=32, hkv=8, window=150),
    "split tiles": dict(lens=[3100, 2600], chunks=[64, 33], hq=8, hkv=1, window=2500),
}


def chunk_case(form, dtype, seed=0, d=128, block_size=16):
    f = CHUNK_FORMS[form]
    return WindowCase(dtype, f["lens"], f["chunks"], f["hq"], f["hkv"], d, block_size, f["window"], 3, seed=seed)


# ---------------------------------------------------------------- FP8 scales over other caches
@pytest.mark.parametrize("form", CHUNK_FORMS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_scales_are_those_of_fp8_caches(dtype, form):
    """k_scale and v_scale mean nothing to other caches, whatever they hold: the bits of the calls without them."""
    import torch
    w = chunk_case(form, dtype)
    d = WindowCase(dtype, [300, 7], [1, 1], 8, 2, 128, 16, 100, 4)
    chunk, step = Step(w).prefill(), Step(d).decode()
    for k_scale, v_scale in ((0.0123, 0.5), (float("nan"), float("nan")), (-1.0, float("inf"))):
        s, t = Step(w), Step(d)
        assert torch.equal(s.prefill(k_scale=k_scale, v_scale=v_scale), chunk)
        assert torch.equal(t.decode(k_scale=k_scale, v_scale=v_scale), step)
        assert int(s.err.item()) == 0 and int(t.err.item()) == 0


# ---------------------------------------------------------------- NaN where it is seen
def nan_key(s, seq, pos, head):
    """The key of a kv head at a position of sequence seq becomes NaN, in all dimensions."""
    w = s.w
    block, off = int(w.table[seq, pos // w.B]), pos % w.B
    s.k[block, head, off] = 0x7F if w.dtype == "fp8" else float("nan")


def check_nan_rows(s, ref, nan):
    """The rows of `nan` [queries, heads] are NaN from end to end, the others right."""
    from harness import out_f64, within_bound
    got = out_f64(s.out)
    assert int(s.err.item()) == 0
    assert np.isnan(got[nan]).all(), f"{np.sum(~np.isnan(got[nan]).all(-1))} of {nan.sum()} rows are not NaN"
    assert not np.isnan(got[~nan]).any()
    ok, err, ratio = within_bound(got[~nan], ref[~nan], s.w.qdt)
    assert ok, f"max abs err {err}, worst err/bound {ratio}"


@pytest.mark.parametrize("dtype,d", [("f32", 128), ("f32", 64), ("f16", 128), ("bf16", 64), ("bf16", 128), ("fp8", 128)])
@pytest.mark.parametrize("lens", [[40, 700, 1, 300], [9001]])
def test_decode_window_nan_is_not_hidden(dtype, d, lens):
    """A NaN in a query, or in a key that it sees, makes the row NaN, whoever computes it (a CTA, a large cluster);
    where nothing sees the key it has no effect."""
    hq, hkv = 8, 2
    w = WindowCase(dtype, lens, [1] * len(lens), hq, hkv, d, 16, 4200 if len(lens) == 1 else 200, 3, seed=3)
    ref = w.reference()
    for what in ("query", "key", "first key", "unseen key"):
        s = Step(w)
        nan = np.zeros((len(lens), hq), bool)
        seq = int(np.argmax(lens))
        if what == "query":
            s.q[seq, 5] = float("nan")
            nan[seq, 5] = True
        else:
            pos = {"key": lens[seq] - 9, "first key": 1, "unseen key": 12}[what]
            if what == "unseen key":  # in the block of the first keys, which is loaded
                assert w.sinks <= pos <= lens[seq] - 1 - w.window and pos // w.B == 0
            nan_key(s, seq, pos, 1)
            nan[seq, hq // hkv:] = what != "unseen key"
        s.decode()
        check_nan_rows(s, ref, nan)


@pytest.mark.parametrize("form", CHUNK_FORMS)
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16", "fp8"])
def test_prefill_window_nan_is_not_hidden(dtype, form):
    """The same for the queries of a chunk: those that see the key are NaN, those before it and those whose window
    has passed it are right."""
    w = chunk_case(form, dtype, seed=3)
    ref = w.reference()
    start, G = w.query_start(), w.hq // w.hkv
    rows = np.arange(start[-1])
    seq = int(np.argmax(w.chunks))
    L, n = w.lens[seq], w.chunks[seq]
    pos = np.arange(L - n, L)  # of the sequence's queries
    for what in ("query", "key", "first key"):
        s = Step(w)
        nan = np.zeros((len(rows), w.hq), bool)
        if what == "query":
            s.q[start[seq] + n // 2, 1] = float("nan")
            nan[start[seq] + n // 2, 1] = True
        else:
            at = L - n + n // 2 if what == "key" else 1
            nan_key(s, seq, at, w.hkv - 1)
            sees = (at <= pos) & ((at > pos - w.window) | (at < w.sinks))
            nan[start[seq]:start[seq + 1], (w.hkv - 1) * G:] = sees[:, None]
            assert sees.any() and (what == "first key" or not sees.all() or n <= 2)
        s.prefill()
        check_nan_rows(s, ref, nan)


# ---------------------------------------------------------------- batches that mix chunk lengths
def mixed(dtype, d, block_size, hq, hkv, n=70, prompt=700, seed=0):
    """n sequences of single tokens, one among them with a prompt, a few with two to nine tokens or none."""
    rng = np.random.default_rng(seed)
    chunks = [1] * n
    chunks[n // 3] = prompt
    for s in range(5, n, 11):
        chunks[s] = int(rng.integers(0, 10))
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 300, n))]
    return WindowCase(dtype, lens, chunks, hq, hkv, d, block_size, 130, 4, seed=seed)


# (block sizes that do not divide 128 and fp32 caches go to the rows kernels, in slots)
MIXED = [("f16", 128, 16, 8, 2), ("bf16", 128, 32, 12, 2), ("bf16", 64, 16, 8, 1), ("fp8", 128, 16, 8, 2),
         ("f16", 64, 48, 8, 2), ("bf16", 128, 48, 12, 2), ("fp8", 128, 48, 8, 1), ("f32", 64, 16, 14, 2),
         ("f32", 128, 5, 4, 4)]


@pytest.mark.parametrize("dtype,d,block_size,hq,hkv", MIXED)
def test_prefill_window_mixed_batch(dtype, d, block_size, hq, hkv):
    """Single tokens, short chunks, empty ones and a prompt in one call."""
    import torch
    from test_gpu_window import check
    w = mixed(dtype, d, block_size, hq, hkv)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "mixed")
    # a looser bound on the chunks: the same rows
    t = Step(w)
    pad = torch.zeros((4000, hq, d), dtype=t.q.dtype, device="cuda")
    t.q, t.out = torch.cat([t.q, pad]), torch.cat([t.out, pad + 123.0])
    t.prefill(max_query_len=4000 + s.q.shape[0])
    n = s.q.shape[0]  # (rows past the last chunk keep what they held)
    assert int(t.err.item()) == 0 and torch.all(t.out[n:] == 123.0)
    t.out = t.out[:n].contiguous()
    check(t, w.reference(), "mixed, loose bound")


def test_prefill_window_mixed_batch_long_windows():
    """fp32 row groups in slots whose keys a cluster shares: all of its CTAs find the same group, or none."""
    from test_gpu_window import check
    rng = np.random.default_rng(4)
    chunks = [1] * 70
    chunks[40] = 700
    lens = [c + int(x) for c, x in zip(chunks, rng.integers(0, 2600, 70))]
    w = WindowCase("f32", lens, chunks, 4, 1, 64, 16, 2500, 4, seed=4)
    s = Step(w)
    s.prefill()
    check(s, w.reference(), "mixed, long windows")


@pytest.mark.parametrize("dtype,d,block_size,hq,hkv", MIXED)
def test_prefill_window_mixed_batch_bad_chunks(dtype, d, block_size, hq, hkv):
    """Inconsistent chunks of a mixed batch are reported and skipped, wherever they stand; the others are right."""
    import torch
    from harness import out_f64, within_bound
    w = mixed(dtype, d, block_size, hq, hkv, seed=1)
    ref, start, n = w.reference(), w.query_start(), len(w.chunks)
    for bad in (0, n // 3, n - 1):
        s = Step(w)
        s.lens[bad] = w.width * block_size + 1
        s.prefill()
        got, rows = out_f64(s.out), np.ones(len(ref), bool)
        rows[start[bad]:start[bad + 1]] = False
        assert int(s.err.item()) == 5 and np.all(got[~rows] == 123.0)
        ok, err, _ = within_bound(got[rows], ref[rows], w.qdt)
        assert ok, err
    # a start that falls: sequence 2 begins before the batch, 1 ends before it starts
    s = Step(w)
    s.start[2] = -4
    s.prefill()
    got, rows = out_f64(s.out), np.ones(len(ref), bool)
    rows[start[1]:start[3]] = False
    assert int(s.err.item()) == 5 and np.all(got[~rows] == 123.0)
    ok, err, _ = within_bound(got[rows], ref[rows], w.qdt)
    assert ok, err
    # chunks that overlap from the start on may not all be done, which is reported
    s = Step(w)
    s.start[:] = torch.arange(n + 1, dtype=torch.int32, device="cuda") % 2 * 600
    s.lens.fill_(w.width * block_size)
    s.table.fill_(0)
    s.prefill()
    assert int(s.err.item()) == 5


@pytest.mark.parametrize("dtype,d,block_size,hq,hkv,n,rows", [
    ("f32", 64, 16, 16, 1, 8200, 131072),    # 2.1e9 groups of rows for a grid of the longest chunk's
    ("bf16", 64, 16, 128, 1, 33000, 65536),  # 2.2e9 tiles
    ("bf16", 64, 16, 128, 1, 4096, 65536),   # 2.7e8 tiles, 1.8 million for each CTA to step over
    ("bf16", 64, 48, 128, 1, 4096, 65536),
])
def test_prefill_window_capacity_buffers(dtype, d, block_size, hq, hkv, n, rows):
    """A batch of single tokens in buffers of a capacity, which also bounds the chunks (a captured graph's): the call
    goes by what is there."""
    import torch
    from test_gpu_window import check
    rng = np.random.default_rng(n)
    lens = [int(x) for x in rng.integers(1, 4, n)]
    w = WindowCase(dtype, lens, [1] * n, hq, hkv, d, block_size, 2, 1, seed=n, slack_blocks=3)
    s = Step(w)
    out = torch.full((rows, hq, d), 123.0, dtype=s.q.dtype, device="cuda")
    q = torch.zeros_like(out)
    q[:n] = s.q
    s.q, s.out = q, out
    s.prefill(max_query_len=rows)
    assert int(s.err.item()) == 0 and torch.all(out[n:] == 123.0)
    s.out = out[:n].contiguous()
    check(s, w.reference(), "capacity buffers")
    del q, out
    torch.cuda.empty_cache()


FIRST_CALL = """
import torch
import paged_kv_cache_32_gb300 as pa
for dtype in (torch.bfloat16, torch.uint8, torch.float32):
    rows = torch.float16 if dtype == torch.uint8 else dtype
    k = torch.randint(0, 64, (600, 1, 16, 128), device="cuda").to(dtype)
    v = k.view(600, 1, 1, 128, 16) if dtype == torch.uint8 else k
    q = torch.ones(1, 8, 128, device="cuda", dtype=rows)
    out, again = torch.zeros_like(q), torch.zeros_like(q)
    table = torch.arange(600, device="cuda", dtype=torch.int32)[None]
    lens, start = (torch.tensor(x, device="cuda", dtype=torch.int32) for x in ([9000], [0, 1]))
    calls = (lambda o: pa.pa_decode_window(o, q, k, v, table, lens, 0.01, 8000, num_sinks=4),
             lambda o: pa.pa_prefill_window(o, q, k, v, table, lens, start, 1, 0.01, 8000, num_sinks=4))
    for call in calls:
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


def test_window_first_call_captured():
    """A process whose first call of each kernel is captured: what the call asks the device once is no obstacle."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stdout + r.stderr
