"""A serving loop over a 4-bit cache whose lengths live on the GPU (needs a GB300): prompts, then drafted tokens of which some
are rejected, requests that end and make room for others.  Each step is pa_tables_trim, pa_tables_extend,
pa_rope_axes_and_cache and pa_prefill_fp4, once called, once replayed from one captured graph, and is checked against a
model of the tables and attention in 64 bits over the rows that the cache holds; the held keys against their rotation."""
import numpy as np
import pytest

import oracle as O
from fp4_ref import K_UNIT, V_UNIT, unpack, values
from harness import out_f64, to_numpy_storage
from test_gpu_fp4 import within_bound
from test_gpu_rope_axes import per_axis
from test_gpu_tables import Device, Model

pytestmark = pytest.mark.gpu

N, HQ, HKV, B, WIDTH, ROWS = 5, 12, 3, 32, 12, 400


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows", ["f16", "bf16"])
def test_steps(rows, captured):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    rng = np.random.default_rng(5)
    t = torch.float16 if rows == "f16" else torch.bfloat16
    m = Model(N, WIDTH, B, N * WIDTH - 9, rng)
    d = Device(m, ROWS)
    pairs = pa.pa_rope_pair_axes((16, 24, 24))
    inv, mag = pa.pa_rope_frequencies(128, 500000.0, device="cuda")
    k, v = pa.fp4_cache(N * WIDTH - 9, HKV, B), pa.fp4_cache(N * WIDTH - 9, HKV, B)
    qkv = torch.zeros(ROWS, HQ + 2 * HKV, 128, dtype=t, device="cuda")
    q, out = torch.zeros(ROWS, HQ, 128, dtype=t, device="cuda"), torch.zeros(ROWS, HQ, 128, dtype=t, device="cuda")
    keep, new = (torch.zeros(N, dtype=torch.int32, device="cuda") for _ in range(2))
    scale = 128 ** -0.5

    def step():
        pa.pa_tables_trim(d.table, d.lens, d.held, d.free, d.top, keep, B, err_flag=d.err)
        pa.pa_tables_extend(d.table, d.lens, d.held, d.free, d.top, new, d.slots, d.pos, d.start, B, err_flag=d.err)
        pos = torch.stack([d.pos, d.pos * 2, d.pos // 3])
        pa.pa_rope_axes_and_cache(q, k, v, qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], pos, d.slots, inv, pairs,
                                  magnitude=mag, err_flag=d.err, k_scale=K_UNIT, v_scale=V_UNIT)
        pa.pa_prefill_fp4(out, q, k, v, d.table, d.lens, d.start, ROWS, scale, K_UNIT, V_UNIT, err_flag=d.err)

    if captured:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        # (nothing ran while it was captured)
        d.check()
    for i in range(8):
        if i == 0:
            kept, want = np.zeros(N, np.int64), rng.integers(1, 90, N)
        else:
            kept = m.lens - rng.integers(0, 4, N) * (m.lens > 4)
            want = np.full(N, 4)
            done = int(rng.integers(N))
            kept[done], want[done] = 0, rng.integers(1, 150)
        keep.copy_(torch.from_numpy(np.asarray(kept, np.int32)))
        new.copy_(torch.from_numpy(np.asarray(want, np.int32)))
        qkv.copy_(torch.from_numpy(rng.standard_normal(qkv.shape)))
        graph.replay() if captured else step()
        m.trim(kept)
        slots, pos, start = m.extend(want, ROWS)
        assert d.error() == 0
        d.check((slots, pos, start))
        x = O.to_f64(to_numpy_storage(qkv, rows), rows)
        y, e = per_axis(x, np.stack([pos, pos * 2, pos // 3]), inv.cpu().numpy(), mag, False, pairs)
        live = slots >= 0
        (kc, ks), (vc, vs) = unpack(k.cpu().numpy()), unpack(v.cpu().numpy())
        blk, off = slots[live] // B, slots[live] % B
        for cache, unit, row in ((values(kc, ks, K_UNIT), K_UNIT, y[live, HQ:HQ + HKV]),
                                 (values(vc, vs, V_UNIT), V_UNIT, x[live, HQ + HKV:])):
            got, amax = cache[blk, :, off], np.abs(row).reshape(-1, HKV, 8, 16).max(-1).repeat(16, -1)
            # half of the widest step, 2 of 6, at a scale off by up to 1/16, and the rows' own rounding
            assert np.all(np.abs(got - row) <= amax * (17 / 16 / 6 + 2.0 ** -7) + 2.0 ** -10 * unit)
        qh, kk, vv = O.to_f64(to_numpy_storage(q, rows), rows), values(kc, ks, K_UNIT), values(vc, vs, V_UNIT)
        ref = np.zeros((int(start[-1]), HQ, 128))
        for s in range(N):
            a, b, L = start[s], start[s + 1], m.lens[s]
            p = np.arange(L)
            block, o = m.table[s, p // B], p % B
            key, val = (np.repeat(c[block, :, o], HQ // HKV, 1) for c in (kk, vv))
            sc = np.einsum("qhd,khd->hqk", qh[a:b], key) * scale
            sc[:, p[None] > np.arange(L - (b - a), L)[:, None]] = -np.inf
            w = np.exp(sc - sc.max(2, keepdims=True))
            ref[a:b] = np.einsum("hqk,khd->qhd", w / w.sum(2, keepdims=True), val)
        ok, err, ratio = within_bound(out_f64(out)[:len(ref)], ref, rows)
        assert ok, (i, err, ratio)
