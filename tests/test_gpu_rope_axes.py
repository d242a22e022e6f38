"""Rotary positions along several axes, and over caches held in 4 bits (needs a GB300).

Bounds per element: those of test_gpu_rope.py.  Over a 4-bit cache the keys are compared as bytes with the quantisation of
the turned keys in their 16-bit type, which the same call gives over a 16-bit cache.
"""
import numpy as np
import pytest

import oracle as O
import workloads as W
from fp4_ref import K_UNIT, V_UNIT, pack, quantise
from harness import to_numpy_storage, to_torch
from test_gpu_rope import Rope, turned

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


class Axes(Rope):
    """As Rope, with pos [axes, tokens]; the reference turns each axis's pairs by themselves."""

    def __init__(self, pa, dtype, tokens, hq, hkv, d, block_size, rotary, interleaved, axes, pair_axis, **kw):
        super().__init__(pa, dtype, tokens, hq, hkv, d, block_size, rotary, interleaved, **kw)
        rng = np.random.default_rng(tokens + axes)
        self.pos = rng.integers(-5, 100000, (axes, tokens)).astype(np.int32)
        self.pair_axis = pair_axis

    def run(self, **kw):
        import torch
        fp8 = self.dtype == "fp8"
        self.pa.pa_rope_axes_and_cache(
            self.q_out if self.hq else None, self.k, self.v, self.q if self.hq else None, self.key, self.value,
            torch.from_numpy(self.pos).cuda(), torch.from_numpy(self.slots).cuda(), self.inv.cuda(), self.pair_axis,
            interleaved=self.interleaved, magnitude=self.mag, err_flag=self.err,
            **(dict(k_scale=0.0123, v_scale=0.0117) if fp8 else {}), **kw)


def per_axis(x, pos, inv, magnitude, interleaved, pair_axis):
    """turned(), where pair j goes by pos[pair_axis[j]]."""
    y, e = np.zeros(x.shape), np.zeros(x.shape)
    r, done = 2 * len(inv), np.zeros(x.shape[-1], bool)
    for a in range(len(pos)):
        ya, ea = turned(x, pos[a], inv, magnitude, interleaved)
        j = np.nonzero(np.asarray(list(pair_axis)) == a)[0]
        at = np.concatenate([2 * j, 2 * j + 1]) if interleaved else np.concatenate([j, j + r // 2])
        y[..., at], e[..., at], done[at] = ya[..., at], ea[..., at], True
    y[..., ~done] = x[..., ~done]
    return y, e


@pytest.mark.parametrize("dtype,d,block_size", [("f32", 64, 5), ("f16", 128, 8), ("bf16", 128, 32), ("bf16", 64, 8),
                                                ("fp8", 128, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,sections,dealt", [(64, (8, 12, 12), False), (64, (8, 12, 12), True), (18, (9,), False),
                                                   (20, (1, 2, 3, 4), True), (128, (16, 24, 24), False)])
def test_rope_axes(pa, monkeypatch, dtype, d, block_size, interleaved, rotary, sections, dealt):
    import test_gpu_rope
    if rotary > d:
        rotary, sections = 64, (16, 16)
    pairs = pa.pa_rope_pair_axes(sections, interleaved=dealt)
    assert len(pairs) == rotary // 2 and [pairs.count(a) for a in range(len(sections))] == list(sections)
    monkeypatch.setattr(test_gpu_rope, "turned", lambda x, pos, inv, mag, inter: per_axis(x, pos, inv, mag, inter, pairs))
    for tokens, hq, hkv in ((1, 7, 1), (67, 4, 4), (500, 12, 2), (3001, 8, 2)):
        r = Axes(pa, dtype, tokens, hq, hkv, d, block_size, rotary, interleaved, len(sections), pairs, seed=tokens,
                 padding=range(3, tokens, 10))
        r.run()
        r.check()


@pytest.mark.parametrize("dtype", ["f16", "bf16", "fp8", "f32"])
def test_one_axis_is_rope(pa, dtype):
    """The same positions along every axis give pa_rope_and_cache's bits."""
    import torch
    a = Axes(pa, dtype, 300, 8, 2, 128, 16, 128, False, 3, pa.pa_rope_pair_axes((16, 24, 24)), seed=1)
    b = Rope(pa, dtype, 300, 8, 2, 128, 16, 128, False, seed=1)
    a.pos = np.tile(b.pos, (3, 1))
    a.run()
    b.run()
    for x, y in ((a.q_out, b.q_out), (a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary,tokens,hq,hkv", [(128, 70, 8, 2), (36, 5, 7, 1), (2, 300, 0, 3), (64, 1000, 17, 4),
                                                  (96, 33, 4, 1), (112, 700, 3, 5), (126, 9, 0, 2), (32, 2500, 6, 2),
                                                  (16, 1301, 1, 16), (128, 1, 64, 8)])
def test_rope_fp4(pa, rows, interleaved, rotary, tokens, hq, hkv):
    """Over a 4-bit cache: the queries of the same call over a 16-bit cache, and its keys held in 4 bits."""
    import torch
    half = rotary // 2
    pairs = bytes(j % 3 for j in range(half))
    r = Axes(pa, rows, tokens, hq, hkv, 128, 16, rotary, interleaved, 3, pairs, seed=tokens, padding=range(2, tokens, 7))
    r.run()
    k = torch.full((r.num_blocks, hkv, 1, 1152), 0x55, dtype=torch.uint8, device="cuda")
    v = k.clone()
    q_out = torch.full_like(r.q_out, 9.0)
    pa.pa_rope_axes_and_cache(q_out if hq else None, k, v, r.q if hq else None, r.key, r.value,
                              torch.from_numpy(r.pos).cuda(), torch.from_numpy(r.slots).cuda(), r.inv.cuda(), pairs,
                              interleaved=interleaved, magnitude=r.mag, err_flag=r.err, k_scale=K_UNIT, v_scale=V_UNIT)
    assert int(r.err.item()) == 0
    # one rounding to the rows' type lies between: queries may differ in the last place where fp32 results do
    a, b = (O.to_f64(to_numpy_storage(t, rows), rows) for t in (q_out, r.q_out))
    y, e = per_axis(r.x, r.pos, r.inv.numpy(), r.mag, interleaved, pairs)
    live = r.slots >= 0
    step = 2.0 ** -11 if rows == "f16" else 2.0 ** -8
    if hq:
        lim = step * np.abs(y[:, :hq]) * (1 + 2 ** -8) + e[:, :hq] + 2.0 ** -25
        assert np.all(np.abs(a - y[:, :hq])[live] <= lim[live]) and np.all(a[~live] == 9.0)
    blk, off = r.slots[live] // 16, r.slots[live] % 16
    kb, vb = k.cpu().numpy(), v.cpu().numpy()
    want_c = np.full((r.num_blocks, hkv, 16, 64), 0x55, np.uint8)
    want_s = np.full((r.num_blocks, hkv, 16, 8), 0x55, np.uint8)
    want_c[blk, :, off], want_s[blk, :, off] = quantise(r.x[live, hq + hkv:], V_UNIT)
    assert np.array_equal(vb, pack(want_c, want_s))
    held = O.to_f64(to_numpy_storage(r.k, rows), rows)[blk, :, off]
    want_c[blk, :, off], want_s[blk, :, off] = quantise(held, K_UNIT)
    assert np.array_equal(kb, pack(want_c, want_s))


def test_in_place_and_bad_slot(pa):
    import torch
    pairs = pa.pa_rope_pair_axes((64,))
    x = torch.randn(40, 6, 128, device="cuda", dtype=torch.bfloat16)
    pos = torch.arange(40, dtype=torch.int32, device="cuda")[None].contiguous()
    slots = torch.arange(40, device="cuda")
    slots[7] = 64
    inv, _ = pa.pa_rope_frequencies(128, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v, out = pa.fp4_cache(4, 1, 16), pa.fp4_cache(4, 1, 16), torch.zeros(40, 4, 128, device="cuda", dtype=torch.bfloat16)
    pa.pa_rope_axes_and_cache(out, k, v, x[:, :4], x[:, 4:5], x[:, 5:], pos, slots, inv, pairs, err_flag=err, k_scale=K_UNIT,
                              v_scale=V_UNIT)
    assert int(err.item()) == 2 and bool((out[7] == 0).all())
    y = x.clone()
    pa.pa_rope_axes_and_cache(y[:, :4], k, v, y[:, :4], y[:, 4:5], y[:, 5:], pos, slots, inv, pairs, k_scale=K_UNIT,
                              v_scale=V_UNIT)
    live = [i for i in range(40) if i != 7]
    assert torch.equal(y[live, :4], out[live]) and torch.equal(y[7], x[7]) and torch.equal(y[:, 4:], x[:, 4:])
