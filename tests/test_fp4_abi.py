"""Caches held in 4 bits, tables and rotary axes without a GPU: refusals, in which nothing is launched, and what the
Python binding passes on."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_32_gb300 as pa
from fp4_ref import quantise, values

FAKE = 0x10000  # never dereferenced: every call below is rejected before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.lib()


def desc(nb=16, bs=16, hkv=2, d=128, dtype=pa.PA_FP4_E2M1):
    return pa.pa_cache_desc(nb, bs, hkv, d, dtype)


def write(lib, d, k=FAKE, v=FAKE, key=FAKE, value=FAKE, ks=256, vs=256, slots=FAKE, t=3, rows=pa.PA_F16, ku=0.01, vu=0.01,
          name="pa_reshape_and_cache_fp4"):
    return getattr(lib, name)(k, v, key, value, ks, vs, slots, t, ctypes.byref(d), rows, ku, vu, None, None)


@pytest.mark.parametrize("name", ["pa_reshape_and_cache_fp4", "pa_read_cache_fp4"])
def test_write_and_read_refusals(lib, name):
    def call(d=desc(), **kw):
        return write(lib, d, name=name, **kw)
    assert call(desc(dtype=pa.PA_FP8_E4M3)) == 2
    assert call(desc(d=64)) == 2
    for bs in (8, 24, 272):
        assert call(desc(bs=bs)) == 2
    assert call(rows=pa.PA_F32) == 2 and call(rows=pa.PA_FP4_E2M1) == 2
    assert call(desc(bs=0)) == 3 and call(desc(hkv=0)) == 3
    assert call(t=-1) == 3
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-31, 1.3e30):
        assert call(ku=bad) == 3 and call(vu=bad) == 3
    assert call(ks=255) == 3 and call(vs=0) == 3
    assert call(key=None) == 1 and call(slots=None) == 1 and call(v=None) == 1
    assert call(key=FAKE + 8) == 5 and call(k=FAKE + 8) == 5 and call(slots=FAKE + 4) == 5 and call(ks=260) == 5
    assert call(ks=1 << 45) == 7 and call(desc(nb=1 << 30)) == 7
    assert call(t=0, key=None) == 0


def decode(lib, d=desc(), out=FAKE, q=FAKE, k=FAKE, v=FAKE, key=None, value=None, bt=FAKE, sl=FAKE, n=2, hq=4, m=4,
           rows=pa.PA_BF16, scale=0.1, window=8, sinks=0, ku=0.01, vu=0.01, slopes=None, ws=None, ws_bytes=0):
    return lib.pa_decode_fp4(out, q, k, v, key, value, bt, sl, n, hq, m, ctypes.byref(d), rows, scale, window, sinks, ku, vu,
                             slopes, 0, ws, ws_bytes, None, None)


def prefill(lib, d=desc(), out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, qs=FAKE, n=2, t=10, hq=4, m=4, most=5,
            rows=pa.PA_F16, scale=0.1, window=8, sinks=0, ku=0.01, vu=0.01):
    return lib.pa_prefill_fp4(out, q, k, v, bt, sl, qs, n, t, hq, m, most, ctypes.byref(d), rows, scale, window, sinks, ku,
                              vu, None, None)


def test_attention_refusals(lib):
    for call in (decode, prefill):
        assert call(lib, desc(dtype=pa.PA_F16)) == 2 and call(lib, desc(bs=8)) == 2 and call(lib, desc(d=64)) == 2
        assert call(lib, rows=pa.PA_F32) == 2
        assert call(lib, hq=3) == 3 and call(lib, n=-1) == 3 and call(lib, window=0) == 3 and call(lib, sinks=-1) == 3
        assert call(lib, scale=math.nan) == 3 and call(lib, ku=0.0) == 3 and call(lib, vu=math.inf) == 3
        assert call(lib, q=None) == 1 and call(lib, k=None) == 1 and call(lib, sl=None) == 1 and call(lib, bt=None) == 1
        assert call(lib, q=FAKE + 8) == 5 and call(lib, v=FAKE + 4) == 5 and call(lib, sl=FAKE + 2) == 5
        assert call(lib, m=1 << 28) == 7
        assert call(lib, n=0, out=None) == 0
    big = desc(bs=64)
    need = pa.pa_decode_fp4_workspace_size(2, 4, 1000, big)
    assert need > 0 and need == pa.pa_decode_fp4_workspace_size(100, 4, 700, big, window=30000)
    assert pa.pa_decode_fp4_workspace_size(2, 4, 4, big) == 0                  # short contexts
    assert pa.pa_decode_fp4_workspace_size(100, 4, 1000, big, window=4096) == 0  # items of nearly one length
    assert pa.pa_decode_fp4_workspace_size(2, 3, 1000, big) == 0 and pa.pa_decode_fp4_workspace_size(2, 4, 1000, desc(bs=8)) == 0
    assert decode(lib, big, m=1000, window=2 ** 31 - 1, ws=FAKE, ws_bytes=need - 1) == 4
    assert decode(lib, big, m=1000, window=2 ** 31 - 1, ws=FAKE + 64, ws_bytes=need) == 5
    assert decode(lib, out=FAKE + 8) == 5
    assert decode(lib, key=FAKE) == 1 and decode(lib, key=FAKE, value=FAKE + 8) == 5 and decode(lib, slopes=FAKE + 2) == 5
    assert prefill(lib, scale=0.0) == 3 and prefill(lib, t=-1) == 3 and prefill(lib, most=-1) == 3
    assert prefill(lib, qs=None) == 1 and prefill(lib, out=FAKE + 8) == 5 and prefill(lib, t=(1 << 31) - 1, hq=1 << 12) == 7
    assert prefill(lib, most=0, out=None) == 0


def test_other_calls_refuse_the_type(lib):
    d = ctypes.byref(desc())
    assert lib.pa_decode(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 4, 1, d, 0.1, 0, None, 0, None, None) == 2
    assert lib.pa_prefill(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 10, 4, 4, 5, d, 0.1, None, None) == 2
    assert lib.pa_reshape_and_cache(FAKE, FAKE, FAKE, FAKE, FAKE, 2, d, None, None) == 2
    assert lib.pa_reshape_and_cache_fp8(FAKE, FAKE, FAKE, FAKE, FAKE, 2, d, 1.0, 1.0, None, None) == 2
    assert lib.pa_decode_window(FAKE, FAKE, FAKE, FAKE, None, None, FAKE, FAKE, 2, 4, 4, d, 0.1, 8, 0, None, None, None) == 2
    assert lib.pa_prefill_window(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 2, 10, 4, 4, 5, d, 0.1, 8, 0, 1.0, 1.0, None,
                                 None) == 2
    assert lib.pa_rope_and_cache(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 512, 512, 256, 256, FAKE, FAKE, FAKE, 4, 4, 128, 0, 1.0, d,
                                 1.0, 1.0, None, None) == 2
    assert lib.pa_copy_blocks(FAKE, FAKE, FAKE, -1, d, None, None) == 3
    assert lib.pa_copy_blocks(FAKE, FAKE, FAKE, 2, ctypes.byref(desc(bs=8)), None, None) == 2


def rope(lib, d=desc(dtype=pa.PA_F16), q_out=FAKE, k=FAKE, v=FAKE, q=0x900000, key=0x1900000, value=0x2900000, axes=3,
         pairs=bytes([0, 1, 2, 2]), pos=FAKE, t=4, hq=4, rotary=8, rows=pa.PA_F16, ku=0.0, vu=0.0, ks=256):
    return lib.pa_rope_axes_and_cache(q_out, k, v, q, key, value, 512, 512, ks, 256, pos, axes, pairs, FAKE, FAKE, t, hq,
                                      rotary, 0, 1.0, ctypes.byref(d), rows, ku, vu, None, None)


def test_rope_axes_refusals(lib):
    assert rope(lib, axes=0) == 3 and rope(lib, axes=5) == 3 and rope(lib, axes=2) == 3  # an axis that is not there
    assert rope(lib, pairs=None) == 1 and rope(lib, pos=None) == 1
    assert rope(lib, rotary=7) == 3 and rope(lib, rotary=130) == 3
    assert rope(lib, desc(d=96, dtype=pa.PA_F16)) == 2 and rope(lib, desc(dtype=9)) == 2
    assert rope(lib, desc(), rows=pa.PA_F32, ku=1.0, vu=1.0) == 2
    assert rope(lib, desc(), ku=0.0, vu=1.0) == 3 and rope(lib, desc(), ku=1.0, vu=math.nan) == 3
    assert rope(lib, ks=248) == 3 and rope(lib, ks=260) == 5
    assert rope(lib, t=0, key=None) == 0


def extend(lib, bt=FAKE, sl=FAKE, held=FAKE, free=FAKE, nf=FAKE, new=FAKE, slots=FAKE, pos=FAKE, qs=FAKE, n=3, rows=9, m=4,
           bs=16, nb=20):
    return lib.pa_tables_extend(bt, sl, held, free, nf, new, slots, pos, qs, n, rows, m, bs, nb, None, None)


def trim(lib, bt=FAKE, sl=FAKE, held=FAKE, free=FAKE, nf=FAKE, new=FAKE, n=3, m=4, bs=16, nb=20):
    return lib.pa_tables_trim(bt, sl, held, free, nf, new, n, m, bs, nb, None, None)


def test_tables_refusals(lib):
    for call in (extend, trim):
        for kw in (dict(n=-1), dict(m=-1), dict(bs=0), dict(nb=-1)):
            assert call(lib, **kw) == 3, kw
        for name in ("bt", "sl", "held", "free", "nf", "new"):
            assert call(lib, **{name: None}) == 1
            assert call(lib, **{name: FAKE + 2}) == 5
        assert call(lib, n=16385) == 7 and call(lib, m=1 << 28) == 7
    assert extend(lib, rows=-1) == 3 and extend(lib, qs=None) == 1 and extend(lib, slots=None) == 1
    assert extend(lib, slots=FAKE + 4) == 5 and extend(lib, qs=FAKE + 1) == 5
    assert extend(lib, n=0, rows=0, nf=None) == 0 and trim(lib, n=0, nf=None) == 0


def test_binding_refusals():
    import torch
    k, v = pa.fp4_cache(2, 1, 32, device="cpu"), pa.fp4_cache(2, 1, 32, device="cpu")
    assert k.shape == (2, 1, 2, 1152)
    d = pa.fp4_cache_desc(k)
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype) == (2, 32, 1, 128, pa.PA_FP4_E2M1)
    with pytest.raises(ValueError):
        pa.fp4_cache(2, 1, 24, device="cpu")
    with pytest.raises(ValueError):
        pa.fp4_cache_desc(torch.zeros(2, 1, 32, 128, dtype=torch.uint8))
    x = torch.zeros(1, 1, 128, dtype=torch.float16)
    with pytest.raises(ValueError):  # host caches
        pa.pa_reshape_and_cache_fp4(k, v, x, x, torch.zeros(1, dtype=torch.int64), 1.0, 1.0)
    with pytest.raises(ValueError):
        pa.pa_tables_trim(*(torch.zeros(1, 1, dtype=torch.int32),) * 6, 16)
    assert pa.pa_rope_pair_axes((1, 3, 2)) == bytes([0, 1, 1, 1, 2, 2])
    assert pa.pa_rope_pair_axes((1, 3, 2), interleaved=True) == bytes([0, 1, 2, 1, 2, 1])


def test_reference_rounds_to_the_nearest():
    """The tests' own quantisation against a search over every number that a group of its scale can hold."""
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 128)) * 2.0 ** rng.integers(-8, 4, (50, 1))).astype(np.float32)
    unit = np.float32(0.01)
    codes, scales = quantise(x, unit)
    got = values(codes, scales, unit).reshape(50, 8, 16)
    step = values(np.full((50, 64), 0x22, np.uint8), scales, unit).reshape(50, 8, 16)  # 1.0 of each group
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    grid = np.concatenate([-grid, grid])
    far = np.abs(x.reshape(50, 8, 16)[..., None].astype(np.float64) - grid * step[..., None])
    assert np.all(np.abs(got - x.reshape(50, 8, 16)) <= far.min(-1) + np.abs(x.reshape(50, 8, 16)) * 2.0 ** -22)
