"""Rotary positions and windowed attention without a GPU: refusals, in which nothing is launched, and the frequencies."""
import ctypes
import math

import numpy as np
import pytest

import paged_kv_cache_32_gb300 as pa

FAKE = 0x10000  # never dereferenced: every call below is rejected before any CUDA call


@pytest.fixture(scope="module")
def lib():
    pa.build()
    return pa.lib()


def desc(nb=16, bs=16, hkv=2, d=128, dtype=pa.PA_F16):
    return pa.pa_cache_desc(nb, bs, hkv, d, dtype)


def decode(lib, d, out=FAKE, q=FAKE, k=FAKE, v=FAKE, key=None, value=None, bt=FAKE, sl=FAKE, n=2, hq=4, m=4, scale=0.1,
           window=8, sinks=0, opts=None):
    return lib.pa_decode_window(out, q, k, v, key, value, bt, sl, n, hq, m, ctypes.byref(d), scale, window, sinks, None,
                                None, opts)


def test_decode_window_refusals(lib):
    assert decode(lib, desc(d=96)) == 2
    assert decode(lib, desc(dtype=7)) == 2
    assert decode(lib, desc(bs=24)) == 2
    assert decode(lib, desc(bs=8, dtype=pa.PA_FP8_E4M3)) == 2
    assert decode(lib, desc(), hq=3) == 3
    assert decode(lib, desc(), n=-1) == 3
    assert decode(lib, desc(), window=0) == 3
    assert decode(lib, desc(), window=-5) == 3
    assert decode(lib, desc(), sinks=-1) == 3
    assert decode(lib, desc(), scale=float("nan")) == 3
    assert decode(lib, desc(), scale=float("inf")) == 3
    assert decode(lib, desc(), out=None) == 1
    assert decode(lib, desc(), sl=None) == 1
    assert decode(lib, desc(), bt=None) == 1
    assert decode(lib, desc(), key=FAKE) == 1                        # key and value go together
    assert decode(lib, desc(dtype=pa.PA_F32), key=FAKE, value=FAKE) == 2
    assert decode(lib, desc(), k=FAKE + 2) == 5
    assert decode(lib, desc(), q=FAKE + 4) == 5
    assert decode(lib, desc(), key=FAKE, value=FAKE + 8) == 5
    assert decode(lib, desc(), sl=FAKE + 2) == 5
    assert decode(lib, desc(), m=1 << 28) == 7
    assert decode(lib, desc(nb=1 << 30, hkv=8)) == 7
    bad = pa.pa_decode_options(None, -1.0, 0.0, 0)
    assert decode(lib, desc(dtype=pa.PA_FP8_E4M3), opts=ctypes.byref(bad)) == 3
    assert decode(lib, desc(), n=0, out=None) == 0


def prefill(lib, d, out=FAKE, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, sl=FAKE, qs=FAKE, n=2, t=10, hq=4, m=4, most=5, scale=0.1,
            window=8, sinks=0, ks=0.0, vs=0.0):
    return lib.pa_prefill_window(out, q, k, v, bt, sl, qs, n, t, hq, m, most, ctypes.byref(d), scale, window, sinks, ks, vs,
                                 None, None)


def test_prefill_window_refusals(lib):
    assert prefill(lib, desc(d=32)) == 2
    assert prefill(lib, desc(bs=24)) == 2
    assert prefill(lib, desc(), hq=5) == 3
    assert prefill(lib, desc(), t=-1) == 3
    assert prefill(lib, desc(), most=-1) == 3
    assert prefill(lib, desc(), scale=0.0) == 3
    assert prefill(lib, desc(), scale=-1.0) == 3
    assert prefill(lib, desc(), window=0) == 3
    assert prefill(lib, desc(), sinks=-1) == 3
    assert prefill(lib, desc(dtype=pa.PA_FP8_E4M3), ks=float("nan")) == 3
    assert prefill(lib, desc(), qs=None) == 1
    assert prefill(lib, desc(), q=None) == 1
    assert prefill(lib, desc(), out=FAKE + 8) == 5
    assert prefill(lib, desc(), qs=FAKE + 1) == 5
    assert prefill(lib, desc(), m=1 << 28) == 7
    assert prefill(lib, desc(), t=1 << 31 - 1, hq=1 << 12) == 7
    assert prefill(lib, desc(), most=0, out=None) == 0
    assert prefill(lib, desc(), t=0, out=None) == 0


def rope(lib, d, q_out=FAKE, k=FAKE, v=FAKE, q=0x900000, key=0x1900000, value=0x2900000, qos=512, qs=512, ks=256, vs=256,
         pos=FAKE, slot=FAKE, inv=FAKE, t=4, hq=4, rotary=128, inter=0, mag=1.0, k_scale=0.0, v_scale=0.0):
    return lib.pa_rope_and_cache(q_out, k, v, q, key, value, qos, qs, ks, vs, pos, slot, inv, t, hq, rotary, inter, mag,
                                 ctypes.byref(d), k_scale, v_scale, None, None)


def test_rope_refusals(lib):
    assert rope(lib, desc(d=96)) == 2
    for rotary in (0, 1, 3, 130, -2):
        assert rope(lib, desc(), rotary=rotary) == 3
    assert rope(lib, desc(), inter=2) == 3
    assert rope(lib, desc(), mag=float("nan")) == 3
    assert rope(lib, desc(), t=-1) == 3
    assert rope(lib, desc(), hq=-1) == 3
    assert rope(lib, desc(dtype=pa.PA_FP8_E4M3), k_scale=-1.0) == 3
    assert rope(lib, desc(), qs=511 - 7) == 3                        # shorter than the row
    assert rope(lib, desc(), ks=0) == 3
    assert rope(lib, desc(), inv=None) == 1
    assert rope(lib, desc(), slot=None) == 1
    assert rope(lib, desc(), q_out=None) == 1
    assert rope(lib, desc(), qs=516) == 5                            # rows not 16 bytes apart
    assert rope(lib, desc(dtype=pa.PA_F32), ks=258) == 5
    assert rope(lib, desc(), key=0x1900008) == 5
    assert rope(lib, desc(), slot=FAKE + 4) == 5
    assert rope(lib, desc(), inv=FAKE + 4) == 5
    assert rope(lib, desc(), q_out=0x900010) == 3                    # overlaps q without being it
    assert rope(lib, desc(), q_out=0x900000, qos=520) == 3           # q itself, other rows
    assert rope(lib, desc(), q_out=0x1900000) == 3                   # on the keys
    # one fused buffer of rows [q | key | value]: q_out on another row's keys
    fused = dict(q=0x900000, key=0x900000 + 1024, value=0x900000 + 1536, qs=1024, ks=1024, vs=1024, qos=1024)
    assert rope(lib, desc(), q_out=0x900000 + 512, **fused) == 3
    assert rope(lib, desc(), q_out=0x900000 + 2048 * 3, **fused) == 3
    assert rope(lib, desc(), ks=1 << 45) == 7
    assert rope(lib, desc(), t=0, key=None) == 0


def freqs(rotary, base, **kw):
    f, m = pa.pa_rope_frequencies(rotary, base, **kw)
    return f.numpy(), m


def test_rope_frequencies(lib):
    for r in (2, 6, 64, 128):
        j = np.arange(r // 2)
        plain = 10000.0 ** (-2.0 * j / r)
        f, m = freqs(r, 10000.0)
        assert m == 1.0 and np.allclose(f, plain, rtol=1e-14)
        f, m = freqs(r, 10000.0, method=pa.PA_ROPE_LINEAR, factor=8.0)
        assert m == 1.0 and np.allclose(f, plain / 8, rtol=1e-14)
    f, _ = freqs(64, 10000.0, method=pa.PA_ROPE_NTK, factor=4.0)
    j = np.arange(32)
    assert np.allclose(f, (10000.0 * 4.0 ** (64 / 62)) ** (-j / 32.0), rtol=1e-13)
    # the ends of the two ramps: fast pairs stay, slow ones are divided, between them it falls monotonously
    plain = 500000.0 ** (-np.arange(64) / 64.0)
    f, m = freqs(128, 500000.0, method=pa.PA_ROPE_YARN, factor=16.0, original_max_position=8192.0)
    assert abs(m - (0.1 * math.log(16.0) + 1.0)) < 1e-6
    assert freqs(128, 500000.0, method=pa.PA_ROPE_YARN, factor=16.0, original_max_position=8192.0,
                 attention_factor=1.25)[1] == 1.25
    share = f / plain
    turns = 8192.0 * plain / (2 * math.pi)
    # (the ramp's ends are rounded outwards to whole pairs: a pair beyond them by one turns ratio)
    step = 500000.0 ** (1 / 64)
    assert np.allclose(share[turns > 32 * step], 1.0) and np.allclose(share[turns < 1 / step], 1 / 16)
    assert np.all(np.diff(share) <= 1e-15)
    f, m = freqs(128, 500000.0, method=pa.PA_ROPE_BANDS, factor=8.0, original_max_position=8192.0)
    assert m == 1.0
    share = f / plain
    keep = np.clip((turns - 1.0) / 3.0, 0, 1)
    assert np.allclose(share, keep + (1 - keep) / 8, rtol=1e-13)


def test_rope_frequencies_refusals(lib):
    for args in ((3, 1e4), (0, 1e4), (130, 1e4), (64, 0.0), (64, float("inf")), (64, float("nan"))):
        with pytest.raises(pa.PaError):
            pa.pa_rope_frequencies(*args)
    for kw in (dict(method=5), dict(method=-1), dict(method=1, factor=0.0), dict(method=3, factor=2.0),
               dict(method=3, factor=2.0, original_max_position=100.0, beta_fast=0.0),
               dict(method=3, factor=2.0, original_max_position=100.0, attention_factor=-1.0),
               dict(method=4, factor=2.0, original_max_position=100.0, low_freq_factor=4.0),
               dict(method=4, factor=float("nan"), original_max_position=100.0)):
        with pytest.raises(pa.PaError):
            pa.pa_rope_frequencies(64, 1e4, **kw)
    with pytest.raises(pa.PaError):
        pa.pa_rope_frequencies(2, 1e4, method=pa.PA_ROPE_NTK, factor=2.0)


def test_binding_refuses_host_tensors(lib):
    import torch
    k = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        pa.pa_decode_window(q, q, k, k, i[:, None], i, 0.1, 8)
    with pytest.raises(ValueError):
        pa.pa_prefill_window(q, q, k, k, i[:, None], i, torch.zeros(3, dtype=torch.int32), 1, 0.1, 8)
    with pytest.raises(ValueError):
        pa.pa_rope_and_cache(q, k, k, q, q[:, :2], q[:, :2], i, i.long(), torch.ones(64, dtype=torch.float64))
