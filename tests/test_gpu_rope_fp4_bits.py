"""Rotary positions with the write: a call over a 4-bit cache turns rows to the bits of the same call over a 16-bit one,
whichever kernel the turned size takes (needs a GB300)."""
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


@pytest.mark.parametrize("rows", ["f16", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [128, 96, 32, 2, 24, 26, 34, 36, 48, 114, 126])
def test_same_bits(pa, rows, interleaved, rotary):
    import torch
    t = torch.float16 if rows == "f16" else torch.bfloat16
    T, hq, hkv, B = 4096, 8, 4, 32
    g = torch.Generator(device="cuda").manual_seed(rotary)
    x = torch.randn(T, hq + 2 * hkv, 128, generator=g, device="cuda").to(t)
    q, key, value = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    pos = torch.randint(0, 200000, (3, T), generator=g, device="cuda", dtype=torch.int32)
    slots = torch.randperm(T, generator=g, device="cuda")
    inv, mag = pa.pa_rope_frequencies(rotary, device="cuda")
    pairs = bytes(j % 3 for j in range(rotary // 2))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    k16, v16 = (torch.zeros(T // B, hkv, B, 128, dtype=t, device="cuda") for _ in range(2))
    k4, v4, k4b, v4b = (pa.fp4_cache(T // B, hkv, B) for _ in range(4))
    out16, out4 = torch.zeros(T, hq, 128, dtype=t, device="cuda"), torch.zeros(T, hq, 128, dtype=t, device="cuda")
    kw = dict(interleaved=interleaved, magnitude=mag, err_flag=err)
    pa.pa_rope_axes_and_cache(out16, k16, v16, q, key, value, pos, slots, inv, pairs, **kw)
    pa.pa_rope_axes_and_cache(out4, k4, v4, q, key, value, pos, slots, inv, pairs, k_scale=0.0025, v_scale=0.0031, **kw)
    assert torch.equal(out4.view(torch.int16), out16.view(torch.int16))
    # the rows that the 16-bit cache holds, through the append
    turned = k16.transpose(1, 2).reshape(T, hkv, 128)[slots].contiguous()
    pa.pa_reshape_and_cache_fp4(k4b, v4b, turned, value, slots, 0.0025, 0.0031, err_flag=err)
    assert int(err.item()) == 0 and torch.equal(k4, k4b) and torch.equal(v4, v4b)
