"""What the Python binding of 4-bit caches, tables and rotary axes passes on, without a GPU."""
import ctypes

import pytest
import torch

import paged_kv_cache_32_gb300 as pa


@pytest.fixture()
def rope(monkeypatch):
    """pa_rope_axes_and_cache over a 4-bit cache of host memory; returns the arguments of the C call."""
    args = []
    desc = pa.pa_cache_desc(4, 16, 1, 128, pa.PA_FP4_E2M1)
    monkeypatch.setattr(pa, "_caches_fp4", lambda k, v, d, rows, where: (0, desc, pa.PA_F16))
    monkeypatch.setattr(pa, "_rope", lambda *a: (2, 3, 0, 0, 384, 384, 128, 128, None))
    monkeypatch.setattr(pa, "_launch", lambda fn, dev, a, where: args.append(a))
    cache = pa.fp4_cache(4, 1, 16, device="cpu")
    q, kv = torch.zeros(2, 3, 128, dtype=torch.float16), torch.zeros(2, 1, 128, dtype=torch.float16)
    pos, slots = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64)

    def call(pair_axis=bytes([0, 1, 1, 0]), **kw):
        pairs = 4
        pa.pa_rope_axes_and_cache(q, cache, cache, q, kv, kv, pos, slots, torch.zeros(pairs, dtype=torch.float64), pair_axis,
                                  stream=0, **kw)
        return args[-1]

    return call


@pytest.mark.parametrize("kw", [{}, dict(k_scale=0.1), dict(v_scale=0.1), dict(k_scale=None, v_scale=0.1)])
def test_rope_over_a_4_bit_cache_needs_its_units(rope, kw):
    with pytest.raises(ValueError, match="units"):
        rope(**kw)


@pytest.mark.parametrize("k_unit,v_unit", [(0.25, 0.5), (0.0, 0.5), (0.25, 0.0), (-1.0, 0.5)])
def test_rope_passes_units_as_they_are(rope, k_unit, v_unit):
    """No number becomes another one: the C call refuses those that are no unit."""
    assert rope(k_scale=k_unit, v_scale=v_unit)[-4:-2] == (k_unit, v_unit)


@pytest.mark.parametrize("given", [bytes([0, 1, 1, 0]), bytearray([0, 1, 1, 0]), [0, 1, 1, 0], (0, 1, 1, 0),
                                   torch.tensor([0, 1, 1, 0]), torch.tensor([0, 1, 1, 0], dtype=torch.int32).numpy(),
                                   torch.tensor([0, 1, 1, 0], dtype=torch.uint8).numpy()])
def test_pair_axis_in_any_form(rope, given):
    assert rope(given, k_scale=0.1, v_scale=0.1)[12] == bytes([0, 1, 1, 0])


@pytest.mark.parametrize("given", [4, [0, 1, 1], torch.zeros(1, dtype=torch.int32).numpy(), [0, 256, 0, 0], [0, -1, 0, 0], None])
def test_pair_axis_that_is_none(rope, given):
    """A number is no sequence, and four bytes of one element are not four axes."""
    with pytest.raises((TypeError, ValueError)):
        rope(given, k_scale=0.1, v_scale=0.1)


def test_descriptor_of_a_4_bit_cache():
    """A cache's own descriptor is the one that pa_copy_blocks takes; those of other caches stay what they were."""
    k = pa.fp4_cache(5, 2, 48, device="cpu")
    d = pa.cache_desc(k)
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype) == (5, 48, 2, 128, pa.PA_FP4_E2M1)
    d = pa.cache_desc(torch.zeros(5, 2, 32, 128, dtype=torch.uint8))
    assert (d.num_blocks, d.block_size, d.num_kv_heads, d.head_size, d.dtype) == (5, 32, 2, 128, pa.PA_FP8_E4M3)
    d = pa.cache_desc(torch.zeros(1, 1, 1, 1152))
    assert (d.head_size, d.dtype) == (1152, pa.PA_F32)


def test_copy_blocks_knows_a_4_bit_cache(monkeypatch):
    got = []

    class Library:
        def pa_copy_blocks(self, *args):
            d = ctypes.cast(args[4], ctypes.POINTER(pa.pa_cache_desc)).contents
            got.append((d.block_size, d.dtype))  # (it lives as long as the call)
            return 0

    monkeypatch.setattr(pa, "lib", Library)
    k = pa.fp4_cache(5, 2, 48, device="cpu")
    pa.pa_copy_blocks(k, k, torch.zeros(1, 2, dtype=torch.int32), stream=0)
    assert got == [(48, pa.PA_FP4_E2M1)]
