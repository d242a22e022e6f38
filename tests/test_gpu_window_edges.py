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
