"""Block tables on the GPU: batches without a request, and decode calls right behind (needs a GB300)."""
import numpy as np
import pytest

from test_gpu_tables import Device, Model

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


@pytest.mark.parametrize("rows", [0, 3])
def test_no_requests(pa, rows):
    """query_start is the one sum there is, 0, whatever it held; the stack stays."""
    d = Device(Model(0, 4, 16, 8, np.random.default_rng(0)), rows)
    free = d.free.clone()
    for _ in range(2):
        d.extend(pa, [])
        assert d.error() == 0 and d.start.tolist() == [0] and d.slots.tolist() == [-1] * rows
        d.start.fill_(77)
        d.trim(pa, [])
    assert d.top.tolist() == [8] and d.free.tolist() == free.tolist()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp4"])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_right_behind(pa, dtype, captured):
    """Decode launched behind extend and trim sees their lengths and tables: every value is its offset in the block and
    every weight the same, so that an output is the mean of a length's offsets."""
    import torch
    n, B, width, steps = 64, 16, 20, 40
    m = Model(n, width, B, n * width, np.random.default_rng(1))
    d = Device(m, 3 * n)
    nb, rows = n * width, {"f32": torch.float32, "bf16": torch.bfloat16, "fp4": torch.float16}[dtype]
    off = torch.arange(B, device="cuda", dtype=rows)
    if dtype == "fp4":
        k, v = pa.fp4_cache(nb, 1, B), pa.fp4_cache(nb, 1, B)
        # (offsets 0, 8, 16 .. of E2M1: what a group of equal numbers holds exactly)
        value = (off[:, None, None] * 8).expand(B, 1, 128).repeat(nb, 1, 1).contiguous()
        pa.pa_reshape_and_cache_fp4(k, v, torch.zeros_like(value), value, torch.arange(nb * B, device="cuda"), 1.0, 1.0)
        off = torch.zeros_like(value)
        pa.pa_read_cache_fp4(off, off.clone(), v, v, torch.arange(nb * B, device="cuda"), 1.0, 1.0)
        off = off[:B, 0, 0]
    else:
        k = torch.zeros(nb, 1, B, 128, dtype=rows, device="cuda")
        v = off[None, None, :, None].expand(nb, 1, B, 128).contiguous()
    q = torch.ones(n, 2, 128, dtype=rows, device="cuda")
    out = torch.zeros_like(q)
    new, keep = (torch.zeros(n, dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        pa.pa_tables_trim(d.table, d.lens, d.held, d.free, d.top, keep, B, err_flag=d.err)
        pa.pa_tables_extend(d.table, d.lens, d.held, d.free, d.top, new, d.slots, d.pos, d.start, B, err_flag=d.err)
        if dtype == "fp4":
            pa.pa_decode_fp4(out, q, k, v, d.table, d.lens, 0.1, 1.0, 1.0, err_flag=d.err)
        else:
            pa.pa_decode(out, q, k, v, d.table, d.lens, 0.1, err_flag=d.err)

    step()
    torch.cuda.synchronize()
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    outs, want = [], []
    mean = np.cumsum(np.tile(off.double().cpu().numpy(), width)) / np.arange(1, width * B + 1)
    for i in range(steps):
        kept = np.maximum(0, m.lens - (np.arange(n) + i) % 3)
        grown = (np.arange(n) * 7 + i * 5) % 4 * (np.arange(n) % 5 != i % 5) if i else np.arange(n) % 3
        keep.copy_(torch.from_numpy(kept.astype(np.int32)))
        new.copy_(torch.from_numpy(grown.astype(np.int32)))
        graph.replay() if captured else step()
        outs.append(out[:, :, 0].clone())
        m.trim(kept)
        m.extend(grown, 3 * n)
        want.append(np.where(m.lens > 0, mean[np.maximum(m.lens, 1) - 1], 0.0))
    torch.cuda.synchronize()
    d.check()
    assert d.error() == 0
    got, want = torch.stack(outs).double().cpu().numpy(), np.stack(want)[:, :, None]
    # equal weights: rounding of fp32 sums, and of the output to its type
    eps = {"f32": 2.0 ** -18, "bf16": 2.0 ** -8, "fp4": 2.0 ** -10}[dtype]
    assert np.all(np.abs(got - want) <= eps * want)
