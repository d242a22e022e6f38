"""Decode calls that take their own workspace: queries in pinned host memory, several streams (needs a GB300)."""
import numpy as np
import pytest

import workloads as W
from fp4_ref import K_UNIT, V_UNIT, Fp4Case
from harness import GpuStep, oracle_step, out_f64, to_torch, within_bound
from test_gpu_fp4 import within_bound as within_bound_fp4

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def pa():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_32_gb300 as pa
    pa.build()
    return pa


def pinned(t):
    import torch
    h = torch.empty(t.shape, dtype=t.dtype).pin_memory()
    h.copy_(t.cpu())
    return h


class Fp4:
    """A decode step over a 4-bit cache whose sizes take a workspace."""

    def __init__(self, pa, seed):
        import torch
        self.pa, rng = pa, np.random.default_rng(seed)
        lens = [int(x) for x in rng.integers(1, 700, 20)] + [3000]
        self.w = w = Fp4Case("f16", lens, [1] * len(lens), 8, 2, 16, 2 ** 31 - 1, 0, seed=seed, slack_blocks=2300)
        self.k, self.v = torch.from_numpy(w.k_cache).cuda(), torch.from_numpy(w.v_cache).cuda()
        self.q, self.table = to_torch(w.q, "f16"), torch.from_numpy(w.table).cuda()
        self.lens = torch.tensor(w.lens, dtype=torch.int32, device="cuda")
        self.out, self.err = torch.zeros_like(self.q), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.need = pa.pa_decode_fp4_workspace_size(len(lens), 8, w.width, pa.fp4_cache_desc(self.k))
        assert self.need > 0

    def run(self, q=None, out=None, **kw):
        self.pa.pa_decode_fp4(self.out if out is None else out, self.q if q is None else q, self.k, self.v, self.table,
                              self.lens, self.w.scale, K_UNIT, V_UNIT, err_flag=self.err, **kw)

    def check(self, out=None):
        import torch
        torch.cuda.synchronize()
        assert int(self.err.item()) == 0
        ok, err, ratio = within_bound_fp4(out_f64(self.out if out is None else out), self.w.reference(), "f16")
        assert ok, f"max abs err {err}, worst err/bound {ratio}"


def test_fp4_decode_with_host_queries(pa):
    s = Fp4(pa, 1)
    out = pinned(s.out)
    s.run(q=pinned(s.q), out=out)
    s.check(out)


@pytest.mark.parametrize("append", [False, True])
def test_decode_with_host_queries(pa, append):
    """Long contexts in partitions: their partial results go through the workspace."""
    import torch
    w = W.build_decode("host_ws", seed=6, dtype="f16", seq_lens=[3000, 17, 1500], num_q_heads=8, num_kv_heads=2, head_size=128,
                       block_size=16, pool_factor=1.2, append_last=append, partition_size=512)
    s = GpuStep(w)
    assert pa.pa_decode_workspace_size(3, 8, s.tables.shape[1], s.desc, 512) > 0
    out = pinned(s.out)
    if append:
        pa.pa_decode_append(out, pinned(s.q), s.k, s.v, pinned(s.nk), pinned(s.nv), s.tables, s.lens, w.scale,
                            partition_size=512, err_flag=s.err, desc=s.desc)
    else:
        pa.pa_decode(out, pinned(s.q), s.k, s.v, s.tables, s.lens, w.scale, partition_size=512, err_flag=s.err, desc=s.desc)
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0
    ok, err, ratio = within_bound(out_f64(out), oracle_step(w)[2], "f16")
    assert ok, f"max abs err {err}, worst err/bound {ratio}"


def busy(torch, stream, us=3000):
    with torch.cuda.stream(stream):
        torch.cuda._sleep(int(us * 2000))


@pytest.mark.parametrize("form", ["object", "handle"])
def test_fp4_decode_on_streams_of_its_own(pa, form):
    """Two calls on two streams that are not torch's current one, at once, and tensors made on the current one meanwhile:
    each call's scratch is its own."""
    import torch
    steps, streams = [Fp4(pa, 3), Fp4(pa, 4)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for st in streams:
            busy(torch, st)
        for s, st in zip(steps, streams):
            s.run(stream=st if form == "object" else st.cuda_stream)
            junk = [torch.full((s.need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        for s in steps:
            s.check()
            s.out.zero_()
        del junk


def test_decode_on_a_stream_of_its_own(pa):
    import torch
    w = W.build_decode("stream_ws", seed=7, dtype="bf16", seq_lens=[3000, 17, 1500], num_q_heads=8, num_kv_heads=2,
                       head_size=128, block_size=16, pool_factor=1.2, partition_size=512)
    s, st = GpuStep(w), torch.cuda.Stream()
    need = pa.pa_decode_workspace_size(3, 8, s.tables.shape[1], s.desc, 512)
    torch.cuda.synchronize()
    busy(torch, st)
    pa.pa_decode(s.out, s.q, s.k, s.v, s.tables, s.lens, w.scale, partition_size=512, err_flag=s.err, stream=st, desc=s.desc)
    junk = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert int(s.err.item()) == 0 and bool((junk == 0xFF).all())
    ok, err, ratio = within_bound(out_f64(s.out), oracle_step(w)[2], "bf16")
    assert ok, f"max abs err {err}, worst err/bound {ratio}"


def test_fp4_decode_captured_on_a_stream_of_its_own(pa):
    """In a capture the scratch comes from the graph's memory; replayed beside other work it is still the graph's."""
    import torch
    s, st = Fp4(pa, 5), torch.cuda.Stream()
    s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        s.run(stream=st)
    s.out.zero_()
    junk = [torch.full((s.need,), 0xFF, dtype=torch.uint8, device="cuda") for _ in range(4)]
    graph.replay()
    s.check()
    assert all(bool((x == 0xFF).all()) for x in junk)
