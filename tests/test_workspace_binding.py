"""The workspace that the Python binding takes for a decode call that was given none, without a GPU: its device and the
stream whose memory it is."""
import pytest
import torch

import paged_kv_cache_32_gb300 as pa

NEED, CURRENT = 4096, 0x7000


class Library:
    """In the library's place: every call succeeds, and a workspace is wanted."""

    def __getattr__(self, name):
        return lambda *args: NEED if name.endswith("workspace_size") else 0


@pytest.fixture()
def taken(monkeypatch):
    """(device, stream) of each workspace; the stream as its handle, None for the current one."""
    log, inside, real = [], [None], torch.empty

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            inside.append(self.stream)

        def __exit__(self, *exc):
            inside.pop()

    def empty(*args, device=None, **kw):
        log.append((device, inside[-1]))
        return real(*args, **kw)

    monkeypatch.setattr(pa, "lib", Library)
    monkeypatch.setattr(pa, "_FP4_WORKSPACE", {})
    monkeypatch.setattr(pa, "_launch", lambda fn, dev, args, where: fn(*args))
    monkeypatch.setattr(pa, "_stream", lambda stream: 0)
    monkeypatch.setattr(pa, "_stream_of", lambda dev, stream: 0)
    monkeypatch.setattr(pa, "_attention_fp4", lambda where, host, out, q, k, v, table, lens, err, desc:
                        (0, pa.PA_F16, pa.pa_cache_desc(4, 16, 2, 128, pa.PA_FP4_E2M1), None, q.shape, table.shape))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: handle)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: CURRENT)
    return log


# (caches on a device of their own: the "meta" one; queries in host memory)
Q = torch.zeros(3, 4, 128, dtype=torch.float16)
CACHE = torch.zeros(4, 2, 16, 128, dtype=torch.float16, device="meta")
TABLE, LENS = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
CALLS = {
    "pa_decode": lambda **kw: pa.pa_decode(Q, Q, CACHE, CACHE, TABLE, LENS, 0.1, **kw),
    "pa_decode_append": lambda **kw: pa.pa_decode_append(Q, Q, CACHE, CACHE, Q, Q, TABLE, LENS, 0.1, **kw),
    "pa_decode_fp4": lambda **kw: pa.pa_decode_fp4(Q, Q, CACHE, CACHE, TABLE, LENS, 0.1, 1.0, 1.0, **kw),
}


@pytest.mark.parametrize("name", CALLS)
def test_device_is_the_caches(taken, name):
    """Queries may lie in pinned host memory; the kernels' scratch never does."""
    CALLS[name]()
    assert taken == [(CACHE.device, None)]


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("stream,want", [(0x5550, 0x5550), (type("S", (), {"cuda_stream": 0x6660}), 0x6660), (CURRENT, None),
                                         (None, None), (0, 0), (1, 0), (2, 2)])
def test_memory_is_the_streams(taken, name, stream, want):
    """Taken from another stream's memory, it would go to that stream's next tensors while the call still uses it."""
    CALLS[name](stream=stream)
    assert taken == [(CACHE.device, want)]


def test_alibi_takes_none(taken, monkeypatch):
    """ALiBi decode over a 4-bit cache never uses one."""
    monkeypatch.setattr(pa, "_refuse", lambda *args: None)
    pa.pa_decode_fp4(Q, Q, CACHE, CACHE, TABLE, LENS, 0.1, 1.0, 1.0, alibi_slopes=torch.zeros(4))
    assert taken == []
