"""What the Python binding of rotary positions and windowed attention passes to the C calls, without a GPU: integers
past int32, which ctypes wraps without a word, never arrive as others."""
import ctypes

import pytest

import paged_kv_cache_32_gb300 as pa

WRAPPED = 2 ** 32


class Recorder:
    """In the library's place: a call of any name is kept and reports success."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture()
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(pa, "lib", lambda: r)
    monkeypatch.setattr(pa, "status_string", lambda status: "")
    return r


@pytest.mark.parametrize("rotary_dim", [-WRAPPED + 128, -WRAPPED + 2, -2 ** 31, -2, 0, 1, 130, WRAPPED + 64, WRAPPED])
def test_rope_frequencies_sizes_that_have_no_room(recorder, rotary_dim):
    """The C call writes rotary_dim / 2 numbers: a size that would wrap into another must not reach it."""
    with pytest.raises(pa.PaError):
        pa.pa_rope_frequencies(rotary_dim)
    assert recorder.calls == []


@pytest.mark.parametrize("method", [-WRAPPED, WRAPPED, WRAPPED + 1, -1, 5])
def test_rope_frequencies_methods_that_wrap(recorder, method):
    with pytest.raises(pa.PaError):
        pa.pa_rope_frequencies(64, method=method, factor=2.0)
    assert recorder.calls == []


def test_rope_frequencies_sizes_that_fit(recorder):
    pa.pa_rope_frequencies(128)
    assert recorder.calls[0][1][2] == 128


@pytest.fixture()
def launched(monkeypatch):
    """The calls' integers as the C side gets them, with host tensors in the caches' place."""
    import torch
    args = []
    desc = pa.pa_cache_desc(4, 16, 2, 128, pa.PA_BF16)
    monkeypatch.setattr(pa, "_attention",
                        lambda where, host, out, q, *rest: (-1, q.dtype, desc, None, q.shape, rest[2].shape))
    monkeypatch.setattr(pa, "lib", Recorder)
    monkeypatch.setattr(pa, "_launch", lambda fn, dev, a, where: args.append(a))
    q = torch.zeros(6, 4, 128, dtype=torch.bfloat16)
    cache, table = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16), torch.zeros(6, 2, dtype=torch.int32)

    def decode(window, sinks):
        pa.pa_decode_window(q, q, cache, cache, table, table[:, 0], 0.1, window, num_sinks=sinks, stream=0)
        return [ctypes.c_int32(args[-1][i]).value for i in (13, 14)]

    def prefill(window, sinks, most=3):
        pa.pa_prefill_window(q, q, cache, cache, table, table[:, 0], torch.zeros(7, dtype=torch.int32), most, 0.1, window,
                             num_sinks=sinks, stream=0)
        return [ctypes.c_int32(args[-1][i]).value for i in (14, 15, 11)]

    return decode, prefill


@pytest.mark.parametrize("value", [0, 1, 8, 2 ** 31 - 1, 2 ** 31, WRAPPED + 8, 2 ** 70, -1, -2 ** 31, -2 ** 31 - 1, -WRAPPED,
                                   -WRAPPED + 8, -2 ** 70])
def test_window_integers_keep_their_side_of_zero(launched, value):
    """A window, a number of first tokens or a chunk's bound past int32 arrives as the end of int32 on its own side, which
    the call takes as everything or refuses, never as another number."""
    decode, prefill = launched
    want = max(-2 ** 31, min(value, 2 ** 31 - 1))
    assert decode(value, 0) == [want, 0] and decode(5, value) == [5, want]
    assert prefill(value, 0) == [want, 0, 3] and prefill(5, value) == [5, want, 3]
    assert prefill(5, 0, value) == [5, 0, min(want, 6)]  # (a batch of six queries)


@pytest.mark.parametrize("kw", [
    dict(method=3, factor=2.0, original_max_position=100.0, attention_factor=float("inf")),
    dict(method=3, factor=2.0, original_max_position=100.0, attention_factor=1e39),   # past fp32, the magnitude's type
    dict(method=4, factor=2.0, original_max_position=100.0, high_freq_factor=float("inf")),
    dict(method=1, factor=1e-320),                                                    # 1 / factor past fp64
    dict(method=3, factor=1e-320, original_max_position=100.0),
    dict(method=2, factor=1e300),                                                     # base * factor^(r / (r - 2))
])
def test_rope_frequencies_are_finite(kw):
    """Frequencies and magnitude that come out without a NaN or an infinity, or an error."""
    pa.build()
    with pytest.raises(pa.PaError):
        pa.pa_rope_frequencies(64, **{"base": 10000.0, **kw})
