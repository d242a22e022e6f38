"""What the Python binding of rotary positions and windowed attention passes to the C calls, without a GPU: integers
past int32, which ctypes wraps without a word, never arrive as others."""
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
