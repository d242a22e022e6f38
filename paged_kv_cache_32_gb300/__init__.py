"""paged_kv_cache_32_gb300 - paged decode attention for GB300 (sm_103a).

Thin Python binding of the C ABI in ``include/pa.h`` (``libpa.so``), with the
same entry-point names.  It only marshals arguments: torch tensors provide
device memory and the current CUDA stream; every step of the computation runs
in the library's CUDA kernels.  There is no CPU or PyTorch fallback: if the
library has not been built, every entry point raises.

Cache layout expected by every call: K and V are each a dense tensor
[num_blocks, num_kv_heads, block_size, head_size] of float32, float16 or
bfloat16 on the GPU.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3 = 0, 1, 2, 3
PA_OK = 0
PA_DEVERR = {0: "none", 1: "block id out of range", 2: "slot out of range", 3: "copy pair id out of range",
             4: "wait on an asynchronous copy timed out", 5: "prefill chunk inconsistent with q, grid or sequence"}

EXPORTED = ("pa_decode", "pa_decode_ex", "pa_decode_append", "pa_decode_partition_size", "pa_decode_workspace_size",
            "pa_reshape_and_cache", "pa_copy_blocks", "pa_status_string", "pa_version", "pa_decode_noalloc", "pa_prefill",
            "pa_reshape_and_cache_fp8", "pa_rope_frequencies", "pa_rope_and_cache", "pa_decode_window",
            "pa_prefill_window")


PA_DECODE_TEST_EXPIRE_FIRST_WAIT = 1


class pa_decode_options(ctypes.Structure):
    _fields_ = [("alibi_slopes", ctypes.c_void_p), ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float),
                ("test_flags", ctypes.c_uint32)]


class pa_cache_desc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_size", ctypes.c_int32), ("dtype", ctypes.c_int32)]


PA_ROPE_PLAIN, PA_ROPE_LINEAR, PA_ROPE_NTK, PA_ROPE_YARN, PA_ROPE_BANDS = range(5)


class pa_rope_scaling(ctypes.Structure):
    _fields_ = [("method", ctypes.c_int32), ("factor", ctypes.c_double), ("original_max_position", ctypes.c_double),
                ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("attention_factor", ctypes.c_double),
                ("low_freq_factor", ctypes.c_double), ("high_freq_factor", ctypes.c_double)]


class PaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def lib_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """The loaded libpa.so.  Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(_build.LIB):
            raise ImportError(f"libpa.so is not built ({_build.LIB}); run paged_kv_cache_32_gb300.build.build()")
        L = ctypes.CDLL(_build.LIB)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        desc_p = ctypes.POINTER(pa_cache_desc)
        L.pa_decode.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, desc_p, ctypes.c_float, i32, vp, sz, vp, vp]
        L.pa_decode.restype = ctypes.c_int
        L.pa_decode_ex.argtypes = L.pa_decode.argtypes + [ctypes.POINTER(pa_decode_options)]
        L.pa_decode_ex.restype = ctypes.c_int
        L.pa_decode_append.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, desc_p, ctypes.c_float, i32, vp, sz,
                                       vp, vp, ctypes.POINTER(pa_decode_options)]
        L.pa_decode_append.restype = ctypes.c_int
        L.pa_prefill.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, desc_p, ctypes.c_float, vp, vp]
        L.pa_prefill.restype = ctypes.c_int
        L.pa_decode_partition_size.argtypes = [i32, desc_p, i32]
        L.pa_decode_partition_size.restype = i32
        L.pa_decode_workspace_size.argtypes = [i32, i32, i32, desc_p, i32]
        L.pa_decode_workspace_size.restype = sz
        L.pa_reshape_and_cache.argtypes = [vp, vp, vp, vp, vp, i32, desc_p, vp, vp]
        L.pa_reshape_and_cache.restype = ctypes.c_int
        L.pa_copy_blocks.argtypes = [vp, vp, vp, i32, desc_p, vp, vp]
        L.pa_reshape_and_cache_fp8.argtypes = [vp, vp, vp, vp, vp, i32, desc_p, ctypes.c_float, ctypes.c_float, vp, vp]
        L.pa_reshape_and_cache_fp8.restype = ctypes.c_int
        L.pa_copy_blocks.restype = ctypes.c_int
        f32 = ctypes.c_float
        L.pa_rope_frequencies.argtypes = [vp, vp, i32, ctypes.c_double, ctypes.POINTER(pa_rope_scaling)]
        L.pa_rope_frequencies.restype = ctypes.c_int
        L.pa_rope_and_cache.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp, vp, i32, i32, i32, i32, f32,
                                        desc_p, f32, f32, vp, vp]
        L.pa_rope_and_cache.restype = ctypes.c_int
        L.pa_decode_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, desc_p, f32, i32, i32, vp, vp,
                                       ctypes.POINTER(pa_decode_options)]
        L.pa_decode_window.restype = ctypes.c_int
        L.pa_prefill_window.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, desc_p, f32, i32, i32, f32,
                                        f32, vp, vp]
        L.pa_prefill_window.restype = ctypes.c_int
        L.pa_status_string.argtypes = [ctypes.c_int]
        L.pa_status_string.restype = ctypes.c_char_p
        L.pa_version.argtypes = []
        L.pa_version.restype = ctypes.c_int
        _lib = L
    return _lib


def build(force: bool = False) -> str:
    """Compile libpa.so in-tree for sm_103a (see build.py)."""
    global _lib
    path = _build.build(force=force)
    _lib = None
    return path


def status_string(status: int) -> str:
    return lib().pa_status_string(int(status)).decode()


def version() -> int:
    return lib().pa_version()


# ---------------------------------------------------------------- marshalling helpers
def _dtype_code(t) -> int:
    import torch
    codes = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.uint8: PA_FP8_E4M3}
    if hasattr(torch, "float8_e4m3fn"):
        codes[torch.float8_e4m3fn] = PA_FP8_E4M3
    if t.dtype not in codes:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return codes[t.dtype]


def cache_desc(k_cache) -> pa_cache_desc:
    """Descriptor of a [num_blocks, num_kv_heads, block_size, head_size] key-cache tensor
    (uint8 or float8_e4m3fn storage means an FP8 E4M3 cache, whose values are
    [num_blocks, num_kv_heads, block_size / 16, head_size, 16])."""
    if k_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_size]")
    nb, hkv, bs, d = (int(x) for x in k_cache.shape)
    return pa_cache_desc(nb, bs, hkv, d, _dtype_code(k_cache))


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _dense(t, name: str):
    if t is not None and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    return int(getattr(stream, "cuda_stream", stream))


def _check(status: int, where: str) -> None:
    if status != PA_OK:
        raise PaError(status, where)


# ---------------------------------------------------------------- entry points
def pa_decode_partition_size(max_blocks_per_seq: int, desc: pa_cache_desc, partition_size: int = 0) -> int:
    r = lib().pa_decode_partition_size(int(max_blocks_per_seq), ctypes.byref(desc), int(partition_size))
    if r < 0:
        raise PaError(-r, "pa_decode_partition_size")
    return r


def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, max_blocks_per_seq: int, desc: pa_cache_desc,
                             partition_size: int = 0) -> int:
    return int(lib().pa_decode_workspace_size(int(num_seqs), int(num_q_heads), int(max_blocks_per_seq),
                                              ctypes.byref(desc), int(partition_size)))


def pa_decode(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float, partition_size: int = 0,
              workspace=None, err_flag=None, stream=None, desc: pa_cache_desc | None = None,
              alibi_slopes=None, k_scale: float | None = None, v_scale: float | None = None,
              test_flags: int = 0) -> None:
    """out[s, h] = softmax(scale * q[s, h] K_s^T) V_s over seq_lens[s] paged tokens.

    out, q: [num_seqs, num_q_heads, head_size] (cache dtype); block_tables: int32
    [num_seqs, max_blocks_per_seq]; seq_lens: int32 [num_seqs].  ``workspace`` is a
    uint8 device tensor of at least pa_decode_workspace_size(...) bytes; when None
    and one is needed, it is allocated with torch.  ``alibi_slopes``: optional
    float32 device tensor [num_q_heads] (calls pa_decode_ex).  ``k_scale`` /
    ``v_scale``: dequantisation scales of an FP8 cache (q and out are fp16 then).
    ``test_flags``: 0, or PA_DECODE_TEST_EXPIRE_FIRST_WAIT in tests of the bounded waits.
    """
    desc = desc or cache_desc(k_cache)
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _dense(t, n)
    num_seqs, num_q_heads = int(q.shape[0]), int(q.shape[1])
    max_blocks = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    need = pa_decode_workspace_size(num_seqs, num_q_heads, max_blocks, desc, partition_size)
    if workspace is None and need > 0:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens), num_seqs,
            num_q_heads, max_blocks, ctypes.byref(desc), float(scale), int(partition_size), _ptr(workspace), ws_bytes,
            _ptr(err_flag), _stream(stream))
    if alibi_slopes is None and k_scale is None and v_scale is None and not test_flags:
        _check(lib().pa_decode(*args), "pa_decode")
    else:
        _dense(alibi_slopes, "alibi_slopes")
        opts = pa_decode_options(_ptr(alibi_slopes), float(k_scale or 0.0), float(v_scale or 0.0), int(test_flags))
        _check(lib().pa_decode_ex(*args, ctypes.byref(opts)), "pa_decode_ex")


def pa_decode_append(out, q, k_cache, v_cache, key, value, block_tables, seq_lens, scale: float,
                     partition_size: int = 0, workspace=None, err_flag=None, stream=None,
                     desc: pa_cache_desc | None = None, alibi_slopes=None, k_scale: float | None = None,
                     v_scale: float | None = None) -> None:
    """A decode step with its append: key/value [num_seqs, num_kv_heads, head_size] are each
    sequence's new token, stored at position seq_lens[s] - 1 of both caches (through the block
    table) and attended in the same call.  fp16/bf16 caches, and FP8 caches (key/value fp16,
    quantised with k_scale / v_scale as pa_reshape_and_cache_fp8 does)."""
    desc = desc or cache_desc(k_cache)
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"), (key, "key"), (value, "value"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens")):
        _dense(t, n)
    num_seqs, num_q_heads = int(q.shape[0]), int(q.shape[1])
    max_blocks = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    need = pa_decode_workspace_size(num_seqs, num_q_heads, max_blocks, desc, partition_size)
    if workspace is None and need > 0:
        import torch
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    opts = None
    if alibi_slopes is not None or k_scale is not None or v_scale is not None:
        _dense(alibi_slopes, "alibi_slopes")
        opts = ctypes.byref(pa_decode_options(_ptr(alibi_slopes), float(k_scale or 0.0), float(v_scale or 0.0), 0))
    _check(lib().pa_decode_append(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(key), _ptr(value),
                                  _ptr(block_tables), _ptr(seq_lens), num_seqs, num_q_heads, max_blocks,
                                  ctypes.byref(desc), float(scale), int(partition_size), _ptr(workspace), ws_bytes,
                                  _ptr(err_flag), _stream(stream), opts), "pa_decode_append")


def pa_prefill(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, max_query_len: int, scale: float,
               err_flag=None, stream=None, desc: pa_cache_desc | None = None) -> None:
    """Chunked prefill: the queries q[query_start[s]:query_start[s+1]] are the last
    n_s of seq_lens[s] cached tokens; query j attends to positions 0..L-n_s+j.

    out, q: [num_query_tokens, num_q_heads, 128] (f16/bf16); block_tables int32
    [num_seqs, max_blocks_per_seq]; seq_lens int32 [num_seqs]; query_start int32
    [num_seqs + 1]; max_query_len bounds every n_s (it sizes the grid).
    """
    desc = desc or cache_desc(k_cache)
    for t, n in ((out, "out"), (q, "q"), (k_cache, "k_cache"), (v_cache, "v_cache"),
                 (block_tables, "block_tables"), (seq_lens, "seq_lens"), (query_start, "query_start")):
        _dense(t, n)
    num_seqs = int(seq_lens.shape[0])
    max_blocks = int(block_tables.shape[1]) if block_tables.dim() == 2 else 0
    status = lib().pa_prefill(_ptr(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens),
                              _ptr(query_start), num_seqs, int(q.shape[0]), int(q.shape[1]), max_blocks,
                              int(max_query_len), ctypes.byref(desc), float(scale), _ptr(err_flag), _stream(stream))
    _check(status, "pa_prefill")


def pa_reshape_and_cache(k_cache, v_cache, key, value, slot_mapping, err_flag=None, stream=None,
                         desc: pa_cache_desc | None = None) -> None:
    """Write key/value [num_tokens, num_kv_heads, head_size] into the slots of slot_mapping (int64)."""
    desc = desc or cache_desc(k_cache)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (key, "key"), (value, "value"),
                 (slot_mapping, "slot_mapping")):
        _dense(t, n)
    status = lib().pa_reshape_and_cache(_ptr(k_cache), _ptr(v_cache), _ptr(key), _ptr(value), _ptr(slot_mapping),
                                        int(slot_mapping.shape[0]), ctypes.byref(desc), _ptr(err_flag),
                                        _stream(stream))
    _check(status, "pa_reshape_and_cache")


def pa_reshape_and_cache_fp8(k_cache, v_cache, key, value, slot_mapping, k_scale: float, v_scale: float,
                             err_flag=None, stream=None, desc: pa_cache_desc | None = None) -> None:
    """Write fp16 key/value [num_tokens, num_kv_heads, head_size] into an FP8 cache as
    E4M3 codes of x / k_scale and x / v_scale (values at [block, head, offset / 16, d, offset % 16])."""
    desc = desc or cache_desc(k_cache)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (key, "key"), (value, "value"),
                 (slot_mapping, "slot_mapping")):
        _dense(t, n)
    status = lib().pa_reshape_and_cache_fp8(_ptr(k_cache), _ptr(v_cache), _ptr(key), _ptr(value), _ptr(slot_mapping),
                                            int(slot_mapping.shape[0]), ctypes.byref(desc), float(k_scale),
                                            float(v_scale), _ptr(err_flag), _stream(stream))
    _check(status, "pa_reshape_and_cache_fp8")


def pa_copy_blocks(k_cache, v_cache, block_pairs, err_flag=None, stream=None, desc: pa_cache_desc | None = None) -> None:
    """For each (src, dst) row of block_pairs (int32 [n, 2]) copy whole block src to dst in both caches."""
    desc = desc or cache_desc(k_cache)
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache"), (block_pairs, "block_pairs")):
        _dense(t, n)
    status = lib().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(block_pairs), int(block_pairs.shape[0]),
                                  ctypes.byref(desc), _ptr(err_flag), _stream(stream))
    _check(status, "pa_copy_blocks")


# ---------------------------------------------------------------- rotary positions and windowed attention
# A step makes one of these calls per layer, and a small one takes the GPU a few microseconds, so the checks are
# written out: each call tests types and devices in one expression, and looks for the reason only when that fails.
_INT32_MIN, _INT32_MAX = -2 ** 31, 2 ** 31 - 1
_ROWS: dict = {}  # cache dtype -> (dtype code, dtype of queries and new rows)


def _int32(x) -> int:
    """x, or the end of int32 on its side (ctypes would wrap it into another number)."""
    return max(_INT32_MIN, min(int(x), _INT32_MAX))


def _rows_of(dtype, where: str):
    """(dtype code, dtype of queries and new rows) of a cache dtype."""
    if not _ROWS:
        import torch
        _ROWS.update({torch.float32: (PA_F32, torch.float32), torch.float16: (PA_F16, torch.float16),
                      torch.bfloat16: (PA_BF16, torch.bfloat16), torch.uint8: (PA_FP8_E4M3, torch.float16),
                      torch.float8_e4m3fn: (PA_FP8_E4M3, torch.float16)})
    if dtype not in _ROWS:
        raise TypeError(f"{where}: unsupported cache dtype {dtype}")
    return _ROWS[dtype]


def _refuse(where: str, dev: int, host: bool, *tensors) -> None:
    """Raises for the first (tensor, name, dtype) that has another dtype or is not on device ``dev`` (``host``: nor in
    pinned host memory)."""
    for t, name, dtype in tensors:
        if t.dtype is not dtype:
            raise TypeError(f"{where}: {name} must be {dtype}, got {t.dtype}")
        if t.get_device() != dev and not (host and t.device.type == "cpu" and t.is_pinned()):
            raise ValueError(f"{where}: {name} is on {t.device}, the caches on cuda:{dev}")


def _caches(k_cache, v_cache, desc, where: str):
    """(device index, descriptor, dtype of queries and new rows) of a cache pair."""
    dev, dtype = k_cache.get_device(), k_cache.dtype
    if dev < 0:
        raise ValueError(f"{where}: the caches must be CUDA tensors")
    if v_cache.dtype is not dtype or v_cache.get_device() != dev or v_cache.numel() != k_cache.numel():
        raise ValueError(f"{where}: k_cache and v_cache must match in type, size and device")
    if not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError(f"{where}: the caches must be contiguous")
    if dtype.itemsize > 1 and v_cache.shape != k_cache.shape:
        raise ValueError(f"{where}: k_cache and v_cache must have the same shape")
    code, rows = _ROWS.get(dtype) or _rows_of(dtype, where)
    if desc is None:
        shape = k_cache.shape
        if len(shape) != 4:
            raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_size]")
        desc = pa_cache_desc(shape[0], shape[2], shape[1], shape[3], code)
    elif (desc.dtype != code or
          desc.num_blocks * desc.block_size * desc.num_kv_heads * desc.head_size != k_cache.numel()):
        raise ValueError(f"{where}: desc does not describe the caches")
    return dev, desc, rows


def _stream_of(dev: int, stream) -> int:
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(dev)
    return int(getattr(stream, "cuda_stream", stream))


def _launch(fn, dev: int, args, where: str) -> None:
    """fn(*args) with the tensors' device current."""
    import torch
    if torch._C._cuda_getDevice() == dev:
        status = fn(*args)
    else:
        with torch.cuda.device(dev):
            status = fn(*args)
    if status != PA_OK:
        raise PaError(status, where)


def pa_rope_frequencies(rotary_dim: int, base: float = 10000.0, method: int = PA_ROPE_PLAIN, factor: float = 1.0,
                        original_max_position: float = 0.0, beta_fast: float = 32.0, beta_slow: float = 1.0,
                        attention_factor: float = 0.0, low_freq_factor: float = 1.0, high_freq_factor: float = 4.0,
                        device=None):
    """(inv_freq, magnitude): the angle per position of each of the rotary_dim / 2 pairs, as a float64 tensor
    (on ``device``), and the factor on the turned elements.  ``method``: PA_ROPE_PLAIN, PA_ROPE_LINEAR,
    PA_ROPE_NTK, PA_ROPE_YARN or PA_ROPE_BANDS, the ways to stretch the frequencies for contexts longer than the
    trained one."""
    import torch
    # (the call writes rotary_dim / 2 numbers, and ctypes would wrap an integer past int32 into another)
    if not 2 <= int(rotary_dim) <= 128 or not PA_ROPE_PLAIN <= int(method) <= PA_ROPE_BANDS:
        raise PaError(3, "pa_rope_frequencies")
    inv = torch.empty(int(rotary_dim) // 2, dtype=torch.float64)
    mag = ctypes.c_float(1.0)
    s = pa_rope_scaling(int(method), factor, original_max_position, beta_fast, beta_slow, attention_factor,
                        low_freq_factor, high_freq_factor)
    _check(lib().pa_rope_frequencies(_ptr(inv), ctypes.addressof(mag), int(rotary_dim), float(base), ctypes.byref(s)),
           "pa_rope_frequencies")
    return (inv if device is None else inv.to(device)), mag.value


def _token_rows(t, name: str, shape, where: str) -> int:
    """Elements between the tokens of [tokens, heads, head_size] = shape, where a token's row is dense."""
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must be {list(shape)}, got {list(t.shape)}")
    tokens, heads, d = shape
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != d and heads > 1):
        raise ValueError(f"{where}: the heads of one token of {name} must be dense")
    return s0 if tokens > 1 else heads * d


def pa_rope_and_cache(q_out, k_cache, v_cache, q, key, value, positions, slot_mapping, inv_freq,
                      interleaved: bool = False, magnitude: float = 1.0, err_flag=None, stream=None,
                      desc: pa_cache_desc | None = None, k_scale: float | None = None,
                      v_scale: float | None = None) -> None:
    """Turn the first 2 * len(inv_freq) elements of each head of q and key by positions * inv_freq, write the queries
    to q_out and the keys and values to their cache slots.

    q, q_out [num_tokens, num_q_heads, head_size] (both None: no queries), key, value [num_tokens, num_kv_heads,
    head_size] of the cache's type (fp16 for an FP8 cache): a token's heads are dense, tokens may lie further apart
    (views of a fused projection).  q_out may be q.  positions int32, slot_mapping int64 [num_tokens] (negative:
    padding, nothing is written); inv_freq float64 on the device, magnitude: see pa_rope_frequencies.
    ``interleaved``: pairs (2j, 2j + 1), else (j, j + rotary_dim / 2)."""
    import torch
    where = "pa_rope_and_cache"
    dev, desc, rows = _caches(k_cache, v_cache, desc, where)
    if not (key.dtype is rows and value.dtype is rows and positions.dtype is torch.int32 and
            slot_mapping.dtype is torch.int64 and inv_freq.dtype is torch.float64 and key.get_device() == dev and
            value.get_device() == dev and positions.get_device() == dev and slot_mapping.get_device() == dev and
            inv_freq.get_device() == dev):
        _refuse(where, dev, True, (key, "key", rows), (value, "value", rows), (positions, "positions", torch.int32),
                (slot_mapping, "slot_mapping", torch.int64), (inv_freq, "inv_freq", torch.float64))
    if not (positions.is_contiguous() and slot_mapping.is_contiguous() and inv_freq.is_contiguous()):
        raise ValueError(f"{where}: positions, slot_mapping and inv_freq must be contiguous")
    tokens, d, hkv = key.shape[0], desc.head_size, desc.num_kv_heads
    if positions.numel() != tokens or slot_mapping.numel() != tokens:
        raise ValueError(f"{where}: positions and slot_mapping must hold {tokens} tokens")
    kv_shape = (tokens, hkv, d)
    ks, vs = _token_rows(key, "key", kv_shape, where), _token_rows(value, "value", kv_shape, where)
    hq = qs = os_ = 0
    qp = op = err = None
    if q is not None and q_out is not None:
        if not (q.dtype is rows and q_out.dtype is rows and q.get_device() == dev and q_out.get_device() == dev):
            _refuse(where, dev, True, (q, "q", rows), (q_out, "q_out", rows))
        hq = q.shape[1]
        q_shape = (tokens, hq, d)
        qs, os_ = _token_rows(q, "q", q_shape, where), _token_rows(q_out, "q_out", q_shape, where)
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q is not q_out:
        raise ValueError(f"{where}: q and q_out go together")
    if err_flag is not None:
        _refuse(where, dev, False, (err_flag, "err_flag", torch.int32))
        err = err_flag.data_ptr()
    _launch(lib().pa_rope_and_cache, dev, (
        op, k_cache.data_ptr(), v_cache.data_ptr(), qp, key.data_ptr(), value.data_ptr(), os_, qs, ks, vs,
        positions.data_ptr(), slot_mapping.data_ptr(), inv_freq.data_ptr(), tokens, hq, 2 * inv_freq.numel(),
        1 if interleaved else 0, float(magnitude), desc, float(k_scale or 0.0), float(v_scale or 0.0), err,
        _stream_of(dev, stream)), where)


def _attention(where, host, out, q, k_cache, v_cache, block_tables, seq_lens, err_flag, desc):
    """The checks of both windowed attention calls: (device, rows' dtype, descriptor, address of err_flag, q's shape,
    the table's shape)."""
    import torch
    dev, desc, rows = _caches(k_cache, v_cache, desc, where)
    if not (out.dtype is rows and q.dtype is rows and block_tables.dtype is torch.int32 and
            seq_lens.dtype is torch.int32 and out.get_device() == dev and q.get_device() == dev and
            block_tables.get_device() == dev and seq_lens.get_device() == dev):
        _refuse(where, dev, host, (out, "out", rows), (q, "q", rows), (block_tables, "block_tables", torch.int32),
                (seq_lens, "seq_lens", torch.int32))
    if not (out.is_contiguous() and q.is_contiguous() and block_tables.is_contiguous() and seq_lens.is_contiguous()):
        raise ValueError(f"{where}: out, q, block_tables and seq_lens must be contiguous")
    err = None
    if err_flag is not None:
        _refuse(where, dev, False, (err_flag, "err_flag", torch.int32))
        err = err_flag.data_ptr()
    shape, table = q.shape, block_tables.shape
    if len(shape) != 3 or shape[2] != desc.head_size or out.shape != shape:
        raise ValueError(f"{where}: q and out must be [queries, heads, {desc.head_size}]")
    if len(table) != 2 or seq_lens.dim() != 1 or seq_lens.shape[0] != table[0]:
        raise ValueError(f"{where}: block_tables must be [num_seqs, max_blocks_per_seq], seq_lens [num_seqs]")
    return dev, rows, desc, err, shape, table


def pa_decode_window(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float, window: int, num_sinks: int = 0,
                     key=None, value=None, err_flag=None, stream=None, desc: pa_cache_desc | None = None,
                     alibi_slopes=None, k_scale: float | None = None, v_scale: float | None = None,
                     test_flags: int = 0) -> None:
    """pa_decode where each sequence's query sees the last ``window`` positions and the first ``num_sinks``.

    Table entries of blocks outside are never read (released blocks).  ``key`` / ``value`` [num_seqs, num_kv_heads,
    head_size]: each sequence's new token, stored at position seq_lens[s] - 1 and attended in the same launch
    (16-bit and FP8 caches).  No workspace."""
    where = "pa_decode_window"
    dev, rows, desc, err, shape, table = _attention(where, True, out, q, k_cache, v_cache, block_tables, seq_lens,
                                                    err_flag, desc)
    if table[0] != shape[0]:
        raise ValueError(f"{where}: one query per sequence")
    kp = vp = opts = None
    if key is not None or value is not None:
        if key is None or value is None:
            raise ValueError(f"{where}: key and value go together")
        if not (key.dtype is rows and value.dtype is rows and key.get_device() == dev and value.get_device() == dev):
            _refuse(where, dev, True, (key, "key", rows), (value, "value", rows))
        new = (shape[0], desc.num_kv_heads, desc.head_size)
        if key.shape != new or value.shape != new or not (key.is_contiguous() and value.is_contiguous()):
            raise ValueError(f"{where}: key and value must be {list(new)}, contiguous")
        kp, vp = key.data_ptr(), value.data_ptr()
    if alibi_slopes is not None or k_scale is not None or v_scale is not None or test_flags:
        slopes = None
        if alibi_slopes is not None:
            import torch
            _refuse(where, dev, True, (alibi_slopes, "alibi_slopes", torch.float32))
            if alibi_slopes.numel() != shape[1] or not alibi_slopes.is_contiguous():
                raise ValueError(f"{where}: one ALiBi slope per query head")
            slopes = alibi_slopes.data_ptr()
        opts = pa_decode_options(slopes, float(k_scale or 0.0), float(v_scale or 0.0), int(test_flags))
    _launch(lib().pa_decode_window, dev, (
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kp, vp, block_tables.data_ptr(),
        seq_lens.data_ptr(), shape[0], shape[1], table[1], desc, float(scale), _int32(window),
        _int32(num_sinks), err, _stream_of(dev, stream), opts), where)


def pa_prefill_window(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, max_query_len: int, scale: float,
                      window: int, num_sinks: int = 0, err_flag=None, stream=None, desc: pa_cache_desc | None = None,
                      k_scale: float | None = None, v_scale: float | None = None) -> None:
    """Attention of a chunk of new tokens with a sliding window: the queries q[query_start[s]:query_start[s + 1]] are
    the last n_s of seq_lens[s] cached tokens; the one at position p sees the last ``window`` positions up to p and
    the first ``num_sinks``.  Every cache type, head size and block size; arguments as for pa_prefill, ``k_scale`` /
    ``v_scale`` the scales of an FP8 cache (q and out are fp16 then)."""
    import torch
    where = "pa_prefill_window"
    dev, rows, desc, err, shape, table = _attention(where, False, out, q, k_cache, v_cache, block_tables, seq_lens,
                                                    err_flag, desc)
    if query_start.dtype is not torch.int32 or query_start.get_device() != dev:
        _refuse(where, dev, False, (query_start, "query_start", torch.int32))
    if query_start.dim() != 1 or query_start.shape[0] != table[0] + 1 or not query_start.is_contiguous():
        raise ValueError(f"{where}: query_start must be [num_seqs + 1]")
    _launch(lib().pa_prefill_window, dev, (
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), query_start.data_ptr(), table[0], shape[0], shape[1], table[1],
        min(_int32(max_query_len), shape[0]), desc,
        float(scale), _int32(window), _int32(num_sinks), float(k_scale or 0.0),
        float(v_scale or 0.0), err, _stream_of(dev, stream)), where)
