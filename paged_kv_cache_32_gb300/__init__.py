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

PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3, PA_FP4_E2M1 = 0, 1, 2, 3, 4
PA_OK = 0
PA_DEVERR = {0: "none", 1: "block id out of range", 2: "slot out of range", 3: "copy pair id out of range",
             4: "wait on an asynchronous copy timed out", 5: "prefill chunk inconsistent with q, grid or sequence",
             6: "tables, lengths and wanted tokens do not fit together", 7: "not enough free blocks"}

EXPORTED = ("pa_decode", "pa_decode_ex", "pa_decode_append", "pa_decode_partition_size", "pa_decode_workspace_size",
            "pa_reshape_and_cache", "pa_copy_blocks", "pa_status_string", "pa_version", "pa_decode_noalloc", "pa_prefill",
            "pa_reshape_and_cache_fp8", "pa_rope_frequencies", "pa_rope_and_cache", "pa_decode_window",
            "pa_prefill_window", "pa_reshape_and_cache_fp4", "pa_read_cache_fp4", "pa_decode_fp4",
            "pa_decode_fp4_workspace_size", "pa_prefill_fp4",
            "pa_rope_axes_and_cache", "pa_tables_extend", "pa_tables_trim")


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
        L.pa_reshape_and_cache_fp4.argtypes = [vp, vp, vp, vp, i64, i64, vp, i32, desc_p, i32, f32, f32, vp, vp]
        L.pa_reshape_and_cache_fp4.restype = ctypes.c_int
        L.pa_read_cache_fp4.argtypes = L.pa_reshape_and_cache_fp4.argtypes
        L.pa_read_cache_fp4.restype = ctypes.c_int
        L.pa_decode_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, desc_p, i32, f32, i32, i32, f32, f32, vp,
                                    ctypes.c_uint32, vp, sz, vp, vp]
        L.pa_decode_fp4_workspace_size.argtypes = [i32, i32, i32, desc_p, i32, i32]
        L.pa_decode_fp4_workspace_size.restype = sz
        L.pa_decode_fp4.restype = ctypes.c_int
        L.pa_prefill_fp4.argtypes = [vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, desc_p, i32, f32, i32, i32, f32,
                                     f32, vp, vp]
        L.pa_prefill_fp4.restype = ctypes.c_int
        L.pa_rope_axes_and_cache.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, i32, ctypes.c_char_p, vp, vp,
                                             i32, i32, i32, i32, f32, desc_p, i32, f32, f32, vp, vp]
        L.pa_rope_axes_and_cache.restype = ctypes.c_int
        L.pa_tables_extend.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, vp]
        L.pa_tables_extend.restype = ctypes.c_int
        L.pa_tables_trim.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
        L.pa_tables_trim.restype = ctypes.c_int
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
    [num_blocks, num_kv_heads, block_size / 16, head_size, 16]), or of a 4-bit one (see fp4_cache)."""
    if k_cache.dim() != 4:
        raise ValueError("cache must be [num_blocks, num_kv_heads, block_size, head_size]")
    if k_cache.shape[3] == FP4_TILE_BYTES and k_cache.element_size() == 1:  # (no FP8 cache has such rows)
        return fp4_cache_desc(k_cache)
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


def _workspace(need: int, device, stream):
    """``need`` bytes on ``device`` for a call on ``stream`` (None: torch's current one), taken from that stream's memory:
    they go back when the call returns, and only what runs there afterwards gets them again."""
    import torch
    if stream is not None:
        handle = int(getattr(stream, "cuda_stream", stream))
        if handle != torch._C._cuda_getCurrentRawStream(device.index):
            own = torch.cuda.ExternalStream(handle, device=device) if handle > 1 else \
                torch.cuda.default_stream(device)  # (0, 1: handles of the default stream)
            with torch.cuda.stream(own):
                return torch.empty(need, dtype=torch.uint8, device=device)
    return torch.empty(need, dtype=torch.uint8, device=device)


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
    and one is needed, it is allocated with torch, on the call's stream.  ``alibi_slopes``: optional
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
        workspace = _workspace(need, k_cache.device, stream)
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
        workspace = _workspace(need, k_cache.device, stream)
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
    where = "pa_rope_and_cache"
    dev, desc, rows = _caches(k_cache, v_cache, desc, where)
    tokens, hq, qp, op, qs, os_, ks, vs, err = _rope(where, dev, desc, rows, q_out, q, key, value, positions, slot_mapping,
                                                     inv_freq, 1, err_flag)
    _launch(lib().pa_rope_and_cache, dev, (
        op, k_cache.data_ptr(), v_cache.data_ptr(), qp, key.data_ptr(), value.data_ptr(), os_, qs, ks, vs,
        positions.data_ptr(), slot_mapping.data_ptr(), inv_freq.data_ptr(), tokens, hq, 2 * inv_freq.numel(),
        1 if interleaved else 0, float(magnitude), desc, float(k_scale or 0.0), float(v_scale or 0.0), err,
        _stream_of(dev, stream)), where)


def _rope(where, dev, desc, rows, q_out, q, key, value, positions, slot_mapping, inv_freq, axes, err_flag):
    """The checks of both rotary writes: tokens, query heads, addresses of q and q_out, the four strides, address of
    err_flag."""
    import torch
    if not (key.dtype is rows and value.dtype is rows and positions.dtype is torch.int32 and
            slot_mapping.dtype is torch.int64 and inv_freq.dtype is torch.float64 and key.get_device() == dev and
            value.get_device() == dev and positions.get_device() == dev and slot_mapping.get_device() == dev and
            inv_freq.get_device() == dev):
        _refuse(where, dev, True, (key, "key", rows), (value, "value", rows), (positions, "positions", torch.int32),
                (slot_mapping, "slot_mapping", torch.int64), (inv_freq, "inv_freq", torch.float64))
    if not (positions.is_contiguous() and slot_mapping.is_contiguous() and inv_freq.is_contiguous()):
        raise ValueError(f"{where}: positions, slot_mapping and inv_freq must be contiguous")
    tokens, d, hkv = key.shape[0], desc.head_size, desc.num_kv_heads
    if positions.numel() != axes * tokens or slot_mapping.numel() != tokens:
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
    return tokens, hq, qp, op, qs, os_, ks, vs, err


def pa_rope_axes_and_cache(q_out, k_cache, v_cache, q, key, value, positions, slot_mapping, inv_freq, pair_axis,
                           interleaved: bool = False, magnitude: float = 1.0, err_flag=None, stream=None,
                           desc: pa_cache_desc | None = None, k_scale: float | None = None,
                           v_scale: float | None = None) -> None:
    """pa_rope_and_cache with positions int32 [axes, num_tokens] along 1 to 4 axes: pair j of a head turns by
    positions[pair_axis[j]] * inv_freq[j].  ``pair_axis``: an axis number for each pair (bytes, or any sequence on the
    host; pa_rope_pair_axes makes one).  Over a 4-bit cache (see fp4_cache) the rows are fp16 or bf16, and ``k_scale`` /
    ``v_scale`` its units, which such a call needs."""
    where = "pa_rope_axes_and_cache"
    if k_cache.shape[-1] == FP4_TILE_BYTES:
        dev, desc, code = _caches_fp4(k_cache, v_cache, desc, key.dtype, where)
        rows = key.dtype
        if k_scale is None or v_scale is None:
            raise ValueError(f"{where}: a 4-bit cache needs k_scale and v_scale, its units")
    else:
        dev, desc, rows = _caches(k_cache, v_cache, desc, where)
        code = 0
    if positions.dim() != 2 or not 1 <= positions.shape[0] <= 4:
        raise ValueError(f"{where}: positions must be [axes, num_tokens], 1 to 4 axes")
    axes = positions.shape[0]
    # (bytes() of a number would be that many zeros, and of an array its memory)
    pairs = bytes(pair_axis if isinstance(pair_axis, (bytes, bytearray, list, tuple)) else [int(a) for a in pair_axis])
    if len(pairs) != inv_freq.numel():
        raise ValueError(f"{where}: pair_axis must hold {inv_freq.numel()} axis numbers")
    tokens, hq, qp, op, qs, os_, ks, vs, err = _rope(where, dev, desc, rows, q_out, q, key, value, positions, slot_mapping,
                                                     inv_freq, axes, err_flag)
    _launch(lib().pa_rope_axes_and_cache, dev, (
        op, k_cache.data_ptr(), v_cache.data_ptr(), qp, key.data_ptr(), value.data_ptr(), os_, qs, ks, vs,
        positions.data_ptr(), axes, pairs, slot_mapping.data_ptr(), inv_freq.data_ptr(), tokens, hq, 2 * inv_freq.numel(),
        1 if interleaved else 0, float(magnitude), desc, code, float(k_scale or 0.0), float(v_scale or 0.0), err,
        _stream_of(dev, stream)), where)


def pa_rope_pair_axes(sections, interleaved: bool = False) -> bytes:
    """The axis of each rotary pair: sections[a] pairs for axis a, one section after the other, or dealt out in turn
    (axis 0, 1, 2, 0, 1, ..., an axis whose section is used up left out)."""
    left = [int(n) for n in sections]
    if not interleaved:
        return bytes(a for a, n in enumerate(left) for _ in range(n))
    got = []
    while any(n > 0 for n in left):
        for a in range(len(left)):
            if left[a] > 0:
                got.append(a)
                left[a] -= 1
    return bytes(got)


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


# ---------------------------------------------------------------- caches held in 4 bits
FP4_TILE_BYTES = 1152  # of 16 tokens of a kv head: [16, 64] bytes of codes, [16, 8] of scales
_FP4_ROWS: dict = {}   # dtype of the rows -> code


def fp4_cache(num_blocks: int, num_kv_heads: int, block_size: int, device="cuda"):
    """A zeroed key or value cache held in 4 bits: uint8 [num_blocks, num_kv_heads, block_size / 16, 1152]."""
    import torch
    if block_size <= 0 or block_size % 16:
        raise ValueError("fp4_cache: block_size must be a multiple of 16")
    return torch.zeros((num_blocks, num_kv_heads, block_size // 16, FP4_TILE_BYTES), dtype=torch.uint8, device=device)


def fp4_cache_desc(k_cache) -> pa_cache_desc:
    """Descriptor of a cache made by fp4_cache."""
    if k_cache.dim() != 4 or k_cache.shape[3] != FP4_TILE_BYTES or k_cache.element_size() != 1:
        raise ValueError(f"a 4-bit cache must be uint8 [num_blocks, num_kv_heads, block_size / 16, {FP4_TILE_BYTES}]")
    nb, hkv, tiles, _ = (int(x) for x in k_cache.shape)
    return pa_cache_desc(nb, 16 * tiles, hkv, 128, PA_FP4_E2M1)


def _caches_fp4(k_cache, v_cache, desc, rows, where: str):
    """(device index, descriptor, code of the rows' dtype) of a pair of 4-bit caches."""
    if not _FP4_ROWS:
        import torch
        _FP4_ROWS.update({torch.float16: PA_F16, torch.bfloat16: PA_BF16, torch.uint8: None})
    dev = k_cache.get_device()
    if dev < 0:
        raise ValueError(f"{where}: the caches must be CUDA tensors")
    if k_cache.element_size() != 1 or v_cache.dtype is not k_cache.dtype or v_cache.get_device() != dev or \
            v_cache.shape != k_cache.shape or not (k_cache.is_contiguous() and v_cache.is_contiguous()):
        raise ValueError(f"{where}: k_cache and v_cache must be contiguous uint8 tensors of one shape on one device")
    code = _FP4_ROWS.get(rows)
    if code is None:
        raise TypeError(f"{where}: rows over a 4-bit cache are float16 or bfloat16, got {rows}")
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != FP4_TILE_BYTES:
        raise ValueError(f"{where}: a 4-bit cache must be [num_blocks, num_kv_heads, block_size / 16, {FP4_TILE_BYTES}]")
    if desc is None:
        desc = pa_cache_desc(shape[0], 16 * shape[2], shape[1], 128, PA_FP4_E2M1)
    elif (desc.dtype, desc.num_blocks, desc.num_kv_heads, desc.block_size) != (PA_FP4_E2M1, shape[0], shape[1],
                                                                              16 * shape[2]):
        raise ValueError(f"{where}: desc does not describe the caches")
    return dev, desc, code


def _fp4_rows(name, fn, k_cache, v_cache, key, value, slot_mapping, k_scale, v_scale, err_flag, stream, desc, read):
    import torch
    dev, desc, code = _caches_fp4(k_cache, v_cache, desc, key.dtype, name)
    if not (value.dtype is key.dtype and slot_mapping.dtype is torch.int64 and key.get_device() == dev and
            value.get_device() == dev and slot_mapping.get_device() == dev):
        _refuse(name, dev, True, (key, "key", key.dtype), (value, "value", key.dtype),
                (slot_mapping, "slot_mapping", torch.int64))
    tokens = key.shape[0]
    if slot_mapping.dim() != 1 or slot_mapping.shape[0] != tokens or not slot_mapping.is_contiguous():
        raise ValueError(f"{name}: slot_mapping must be [{tokens}]")
    shape = (tokens, desc.num_kv_heads, 128)
    ks, vs = _token_rows(key, "key", shape, name), _token_rows(value, "value", shape, name)
    err = None
    if err_flag is not None:
        _refuse(name, dev, False, (err_flag, "err_flag", torch.int32))
        err = err_flag.data_ptr()
    caches, rows = (k_cache.data_ptr(), v_cache.data_ptr()), (key.data_ptr(), value.data_ptr())
    _launch(fn, dev, (*(rows + caches if read else caches + rows), ks, vs, slot_mapping.data_ptr(), tokens, desc, code,
                      float(k_scale), float(v_scale), err, _stream_of(dev, stream)), name)


def pa_reshape_and_cache_fp4(k_cache, v_cache, key, value, slot_mapping, k_scale: float, v_scale: float, err_flag=None,
                             stream=None, desc: pa_cache_desc | None = None) -> None:
    """Write key/value [num_tokens, num_kv_heads, 128] (fp16 or bf16; a token's heads dense, tokens may lie further apart)
    into the slots of a 4-bit cache (see fp4_cache): every 16 elements share a scale of 8 bits, k_scale / v_scale are the
    caches' units (2688 units is the largest number that a cache holds)."""
    _fp4_rows("pa_reshape_and_cache_fp4", lib().pa_reshape_and_cache_fp4, k_cache, v_cache, key, value, slot_mapping,
              k_scale, v_scale, err_flag, stream, desc, False)


def pa_read_cache_fp4(key, value, k_cache, v_cache, slot_mapping, k_scale: float, v_scale: float, err_flag=None,
                      stream=None, desc: pa_cache_desc | None = None) -> None:
    """The rows that the slots of a 4-bit cache hold, into key/value [num_tokens, num_kv_heads, 128] (fp16 or bf16)."""
    _fp4_rows("pa_read_cache_fp4", lib().pa_read_cache_fp4, k_cache, v_cache, key, value, slot_mapping, k_scale, v_scale,
              err_flag, stream, desc, True)


def _attention_fp4(where, host, out, q, k_cache, v_cache, block_tables, seq_lens, err_flag, desc):
    """The checks of both attention calls over a 4-bit cache, as _attention."""
    import torch
    rows = q.dtype
    dev, desc, code = _caches_fp4(k_cache, v_cache, desc, rows, where)
    if not (out.dtype is rows and block_tables.dtype is torch.int32 and seq_lens.dtype is torch.int32 and
            out.get_device() == dev and q.get_device() == dev and block_tables.get_device() == dev and
            seq_lens.get_device() == dev):
        _refuse(where, dev, host, (out, "out", rows), (q, "q", rows), (block_tables, "block_tables", torch.int32),
                (seq_lens, "seq_lens", torch.int32))
    if not (out.is_contiguous() and q.is_contiguous() and block_tables.is_contiguous() and seq_lens.is_contiguous()):
        raise ValueError(f"{where}: out, q, block_tables and seq_lens must be contiguous")
    err = None
    if err_flag is not None:
        _refuse(where, dev, False, (err_flag, "err_flag", torch.int32))
        err = err_flag.data_ptr()
    shape, table = q.shape, block_tables.shape
    if len(shape) != 3 or shape[2] != 128 or out.shape != shape:
        raise ValueError(f"{where}: q and out must be [queries, heads, 128]")
    if len(table) != 2 or seq_lens.dim() != 1 or seq_lens.shape[0] != table[0]:
        raise ValueError(f"{where}: block_tables must be [num_seqs, max_blocks_per_seq], seq_lens [num_seqs]")
    return dev, code, desc, err, shape, table


_FP4_WORKSPACE: dict = {}  # sizes of a call -> bytes


def pa_decode_fp4_workspace_size(num_seqs: int, num_q_heads: int, max_blocks_per_seq: int, desc: pa_cache_desc,
                                 window: int | None = None, num_sinks: int = 0) -> int:
    """Bytes of the workspace that pa_decode_fp4 uses for these sizes (0: none)."""
    return int(lib().pa_decode_fp4_workspace_size(_int32(num_seqs), _int32(num_q_heads), _int32(max_blocks_per_seq), desc,
                                                  _INT32_MAX if window is None else _int32(window), _int32(num_sinks)))


def pa_decode_fp4(out, q, k_cache, v_cache, block_tables, seq_lens, scale: float, k_scale: float, v_scale: float,
                  window: int | None = None, num_sinks: int = 0, key=None, value=None, err_flag=None, stream=None,
                  desc: pa_cache_desc | None = None, alibi_slopes=None, workspace=None, test_flags: int = 0) -> None:
    """A decode step over a 4-bit cache (see fp4_cache): out[s, h] = softmax(scale * q[s, h] K_s^T) V_s over the last
    ``window`` (None: all) and the first ``num_sinks`` positions.  out, q [num_seqs, num_q_heads, 128] fp16 or bf16;
    ``key`` / ``value`` [num_seqs, num_kv_heads, 128]: each sequence's new token, stored at position seq_lens[s] - 1 as
    pa_reshape_and_cache_fp4 does and attended in the same call.  ``workspace``: a uint8 device tensor of
    pa_decode_fp4_workspace_size(...) bytes, allocated with torch on the call's stream when None; calls that may overlap
    need one each."""
    where = "pa_decode_fp4"
    dev, code, desc, err, shape, table = _attention_fp4(where, True, out, q, k_cache, v_cache, block_tables, seq_lens,
                                                        err_flag, desc)
    if table[0] != shape[0]:
        raise ValueError(f"{where}: one query per sequence")
    kp = vp = slopes = None
    if key is not None or value is not None:
        if key is None or value is None:
            raise ValueError(f"{where}: key and value go together")
        if not (key.dtype is q.dtype and value.dtype is q.dtype and key.get_device() == dev and value.get_device() == dev):
            _refuse(where, dev, True, (key, "key", q.dtype), (value, "value", q.dtype))
        new = (shape[0], desc.num_kv_heads, 128)
        if key.shape != new or value.shape != new or not (key.is_contiguous() and value.is_contiguous()):
            raise ValueError(f"{where}: key and value must be {list(new)}, contiguous")
        kp, vp = key.data_ptr(), value.data_ptr()
    if alibi_slopes is not None:
        import torch
        _refuse(where, dev, True, (alibi_slopes, "alibi_slopes", torch.float32))
        if alibi_slopes.numel() != shape[1] or not alibi_slopes.is_contiguous():
            raise ValueError(f"{where}: one ALiBi slope per query head")
        slopes = alibi_slopes.data_ptr()
    ws = None
    ws_bytes = 0
    if workspace is None and slopes is None:  # (with ALiBi no call uses one)
        sizes = (shape[0], shape[1], table[1], desc.num_kv_heads, desc.block_size, window, num_sinks)
        need = _FP4_WORKSPACE.get(sizes)
        if need is None:
            if len(_FP4_WORKSPACE) > 4096:
                _FP4_WORKSPACE.clear()
            need = _FP4_WORKSPACE[sizes] = pa_decode_fp4_workspace_size(shape[0], shape[1], table[1], desc, window, num_sinks)
        if need:
            workspace = _workspace(need, k_cache.device, stream)
    elif workspace is not None and (workspace.get_device() != dev or not workspace.is_contiguous()):
        raise ValueError(f"{where}: workspace must be contiguous, on cuda:{dev}")
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    _launch(lib().pa_decode_fp4, dev, (
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), kp, vp, block_tables.data_ptr(),
        seq_lens.data_ptr(), shape[0], shape[1], table[1], desc, code, float(scale),
        _INT32_MAX if window is None else _int32(window), _int32(num_sinks), float(k_scale), float(v_scale), slopes,
        int(test_flags), ws, ws_bytes, err, _stream_of(dev, stream)), where)


def pa_prefill_fp4(out, q, k_cache, v_cache, block_tables, seq_lens, query_start, max_query_len: int, scale: float,
                   k_scale: float, v_scale: float, window: int | None = None, num_sinks: int = 0, err_flag=None, stream=None,
                   desc: pa_cache_desc | None = None) -> None:
    """Attention of a chunk of new tokens over a 4-bit cache that already holds them: the queries
    q[query_start[s]:query_start[s + 1]] are the last n_s of seq_lens[s] tokens; the one at position p sees the positions
    up to p, or the last ``window`` of them and the first ``num_sinks``.  Other arguments as for pa_decode_fp4 and
    pa_prefill_window."""
    import torch
    where = "pa_prefill_fp4"
    dev, code, desc, err, shape, table = _attention_fp4(where, False, out, q, k_cache, v_cache, block_tables, seq_lens,
                                                        err_flag, desc)
    if query_start.dtype is not torch.int32 or query_start.get_device() != dev:
        _refuse(where, dev, False, (query_start, "query_start", torch.int32))
    if query_start.dim() != 1 or query_start.shape[0] != table[0] + 1 or not query_start.is_contiguous():
        raise ValueError(f"{where}: query_start must be [num_seqs + 1]")
    _launch(lib().pa_prefill_fp4, dev, (
        out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
        seq_lens.data_ptr(), query_start.data_ptr(), table[0], shape[0], shape[1], table[1],
        min(_int32(max_query_len), shape[0]), desc, code, float(scale), _INT32_MAX if window is None else _int32(window),
        _int32(num_sinks), float(k_scale), float(v_scale), err, _stream_of(dev, stream)), where)


# ---------------------------------------------------------------- block tables on the GPU
def _tables(where, block_tables, seq_lens, held_blocks, free_blocks, num_free, wanted, err_flag):
    """The checks of both calls: (device, address of err_flag, num_seqs, max_blocks_per_seq)."""
    import torch
    dev, i32 = block_tables.get_device(), torch.int32
    if not (dev >= 0 and block_tables.dtype is i32 and seq_lens.dtype is i32 and held_blocks.dtype is i32 and
            free_blocks.dtype is i32 and num_free.dtype is i32 and wanted.dtype is i32 and seq_lens.get_device() == dev and
            held_blocks.get_device() == dev and free_blocks.get_device() == dev and num_free.get_device() == dev and
            wanted.get_device() == dev and block_tables.is_contiguous() and seq_lens.is_contiguous() and
            held_blocks.is_contiguous() and free_blocks.is_contiguous() and wanted.is_contiguous()):
        if dev < 0:
            raise ValueError(f"{where}: the tables must be CUDA tensors")
        for t, name in ((block_tables, "block_tables"), (seq_lens, "seq_lens"), (held_blocks, "held_blocks"),
                        (free_blocks, "free_blocks"), (num_free, "num_free"), (wanted, "new_tokens / keep_lens")):
            _refuse(where, dev, False, (t, name, i32))
            if not t.is_contiguous():
                raise ValueError(f"{where}: {name} must be contiguous")
    if block_tables.dim() != 2 or num_free.numel() != 1:
        raise ValueError(f"{where}: block_tables must be [num_seqs, max_blocks_per_seq], num_free one number")
    n, width = block_tables.shape
    if seq_lens.numel() != n or held_blocks.numel() != n or wanted.numel() != n:
        raise ValueError(f"{where}: seq_lens, held_blocks and the tokens wanted must hold {n} requests")
    err = None
    if err_flag is not None:
        _refuse(where, dev, False, (err_flag, "err_flag", i32))
        err = err_flag.data_ptr()
    return dev, err, n, width


def pa_tables_extend(block_tables, seq_lens, held_blocks, free_blocks, num_free, new_tokens, slot_mapping, positions,
                     query_start, block_size: int, err_flag=None, stream=None) -> None:
    """Give request s new_tokens[s] more tokens: fresh blocks from the stack free_blocks[:num_free] into its row of
    block_tables, seq_lens, held_blocks and num_free moved on, and for every new token its slot (int64), its position,
    and where its request's rows start (query_start [num_seqs + 1]).  Rows past the last new token get slot -1.
    All state is int32 on the GPU and changed in place; if the requests do not fit, nothing changes and err_flag says why
    (6 or 7, see PA_DEVERR)."""
    import torch
    where = "pa_tables_extend"
    dev, err, n, width = _tables(where, block_tables, seq_lens, held_blocks, free_blocks, num_free, new_tokens, err_flag)
    rows = slot_mapping.numel()
    if not (slot_mapping.dtype is torch.int64 and positions.dtype is torch.int32 and query_start.dtype is torch.int32 and
            slot_mapping.get_device() == dev and positions.get_device() == dev and query_start.get_device() == dev):
        _refuse(where, dev, False, (slot_mapping, "slot_mapping", torch.int64), (positions, "positions", torch.int32),
                (query_start, "query_start", torch.int32))
    if positions.numel() != rows or query_start.numel() != n + 1 or \
            not (slot_mapping.is_contiguous() and positions.is_contiguous() and query_start.is_contiguous()):
        raise ValueError(f"{where}: slot_mapping and positions must have the same rows, query_start {n + 1}, contiguous")
    _launch(lib().pa_tables_extend, dev, (
        block_tables.data_ptr(), seq_lens.data_ptr(), held_blocks.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr(),
        new_tokens.data_ptr(), slot_mapping.data_ptr(), positions.data_ptr(), query_start.data_ptr(), n, rows, width,
        _int32(block_size), free_blocks.numel(), err, _stream_of(dev, stream)), where)


def pa_tables_trim(block_tables, seq_lens, held_blocks, free_blocks, num_free, keep_lens, block_size: int, err_flag=None,
                   stream=None) -> None:
    """Keep the first keep_lens[s] tokens of request s (drafts rejected; 0: the request is done): the blocks past them go
    back on the stack.  State and errors as for pa_tables_extend."""
    where = "pa_tables_trim"
    dev, err, n, width = _tables(where, block_tables, seq_lens, held_blocks, free_blocks, num_free, keep_lens, err_flag)
    _launch(lib().pa_tables_trim, dev, (
        block_tables.data_ptr(), seq_lens.data_ptr(), held_blocks.data_ptr(), free_blocks.data_ptr(), num_free.data_ptr(),
        keep_lens.data_ptr(), n, width, _int32(block_size), free_blocks.numel(), err, _stream_of(dev, stream)), where)
