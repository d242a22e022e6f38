"""Windowed attention and rotary positions in 64 bits, and the inputs of their tests.

The reference gathers each sequence's visible tokens one by one from their definition (position i is visible to
the query at position p if i <= p and (i > p - window or i < sinks)); it shares nothing with the kernels.
"""
from __future__ import annotations

import numpy as np

import oracle as O
import workloads as W

K_SCALE, V_SCALE = 0.0123, 0.0117  # of the FP8 caches
BAD_ENTRIES = (-1, -7, 2 ** 31 - 1, 10 ** 6)  # what the table holds where no visible token lies


def visible(p: int, window: int, sinks: int) -> np.ndarray:
    i = np.arange(p + 1)
    return i[(i > p - window) | (i < sinks)]


class WindowCase:
    """A pool of shuffled blocks that holds NaN wherever no query sees a token, a block table with entries outside
    the pool for blocks without one, and the queries: the last chunk[s] tokens of lens[s].  dtype 'fp8': E4M3
    caches with fp16 queries."""

    def __init__(self, dtype, lens, chunks, hq, hkv, d, block_size, window, sinks, seed=0, append=False, spread=1.0,
                 slack_blocks=1):
        rng = np.random.default_rng(seed)
        self.dtype, self.lens, self.chunks = dtype, list(lens), list(chunks)
        self.hq, self.hkv, self.d, self.B = hq, hkv, d, block_size
        self.window, self.sinks = window, sinks
        self.qdt = "f16" if dtype == "fp8" else dtype
        self.scale = 1.0 / np.sqrt(d)
        B, n = block_size, len(self.lens)
        self.width = max([-(-L // B) for L in self.lens] + [0]) + slack_blocks
        seen = []  # per sequence: positions some query sees
        for L, c in zip(self.lens, self.chunks):
            ps = [visible(p, window, sinks) for p in range(L - c, L)]
            seen.append(np.unique(np.concatenate(ps)) if ps else np.zeros(0, np.int64))
        self.seen = seen
        blocks = [np.unique(s // B) for s in seen]
        total = sum(len(b) for b in blocks)
        self.num_blocks = total + 3
        ids = rng.permutation(self.num_blocks)
        self.table = np.empty((n, self.width), np.int32)
        self.table[:] = rng.choice(np.array(BAD_ENTRIES, np.int64), size=self.table.shape).astype(np.int32)
        shape = (self.num_blocks, hkv, B, d)
        k, v = np.full(shape, np.nan), np.full(shape, np.nan)
        at = 0
        for s in range(n):
            for b in blocks[s]:
                self.table[s, b] = ids[at]
                at += 1
            for i in seen[s]:
                k[self.table[s, i // B], :, i % B] = rng.standard_normal((hkv, d)) * spread
                v[self.table[s, i // B], :, i % B] = rng.standard_normal((hkv, d))
        self.new_key = self.new_value = None
        if append:  # the last token of each sequence arrives with the call: its slot holds NaN before
            self.new_key = W.to_storage(rng.standard_normal((n, hkv, d)), self.qdt)
            self.new_value = W.to_storage(rng.standard_normal((n, hkv, d)), self.qdt)
        q = rng.standard_normal((sum(self.chunks), hq, d)) * spread
        self.q = W.to_storage(q, self.qdt)
        if dtype == "fp8":
            self.k_cache = self._codes(k, K_SCALE)
            self.v_cache = O.values_to_fp8_layout(self._codes(v, V_SCALE))
        else:
            with np.errstate(invalid="ignore"):
                self.k_cache, self.v_cache = self._store(k), self._store(v)
        if append:
            for s, L in enumerate(self.lens):
                if L:
                    self._poison(s, L - 1)

    def _store(self, x):
        y = W.to_storage(np.nan_to_num(x), self.dtype)
        nan = np.isnan(x)
        if self.dtype == "bf16":
            y[nan] = W.NAN_BITS["bf16"]
        else:
            y[nan] = np.nan
        return y

    def _codes(self, x, scale):
        c = O.quantize_e4m3(np.nan_to_num(x) / scale)
        c = np.asarray(c, np.uint8).reshape(x.shape)
        c[np.isnan(x)] = 0x7F
        return np.ascontiguousarray(c)

    def _poison(self, s, i):
        b, o = self.table[s, i // self.B], i % self.B
        if self.dtype == "fp8":
            self.k_cache[b, :, o] = 0x7F
            self.v_cache[b, :, o // 16, :, o % 16] = 0x7F
        else:
            nan = W.NAN_BITS["bf16"] if self.dtype == "bf16" else np.nan
            self.k_cache[b, :, o] = nan
            self.v_cache[b, :, o] = nan

    # ---- fp64
    def rows(self, cache, s, pos, scale, values):
        b, o = self.table[s, pos // self.B], pos % self.B
        if self.dtype == "fp8":
            x = cache[b, :, o // 16, :, o % 16] if values else cache[b, :, o]
            return CODE_VALUES[x] * scale
        return O.to_f64(np.ascontiguousarray(cache[b, :, o]), self.dtype)

    def reference(self, alibi=None):
        """[queries, heads, D] in 64 bits; an appended token's rows are those that the cache then holds."""
        q = O.to_f64(self.q, self.qdt)
        out = np.zeros(q.shape)
        row, G = 0, self.hq // self.hkv
        for s, (L, c) in enumerate(zip(self.lens, self.chunks)):
            if L == 0:
                row += c
                continue
            seen = self.seen[s]
            k, v = self.rows(self.k_cache, s, seen, K_SCALE, False), self.rows(self.v_cache, s, seen, V_SCALE, True)
            if self.new_key is not None:
                nk, nv = O.to_f64(self.new_key[s], self.qdt), O.to_f64(self.new_value[s], self.qdt)
                if self.dtype == "fp8":
                    nk = CODE_VALUES[self._round(nk, K_SCALE)] * K_SCALE
                    nv = CODE_VALUES[self._round(nv, V_SCALE)] * V_SCALE
                k[-1], v[-1] = nk, nv
            for j in range(c):
                p = L - c + j
                at = np.searchsorted(seen, visible(p, self.window, self.sinks))
                kk, vv = np.repeat(k[at], G, 1), np.repeat(v[at], G, 1)  # [tokens, hq, D]
                sc = np.einsum("hd,thd->ht", q[row], kk) * self.scale
                if alibi is not None:
                    sc = sc + np.asarray(alibi, np.float64)[:, None] * (seen[at] - p)[None]
                w = np.exp(sc - sc.max(1, keepdims=True))
                out[row] = np.einsum("ht,thd->hd", w / w.sum(1, keepdims=True), vv)
                row += 1
        return out

    @staticmethod
    def _round(x, scale):
        r = (x.astype(np.float32) / np.float32(scale)).astype(np.float64)  # the append divides in fp32
        return np.asarray(O.quantize_e4m3(r), np.uint8).reshape(x.shape)

    def query_start(self):
        return np.concatenate([[0], np.cumsum(self.chunks)]).astype(np.int32)


CODE_VALUES = np.array([O.e4m3_to_f64(c) for c in range(256)])
