"""Caches held in 4 bits in numpy, from their definition, and the inputs of their attention tests.

A group is 16 neighbouring elements x: s = e4m3(max |x| / (6 u)), codes e2m1(x * (1 / (s u))), each step one fp32
operation, ties to even; a code stands for e2m1 * s * u.
"""
from __future__ import annotations

import numpy as np

import oracle as O
import workloads as W
from window_ref import CODE_VALUES, WindowCase, visible

K_UNIT, V_UNIT = 0.0025, 0.0031
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
TILE, CODES = 1152, 1024
NAN_SCALE = 0x7F


def quantise(x, unit):
    """Code bytes [..., 64] and scale bytes [..., 8] of rows x [..., 128]."""
    x = np.asarray(x, np.float32).reshape(*np.shape(x)[:-1], 8, 16)
    unit = np.float32(unit)
    with np.errstate(all="ignore"):
        amax = np.fmax.reduce(np.abs(x), axis=-1)
        s = np.asarray(O.quantize_e4m3(np.minimum(amax / (np.float32(6) * unit), np.float32(448)).astype(np.float64)),
                       np.uint8).reshape(amax.shape)
        t = CODE_VALUES[s].astype(np.float32) * unit
        inv = np.where(t > 0, np.float32(1) / t, np.float32(0)).astype(np.float32)
        y = x * inv[..., None]
    a = np.abs(y)
    code = np.zeros(a.shape, np.uint8)
    for at, tie_up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (a >= at) if tie_up else (a > at)
    code[np.isnan(y)] = 7
    code |= np.signbit(y).astype(np.uint8) << 3
    code = code.reshape(*code.shape[:-2], 128)
    return code[..., 0::2] | code[..., 1::2] << 4, s


def pack(codes, scales):
    """Rows [blocks, heads, B, ...] as a cache [blocks, heads, B / 16, 1152]."""
    nb, h, B, _ = codes.shape
    return np.ascontiguousarray(np.concatenate([codes.reshape(nb, h, B // 16, CODES), scales.reshape(nb, h, B // 16, 128)], -1))


def unpack(cache):
    nb, h, t, _ = cache.shape
    return cache[..., :CODES].reshape(nb, h, 16 * t, 64), cache[..., CODES:].reshape(nb, h, 16 * t, 8)


def values(codes, scales, unit):
    x = np.stack([E2M1[codes & 15], E2M1[codes >> 4]], -1).reshape(*codes.shape[:-1], 8, 16)
    return (x * CODE_VALUES[scales][..., None]).reshape(*codes.shape[:-1], 128) * np.float64(np.float32(unit))


class Fp4Case(WindowCase):
    """WindowCase over caches held in 4 bits; rows: 'f16' or 'bf16'.  Where no query sees a token its scales are NaN."""

    def __init__(self, rows, lens, chunks, hq, hkv, block_size, window, sinks, **kw):
        self._unit = [K_UNIT, V_UNIT]
        super().__init__(rows, lens, chunks, hq, hkv, 128, block_size, window, sinks, **kw)

    def _store(self, x):
        codes, scales = quantise(np.nan_to_num(x), self._unit.pop(0))
        unseen = np.isnan(x).any(-1)
        codes[unseen], scales[unseen] = 0xB7, NAN_SCALE
        return pack(codes, scales)

    def _poison(self, s, i):
        b, o = self.table[s, i // self.B], i % self.B
        for cache in (self.k_cache, self.v_cache):
            cache[b, :, o // 16, CODES + 8 * (o % 16):CODES + 8 * (o % 16) + 8] = NAN_SCALE

    def held(self, cache, s, pos, unit):
        codes, scales = unpack(cache)
        b, o = self.table[s, pos // self.B], pos % self.B
        return values(codes[b, :, o], scales[b, :, o], unit)

    def reference(self, alibi=None):
        q = O.to_f64(self.q, self.qdt)
        out = np.zeros(q.shape)
        row, G = 0, self.hq // self.hkv
        for s, (L, c) in enumerate(zip(self.lens, self.chunks)):
            seen = self.seen[s]
            if L == 0:
                row += c
                continue
            k, v = self.held(self.k_cache, s, seen, K_UNIT), self.held(self.v_cache, s, seen, V_UNIT)
            if self.new_key is not None:
                k[-1] = values(*quantise(O.to_f64(self.new_key[s], self.qdt), K_UNIT), K_UNIT)
                v[-1] = values(*quantise(O.to_f64(self.new_value[s], self.qdt), V_UNIT), V_UNIT)
            for j in range(c):
                p = L - c + j
                at = np.searchsorted(seen, visible(p, self.window, self.sinks))
                kk, vv = k[at].transpose(1, 0, 2), v[at].transpose(1, 0, 2)  # [hkv, tokens, D]
                sc = (q[row].reshape(self.hkv, G, 128) @ kk.transpose(0, 2, 1) * self.scale).reshape(self.hq, -1)
                if alibi is not None:
                    sc = sc + np.asarray(alibi, np.float64)[:, None] * (seen[at] - p)[None]
                w = np.exp(sc - sc.max(1, keepdims=True))
                w /= w.sum(1, keepdims=True)
                out[row] = (w.reshape(self.hkv, G, -1) @ vv).reshape(self.hq, 128)
                row += 1
        return out


def rows_storage(x, dtype):
    return W.to_storage(x, dtype)
