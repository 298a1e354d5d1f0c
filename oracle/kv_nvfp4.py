"""The paged key-value cache held in NVFP4, in NumPy and in 64 bits -- TEST INFRASTRUCTURE ONLY, as oracle/kv_cache.py, whose
attention and eviction it uses on decoded rows.

Tolerances: attention as oracle/kv_cache.py derives them for a cache whose products are in f16 (a code times its block's scale is
exact there); appended codes and block scales bit for bit (IEEE products and divisions in fp32, and one rounding).
"""
from __future__ import annotations

import numpy as np

import workloads as wl
from oracle import kv_cache as base

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])


def e2m1_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E2M1 codes, ties to the even code, saturating at 6; the sign stays on a zero."""
    a, mags = np.abs(x), E2M1[:8]
    hi = np.clip(np.searchsorted(mags, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - mags[lo], mags[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 6, 7, code)
    return (code | np.where(np.signbit(x), 8, 0)).astype(np.uint8)


def encode(x: np.ndarray, s: float):
    """Rows [..., d] -> (codes [..., d / 2], block scales [..., d / 16]). A block with a NaN: the scale NaN, zero codes."""
    y, s = x.astype(np.float32).reshape(x.shape[:-1] + (-1, 16)), np.float32(s)
    amax = np.abs(y).max(-1)
    sf = np.where(np.isnan(amax), np.uint8(0x7F), base.e4m3_codes(amax / (np.float32(6) * s)))
    scale = (base.E4M3[sf].astype(np.float32) * s)[..., None]
    q = np.where(scale > 0, e2m1_codes(y / np.where(scale > 0, scale, np.float32(1))), 0).astype(np.uint8).reshape(x.shape)
    return q[..., 0::2] | (q[..., 1::2] << 4), sf


def decode(codes: np.ndarray, sf: np.ndarray, s: float) -> np.ndarray:
    q = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1, 16))
    return (E2M1[q] * base.E4M3[sf][..., None] * s).reshape(codes.shape[:-1] + (-1,))


class Cache(base.Cache):
    """As oracle/kv_cache.py's: a page holds the codes of its heads and slots and behind them the scales of their blocks."""

    def __init__(self, rng, lens, hkv, d, page, spare=2, width=0, gap=0, meta=True, fill=True, scales=(2.0 ** -9, 3 * 2.0 ** -11)):
        super().__init__(rng, lens, hkv, d, page, "fp8", "static", spare, width, 0, meta, False)
        self.fmt, self.mode, self.gap = "nvfp4", "static", gap
        self.stride = (hkv * page * d // 16 * 9 + 15) // 16 * 16 + gap
        self.k_raw, self.v_raw = (np.full(self.n_pages * self.stride, 0x7F, np.uint8) for _ in range(2))
        self.ks, self.vs = (np.array([s], np.float32) for s in scales)
        if fill:
            for b, length in enumerate(self.lens):
                if length:
                    rows = rng.standard_normal((2, length, hkv, d)).astype(np.float32)
                    self.store(b, np.arange(length), wl.f32_to_bf16_bits(rows[0]), wl.f32_to_bf16_bits(rows[1]))
                    if meta:
                        p, h, s = self.at(b, np.arange(length))
                        self.weight[p, :, s] = rng.random((length, hkv)).astype(np.float32) ** 4

    def _part(self, raw, offset, row):
        return np.lib.stride_tricks.as_strided(raw[offset:], (self.n_pages, self.hkv, self.page, row),
                                               (self.stride, self.page * row, row, 1))

    def view(self, raw):
        return self._part(raw, 0, self.d // 2)

    def blocks(self, raw):
        return self._part(raw, self.hkv * self.page * self.d // 2, self.d // 16)

    def store(self, b, slots, k_bits, v_bits, positions=None):
        p, _, s = self.at(b, slots)
        for raw, scale, bits in ((self.k_raw, self.ks, k_bits), (self.v_raw, self.vs, v_bits)):
            self.view(raw)[p, :, s], self.blocks(raw)[p, :, s] = encode(wl.bf16_bits_to_f32(bits), float(scale[0]))
        if self.weight is not None:
            self.weight[p, :, s] = 0
            self.position[p, :, s] = (np.asarray(slots) if positions is None else np.asarray(positions))[:, None]

    def rows(self, b, slots):
        p, _, s = self.at(b, slots)
        return [np.swapaxes(decode(self.view(raw)[p, :, s], self.blocks(raw)[p, :, s], float(scale[0])), 0, 1)
                for raw, scale in ((self.k_raw, self.ks), (self.v_raw, self.vs))]

    def evict(self, budget, recent):
        """The base's eviction moves a scale for each row: here the scales of its blocks."""
        kept = self.fmt, self.mode, self.ks, self.vs
        self.fmt, self.mode, self.ks, self.vs = "fp8", "dynamic", self.blocks(self.k_raw), self.blocks(self.v_raw)
        try:
            return super().evict(budget, recent)
        finally:
            self.fmt, self.mode, self.ks, self.vs = kept
