"""The paged key-value cache in NumPy, from the definitions and in 64 bits -- TEST INFRASTRUCTURE ONLY, as the C oracle: what
the tests and the smoke check compare with. Also the caches they run on, with every byte that no call may read (or write)
poisoned. It shares no code with the CUDA library.

Tolerances, derived before the kernels ran:
  * appended rows, scales, positions, evicted caches, lengths: bit for bit (values are copied, or come from IEEE
    divisions and one rounding to E4M3);
  * logits: each is a sum of D products of short mantissas, exact in fp32, whose D - 1 additions round or truncate to
    24 bits: off by at most dx = (D 2^-23 + 2^-22) scale sum_i |q_i k_ij| (the second term: the scale's rounding, the
    change to units of log2 and, in FP8, the code's scale), the largest over the slots in view;
  * lse: dx, and the sum's own rounding: L additions of positive terms in at least 32 partial sums, with an exp2 of
    2^-22 each: (L / 32 + 8) 2^-23, plus 2^-22 |lse| for the logarithm and its change of base;
  * probabilities: relative 2 dx + (L / 32 + 8) 2^-23 =: dp; weights: dp times what was added, plus one rounding of the
    new weight, 2^-23 of it;
  * out: half a step of bf16, 2^-8 relative, plus the products' errors, relative to A = sum_j p_j |v_j|: dp, and the
    rounding of the probabilities before the product: two bf16 terms, (2^-8)^2, for a bf16 cache, one f16 term, 2^-11,
    for an FP8 cache; their sums as for the logits, D replaced by L / 32 + 64 additions of 2^-23.
"""
from __future__ import annotations

import numpy as np

import workloads as wl

LOG2E = 1.4426950408889634


def _e4m3_table():
    c = np.arange(256)
    s, e, m = np.where(c & 0x80, -1.0, 1.0), (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e.astype(np.float64) - 10))
    v[(c & 0x7F) == 0x7F] = np.nan
    return s * v


E4M3 = _e4m3_table()
_MAGNITUDES = E4M3[:127]


def e4m3_codes(x: np.ndarray) -> np.ndarray:
    """Nearest E4M3 codes of finite values, ties to even, saturating at 448; the sign stays on a zero."""
    a = np.abs(x).astype(np.float64)
    hi = np.clip(np.searchsorted(_MAGNITUDES, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _MAGNITUDES[lo], _MAGNITUDES[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a >= 448, 126, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def quantise(x32: np.ndarray, mode: str, scale=None):
    """Codes and scales [..., D] -> ([..., D] uint8, [...] float32): value / scale in fp32, then to E4M3."""
    if mode == "dynamic":
        scale = (np.abs(x32).max(-1) / np.float32(448)).astype(np.float32)
        safe = np.where(scale == 0, np.float32(1), scale)[..., None]
        codes = e4m3_codes((x32 / safe).astype(np.float32))
        return np.where(scale[..., None] == 0, 0, codes).astype(np.uint8), scale
    return e4m3_codes((x32 / np.float32(scale)).astype(np.float32)), np.float32(scale)


class Cache:
    """A paged cache on the host (bit patterns) and, once device() was called, its copy on the GPU between guard
    bands. Slots without a token hold NaN patterns, weights NaN, positions INT_MIN; the table's entries behind a
    sequence's pages name no page."""

    def __init__(self, rng, lens, hkv, d, page, fmt, mode="static", spare=2, width=0, gap=0, meta=True, fill=True):
        self.lens = np.asarray(lens, np.int32)
        n = len(lens)
        self.hkv, self.d, self.page, self.fmt, self.mode = hkv, d, page, fmt, mode
        used = [-(-int(x) // page) for x in lens]
        self.width = max(1, max(used, default=1), width)
        self.n_pages = sum(used) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.where(rng.random((n, self.width)) < 0.5, -1, 1 << 30).astype(np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.gap = gap                                    # elements between pages
        dense = hkv * page * d
        self.stride = dense + gap
        dt, poison = (np.uint16, 0x7FC1) if fmt == "bf16" else (np.uint8, 0x7F)
        self.k_raw, self.v_raw = (np.full(self.n_pages * self.stride, poison, dt) for _ in range(2))
        shape = (self.n_pages, hkv, page)
        self.ks = self.vs = None
        if fmt == "fp8":
            if mode == "static":
                self.ks, self.vs = np.array([0.03125], np.float32), np.array([0.0234375], np.float32)
            else:
                self.ks, self.vs = (np.full(shape, np.nan, np.float32) for _ in range(2))
        self.weight = np.full(shape, np.nan, np.float32) if meta else None
        self.position = np.full(shape, -(1 << 31), np.int32) if meta else None
        if fill:
            for b, length in enumerate(self.lens):
                if length:
                    rows = rng.standard_normal((2, length, hkv, d)).astype(np.float32)
                    self.store(b, np.arange(length), wl.f32_to_bf16_bits(rows[0]), wl.f32_to_bf16_bits(rows[1]))
                    if meta:
                        w = rng.random((length, hkv)).astype(np.float32) ** 4
                        p, h, s = self.at(b, np.arange(length))
                        self.weight[p, :, s] = w

    def view(self, raw):
        return np.lib.stride_tricks.as_strided(
            raw, (self.n_pages, self.hkv, self.page, self.d),
            tuple(x * raw.itemsize for x in (self.stride, self.page * self.d, self.d, 1)))

    def at(self, b, slots):
        slots = np.asarray(slots, np.int64)
        return self.table[b, slots // self.page].astype(np.int64), None, slots % self.page

    def store(self, b, slots, k_bits, v_bits, positions=None):
        """Rows [n, hkv, d] of bf16 bits into slots, as the append defines it."""
        p, _, s = self.at(b, slots)
        for raw, scales, bits in ((self.k_raw, self.ks, k_bits), (self.v_raw, self.vs, v_bits)):
            if self.fmt == "bf16":
                self.view(raw)[p, :, s] = bits
                continue
            codes, sc = quantise(wl.bf16_bits_to_f32(bits), self.mode, None if self.mode == "dynamic" else scales[0])
            self.view(raw)[p, :, s] = codes
            if self.mode == "dynamic":
                scales[p, :, s] = sc
        if self.weight is not None:
            self.weight[p, :, s] = 0
            self.position[p, :, s] = (np.asarray(slots) if positions is None else np.asarray(positions))[:, None]

    def rows(self, b, slots):
        """k and v of slots in 64 bits, [2][hkv, n, d]."""
        p, _, s = self.at(b, slots)
        out = []
        for raw, scales in ((self.k_raw, self.ks), (self.v_raw, self.vs)):
            x = self.view(raw)[p, :, s]
            x = wl.bf16_bits_to_f32(x).astype(np.float64) if self.fmt == "bf16" else E4M3[x]
            if self.fmt == "fp8":
                x = x * (float(scales[0]) if self.mode == "static" else scales[p, :, s].astype(np.float64)[..., None])
            out.append(np.swapaxes(x, 0, 1))
        return out

    # -------------------------------------------------------------------------------------------- operators

    def attend(self, q_bits, hq, scale, window=0, accumulate=False):
        """(out, lse, tolerances of both, weight increments and their tolerance) in 64 bits."""
        n, d, g = len(self.lens), self.d, hq // self.hkv
        out, lse = np.zeros((n, hq, d)), np.full((n, hq), -np.inf)
        t_out, t_lse = np.zeros_like(out), np.zeros_like(lse)
        if accumulate:
            t_w = np.zeros(self.weight.shape)
            new_w = self.weight.astype(np.float64)
        q = wl.bf16_bits_to_f32(q_bits).astype(np.float64).reshape(n, self.hkv, g, d)
        for b, length in enumerate(self.lens):
            first = max(0, int(length) - window) if window else 0
            if length <= first:
                continue
            slots = np.arange(first, length)
            k, v = self.rows(b, slots)
            x = np.einsum("hgd,hld->hgl", q[b], k) * scale
            size = np.einsum("hgd,hld->hgl", np.abs(q[b]), np.abs(k)) * abs(scale)
            dx = (d * 2.0 ** -23 + 2.0 ** -22) * size.max(-1)
            m = x.max(-1, keepdims=True)
            e = np.exp(x - m)
            total = e.sum(-1, keepdims=True)
            p = e / total
            L = len(slots)
            out[b] = np.einsum("hgl,hld->hgd", p, v).reshape(hq, d)
            lse[b] = (m + np.log(total)).reshape(hq)
            dsum = (L / 32 + 8) * 2.0 ** -23
            dp = 2 * dx + dsum
            rounding = 2.0 ** -16 if self.fmt == "bf16" else 2.0 ** -11
            a = np.einsum("hgl,hld->hgd", p, np.abs(v))
            t_out[b] = (a * (dp + rounding + (L / 32 + 64) * 2.0 ** -23)[..., None]).reshape(hq, d) \
                + 2.0 ** -8 * np.abs(out[b])
            t_lse[b] = (dx + dsum).reshape(hq) + 2.0 ** -22 * np.abs(lse[b])
            if accumulate:
                pg, _, s = self.at(b, slots)
                new_w[pg, :, s] += p.sum(1).T
                t_w[pg, :, s] = (p * dp[..., None]).sum(1).T
        if accumulate:
            t_w += 2.0 ** -23 * np.abs(np.nan_to_num(new_w))
            return out, lse, t_out, t_lse, new_w, t_w
        return out, lse, t_out, t_lse

    def evict(self, budget, recent):
        """The eviction, in place; returns the new lengths. One head at a time, one move at a time."""
        pools = [self.view(self.k_raw), self.view(self.v_raw), self.weight, self.position]
        if self.fmt == "fp8" and self.mode == "dynamic":
            pools += [self.ks, self.vs]
        for b, length in enumerate(self.lens):
            if length <= budget:
                continue
            p, _, s = self.at(b, np.arange(length))
            bad = (p < 0) | (p >= self.n_pages)               # no page of the pool: no row, and no room for one
            p = np.where(bad, 0, p)
            stuck = bad & (np.arange(length) < budget)
            for h in range(self.hkv):
                w, pos = self.weight[p, h, s], self.position[p, h, s].astype(np.int64)
                w[bad], pos[bad] = np.nan, -(1 << 40)
                safe = pos > pos.max() - recent if recent > 0 else np.zeros(length, bool)
                safe |= stuck
                worst = np.isnan(w)
                w = np.where(np.isnan(w), -np.inf, w) + 0.0
                order = np.lexsort((np.arange(length), -w, worst & ~safe, ~safe)) if not safe.any() else \
                    np.lexsort((np.arange(length), np.where(safe, 0, -w), worst & ~safe, ~safe))
                kept = np.zeros(length, bool)
                kept[order[:budget]] = True
                holes = np.flatnonzero(~kept[:budget])
                movers = budget + np.flatnonzero(kept[budget:])
                for to, src in zip(holes, movers):
                    for x in pools:
                        x[p[to], h, s[to]] = x[p[src], h, s[src]]
        return np.minimum(self.lens, budget).astype(np.int32)


def check_close(got, want, tol, what):
    """|got - want| <= tol, and equal where want is infinite."""
    got = np.asarray(got, np.float64)
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    bad = ~(np.abs(np.where(inf, 0, got - np.where(inf, 0, want))) <= np.where(inf, 0, tol) + 1e-30)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of tolerance; first at {i}: got {got[i]!r}, "
                             f"want {want[i]!r}, tolerance {tol[i]!r}")
