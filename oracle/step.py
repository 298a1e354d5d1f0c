"""What goes with the key-value cache in a serving step, in NumPy, from the definitions and in 64 bits -- TEST INFRASTRUCTURE
ONLY, as the C oracle: pages and slots, rotary positions, the attention of whole prompts. It shares no code with the CUDA
library.

Tolerances, derived before the kernels ran:
  * pages, lengths, offsets, positions, slots: whole numbers, equal;
  * rotary: the fraction of a turn in fp32 is off by 2^-24 of it, so the angle by at most pi 2^-24 and sine and cosine by that and
    their own error of 2 units in the last place, 2^-23 each (values up to 1): 2^-21.7; the amplitude's product, the pair's
    products and their sum another 3 roundings of 2^-24: relative to amplitude (|a| + |b|) together at most 2^-21; and half a step
    of bf16, 2^-8 relative;
  * prompt attention: logits, lse and probabilities as oracle/kv_cache.py derives them for decode attention, with L / 8 for L / 32 (a
    row's sum is kept in at least 8 partial sums); out: half a step of bf16, 2^-8 relative; relative to A = sum_j p_j |v_j|: dp,
    the rounding of the probabilities to bf16 before the product, 2^-8, and the sums' (L / 8 + 64) 2^-23.
"""
from __future__ import annotations

import numpy as np

import workloads as wl


# ------------------------------------------------------------------------------------------------ pages

class Pages:
    """A page table with its ring of free pages, lengths and tokens seen."""

    def __init__(self, rng, lens, page, width, spare):
        self.page, self.width = page, width
        self.lens = np.asarray(lens, np.int32).copy()
        used = [-(-int(x) // page) for x in lens]
        self.n_pages = max(1, sum(used) + spare)
        order = rng.permutation(self.n_pages)
        self.table = np.full((len(lens), width), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        free = order[at:]
        self.ring = np.full(self.n_pages, -7, np.int32)
        head = int(rng.integers(self.n_pages))
        self.ring[(head + np.arange(len(free))) % self.n_pages] = free
        self.ends = np.array([head, len(free)], np.int32)
        self.seen = (self.lens + np.where(self.lens > 0, rng.integers(0, 3, len(lens)) * 50, 0)).astype(np.int32)

    def resize(self, want, n_tokens):
        """(cu, positions, slots); the state changes in place. A queue, one sequence after another."""
        cap = self.width * self.page
        pages = lambda x: -(-int(x) // self.page)
        n = len(self.lens)
        fits = [0 <= int(o) <= cap and 0 <= int(w) <= cap for o, w in zip(self.lens, want)]
        head, count = (int(x) for x in self.ends)
        for b in range(n):
            if fits[b]:
                for p in range(pages(want[b]), pages(self.lens[b])):
                    self.ring[(head + count) % self.n_pages] = self.table[b, p]
                    self.table[b, p] = -1
                    count += 1
        there, asked_pages, asked_rows = count, 0, 0
        cu, positions, slots = [0], np.zeros(n_tokens, np.int32), np.full(n_tokens, -1, np.int64)
        for b in range(n):
            old, new = int(self.lens[b]), int(want[b])
            cu.append(cu[-1])
            if not fits[b]:
                continue
            if new <= old:
                self.lens[b] = new
                if new == 0:
                    self.seen[b] = 0
                continue
            more = pages(new) - pages(old)
            asked_pages += more
            asked_rows += new - old
            if (more and asked_pages > there) or asked_rows > n_tokens:
                continue
            for p in range(pages(old), pages(new)):
                self.table[b, p] = self.ring[head]
                head, count = (head + 1) % self.n_pages, count - 1
            for slot in range(old, new):
                row = cu[-1] + slot - old
                positions[row] = self.seen[b] + slot - old
                slots[row] = int(self.table[b, slot // self.page]) * self.page + slot % self.page
            cu[-1] += new - old
            self.lens[b] = new
            self.seen[b] += new - old
        self.ends[:] = head, count
        return np.array(cu, np.int32), positions, slots


# ------------------------------------------------------------------------------------------------ rotary positions

def rotary(x_bits, positions, turns, amplitude, heads, d, dim, layout):
    """([n, heads, d] turned rows in 64 bits, their tolerance); turns: [dim / 2] Python integers or uint64."""
    x = wl.bf16_bits_to_f32(x_bits).astype(np.float64).reshape(len(x_bits), heads, d)
    whole = np.asarray(positions, np.int64).astype(np.uint64)[:, None] * np.asarray(turns, np.uint64)   # modulo 2^64
    part = whole.view(np.int64).astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    cos, sin = amplitude * np.cos(part)[:, None], amplitude * np.sin(part)[:, None]
    a = slice(0, dim // 2) if layout == "half" else slice(0, dim, 2)
    b = slice(dim // 2, dim) if layout == "half" else slice(1, dim, 2)
    out, size = x.copy(), np.zeros_like(x)
    out[..., a], out[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    size[..., a] = size[..., b] = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    return out, 2.0 ** -8 * np.abs(out) * (size > 0) + 2.0 ** -21 * size


# ------------------------------------------------------------------------------------------------ prompts

def prompt(q_bits, k_bits, v_bits, cu, hq, hkv, d, scale, window=0):
    """(out, lse, tolerances of both) of packed prompts; rows behind the last sequence's: NaN."""
    n, g = len(q_bits), hq // hkv
    f64 = lambda x, h: wl.bf16_bits_to_f32(x).astype(np.float64).reshape(n, h, d)
    q, k, v = f64(q_bits, hq), f64(k_bits, hkv), f64(v_bits, hkv)
    out, lse = np.full((n, hq, d), np.nan), np.full((n, hq), np.nan)
    t_out, t_lse = np.zeros_like(out), np.zeros_like(lse)
    for s, e in zip(cu[:-1], cu[1:]):
        i = np.arange(e - s)
        seen = i[None] <= i[:, None]
        if window:
            seen &= i[None] > i[:, None] - window
        for h in range(hq):
            K, V, Q = k[s:e, h // g], v[s:e, h // g], q[s:e, h]
            with np.errstate(invalid="ignore", over="ignore"):
                x = np.where(seen, Q @ K.T * scale, -np.inf)
                size = np.where(seen, np.abs(Q) @ np.abs(K).T * abs(scale), 0).max(-1, initial=0)
                dx = (d * 2.0 ** -23 + 2.0 ** -22) * size
                m = x.max(-1, initial=-np.inf)
                p = np.exp(x - np.where(np.isfinite(m), m, 0)[:, None])
                total = p.sum(-1)
                p /= np.where(total > 0, total, 1)[:, None]
                L = seen.sum(-1)
                dsum = (L / 8 + 8) * 2.0 ** -23
                dp = 2 * dx + dsum
                # Rows that a value is masked for do not see it, whatever it is.
                far = ~np.isfinite(V)
                out[s:e, h] = p @ np.where(far, 0, V)
                for j, c in zip(*np.nonzero(far)):
                    out[s:e, h, c] += np.where(seen[:, j], V[j, c], 0)
                a = p @ np.abs(np.where(far, 0, V))
                t_out[s:e, h] = a * (dp + 2.0 ** -8 + (L / 8 + 64) * 2.0 ** -23)[:, None] + 2.0 ** -8 * np.abs(out[s:e, h])
                with np.errstate(divide="ignore"):
                    lse[s:e, h] = np.where(np.isfinite(m), m, 0) + np.log(total)
                t_lse[s:e, h] = dx + dsum + 2.0 ** -22 * np.abs(lse[s:e, h])
    return out, lse, t_out, t_lse
