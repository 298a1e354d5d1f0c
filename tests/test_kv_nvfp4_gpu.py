"""The key-value cache held in NVFP4 on the GPU: attention over it within the tolerances that oracle/kv_cache.py derives, the
append's codes and evicted caches byte for byte. What a call must not touch or use is poisoned as in the
other formats' tests."""
import numpy as np
import pytest

import workloads as wl
from oracle import kv_nvfp4 as ref
from oracle.kv_cache import check_close
from tests.parity import Guarded
from tests.test_kv_gpu import bits, check_attend, mbd, run_attend, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


class Cache(ref.Cache):
    """With a copy on the GPU between guard bands."""

    def device(self, mbd):
        put = lambda a, dt: None if a is None else Guarded(torch, a.size, dt, fill=a)
        self.g = dict(k=put(self.k_raw, torch.uint8), v=put(self.v_raw, torch.uint8), ks=put(self.ks, torch.float32),
                      vs=put(self.vs, torch.float32), weight=put(self.weight, torch.float32),
                      position=put(self.position, torch.int32), table=put(self.table, torch.int32),
                      lens=put(self.lens, torch.int32))
        w = {n: (None if g is None else g.view) for n, g in self.g.items()}
        self.table_d, self.lens_d = w["table"], w["lens"]
        self.c = mbd.kv_cache(w["k"], w["v"], self.n_pages, self.page, self.hkv, self.d, "nvfp4", "static", w["ks"], w["vs"],
                              w["weight"], w["position"], self.stride if self.gap else 0)
        return self.c

    def check_equal(self, what="", skip=()):
        host = dict(k=self.k_raw, v=self.v_raw, ks=self.ks, vs=self.vs, weight=self.weight, position=self.position,
                    table=self.table, lens=self.lens)
        for name, g in self.g.items():
            if g is None:
                continue
            g.check_guards(f"{what} {name}")
            if name not in skip:
                as_bits = {1: np.uint8, 4: np.uint32}[host[name].dtype.itemsize]
                np.testing.assert_array_equal(g.numpy(as_bits), host[name].reshape(-1).view(as_bits), f"{what}: {name}")


# ------------------------------------------------------------------------------------------------ attention

@pytest.mark.parametrize("hq,hkv,d", [(12, 2, 128), (32, 8, 128), (8, 1, 128), (16, 1, 128), (5, 5, 64), (16, 1, 64), (6, 2, 256),
                                      (9, 1, 256), (40, 2, 128), (17, 1, 64), (64, 1, 128)])
def test_attention_head_layouts(mbd, hq, hkv, d):
    rng = np.random.default_rng(hq + d)
    c = Cache(rng, [37, 0, 1, 200, 129, 1000], hkv, d, 16)
    c.device(mbd)
    check_attend(mbd, c, rng, hq)
    check_attend(mbd, c, rng, hq, accumulate=True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [1, 2, 4, 8, 16, 32, 64, 256, 1024])
def test_attention_lengths_and_pages(mbd, page, d):
    """Lengths around the sizes that the work is cut into, in every order, pages that end inside a step."""
    rng = np.random.default_rng(page)
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 511, 513, 1000]
    c = Cache(rng, rng.permutation(lens), 2, d, page)
    c.device(mbd)
    check_attend(mbd, c, rng, 6, accumulate=True, q_gap=64)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 5000])
def test_attention_window(mbd, window):
    rng = np.random.default_rng(window)
    c = Cache(rng, [0, 1, 5, 16, 99, 100, 101, 640, 1500], 1, 128, 32)
    c.device(mbd)
    check_attend(mbd, c, rng, 4, window=window, accumulate=True)


@pytest.mark.parametrize("n,length,hq,hkv,d", [(1, 40000, 16, 2, 128), (1, 9000, 32, 8, 128), (2, 20001, 4, 1, 256),
                                               (300, 40, 8, 2, 64), (1, 1, 1, 1, 64), (700, 3, 2, 1, 128), (1, 30000, 16, 1, 64)])
def test_attention_shapes(mbd, n, length, hq, hkv, d):
    rng = np.random.default_rng(n)
    lens = np.full(n, length) if n == 1 else rng.integers(0, length + 1, n)
    c = Cache(rng, lens, hkv, d, 16)
    c.device(mbd)
    check_attend(mbd, c, rng, hq, accumulate=n < 500)


def test_attention_strides_and_width(mbd):
    """Pages apart in the pool, a page table wider than any sequence, no lse; interleaved halves of one pool's pages."""
    rng = np.random.default_rng(5)
    c = Cache(rng, [70, 3, 200], 2, 128, 16, width=50, gap=48)
    c.device(mbd)
    check_attend(mbd, c, rng, 8, accumulate=True)
    check_attend(mbd, c, rng, 8, lse=False)
    c = Cache(rng, [33, 7], 2, 64, 8, gap=2 * 8 * 36, meta=False)
    c.device(mbd)
    pool = np.zeros((c.n_pages, 2, 2 * 8 * 36), np.uint8)
    pool[:, 0], pool[:, 1] = (x.reshape(c.n_pages, -1)[:, :2 * 8 * 36] for x in (c.k_raw, c.v_raw))
    p = up(pool)
    c.c = mbd.kv_cache(p, p[:, 1], c.n_pages, 8, 2, 64, "nvfp4", k_scale=c.g["ks"].view, v_scale=c.g["vs"].view, page_stride=c.stride)
    check_attend(mbd, c, rng, 4)


def test_attention_offsets_beyond_32_bits(mbd):
    """Pages 2 GiB apart in a pool, in the attention and in the append."""
    rng = np.random.default_rng(13)
    c = Cache(rng, [40], 1, 128, 16, spare=1, meta=False)
    stride, page = 1 << 31, 16 * 72
    pools = [torch.zeros((c.n_pages - 1) * stride + page, dtype=torch.uint8, device="cuda") for _ in range(2)]
    for pool, raw in zip(pools, (c.k_raw, c.v_raw)):
        for i in range(c.n_pages):
            pool[i * stride:i * stride + page] = up(raw.reshape(c.n_pages, -1)[i])
    c.device(mbd)
    c.c = mbd.kv_cache(pools[0], pools[1], c.n_pages, 16, 1, 128, "nvfp4", k_scale=c.g["ks"].view, v_scale=c.g["vs"].view,
                       page_stride=stride)
    check_attend(mbd, c, rng, 2)
    k, v = bits(rng, 1, 128), bits(rng, 1, 128)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 1, 1)
    c.store(0, [39], k.reshape(1, 1, 128), v.reshape(1, 1, 128))
    for name, pool in zip("kv", pools):
        c.g[name].view.copy_(torch.stack([pool[i * stride:i * stride + page] for i in range(c.n_pages)]).view(-1))
    c.check_equal("append")


def test_attention_masked_and_unusable_scales(mbd):
    """Slots without a token hold NaN scales (the poison); a tensor scale out of range counts as 0: equal weights, zeros."""
    rng = np.random.default_rng(7)
    c = Cache(rng, [37, 100], 2, 128, 16)
    c.device(mbd)
    for bad in (0.0, -1.0, float("nan"), float("inf"), 2.0 ** 65):
        c.g["ks"].view.fill_(bad)
        c.g["vs"].view.fill_(bad)
        _, out, lse, _ = run_attend(mbd, c, rng, 4)
        assert not (out & 0x7FFF).any()
        np.testing.assert_allclose(lse, np.log([[37] * 4, [100] * 4]), rtol=1e-6)


def test_attention_bad_pages(mbd):
    """A page number outside the pool counts as masked, and is flagged."""
    rng = np.random.default_rng(8)
    c = Cache(rng, [64, 40], 1, 128, 16)
    c.device(mbd)
    c.table_d.view(2, -1)[0, 1] = 1 << 29
    mbd.device_error_flags(clear=True)
    q, out, lse, scale = run_attend(mbd, c, rng, 4)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    k, v = (x[0] for x in c.rows(0, np.r_[0:16, 32:64]))
    x = wl.bf16_bits_to_f32(q[0]).astype(np.float64).reshape(4, 128) @ k.T * scale
    p = np.exp(x - x.max(-1, keepdims=True))
    want = p / p.sum(-1, keepdims=True) @ v
    # rows as usual: half a step of bf16, and 2^-10 of sum p |v| for everything else
    check_close(wl.bf16_bits_to_f32(out)[0], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * (p / p.sum(-1, keepdims=True) @ np.abs(v)), "out")


def test_attention_replayed_with_many_parts(mbd):
    rng = np.random.default_rng(14)
    c, other = Cache(rng, [30011], 1, 128, 64), Cache(rng, [5000, 7], 2, 128, 64)
    c.device(mbd)
    other.device(mbd)
    q, q2 = up(bits(rng, 1, 8 * 128)), up(bits(rng, 2, 4 * 128))
    nb = max(mbd.paged_attention_workspace_bytes(c.c, c.width, 1, 8), mbd.paged_attention_workspace_bytes(other.c, other.width, 2, 4))
    ws = torch.full((nb,), 0xAB, dtype=torch.uint8, device="cuda")
    out, out2 = torch.empty(1, 1024, dtype=torch.bfloat16, device="cuda"), torch.empty(2, 512, dtype=torch.bfloat16, device="cuda")
    call = lambda: mbd.paged_attention_decode(out, q, 0, c.c, c.table_d, c.width, c.lens_d, 1, 8, 0.09, 0, None, False, ws, nb)
    call()
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(6):
        if i % 2:
            mbd.paged_attention_decode(out2, q2, 0, other.c, other.table_d, other.width, other.lens_d, 2, 4, 0.09, 0, None,
                                       False, ws, nb)
        out.zero_()
        g.replay()
        assert torch.equal(out, want), f"replay {i}"


# ------------------------------------------------------------------------------------------------ append and eviction

@pytest.mark.parametrize("hkv,d,page", [(1, 64, 1), (2, 64, 2), (8, 128, 16), (3, 128, 64), (2, 256, 8), (5, 64, 32), (40, 128, 16)])
def test_append_single_tokens(mbd, hkv, d, page):
    rng = np.random.default_rng(hkv)
    c = Cache(rng, rng.integers(1, 300, 37), hkv, d, page)
    c.device(mbd)
    k, v = bits(rng, 37, hkv * d + 64), bits(rng, 37, hkv * d + 64, sigma=30.0)   # blocks past 6 * 448 S saturate
    k[5, :32] = 0                                            # zero blocks
    pos = rng.integers(0, 1 << 30, 37).astype(np.int32)
    mbd.kv_cache_append(c.c, up(k), up(v), hkv * d + 64, c.table_d, c.width, c.lens_d, 37, 37, None, up(pos))
    torch.cuda.synchronize()
    for b in range(37):
        c.store(b, [c.lens[b] - 1], k[b:b + 1, :hkv * d].reshape(1, hkv, d), v[b:b + 1, :hkv * d].reshape(1, hkv, d), [pos[b]])
    c.check_equal("append")


@pytest.mark.parametrize("scales", [(1e-3, 0.77), (2.0 ** -20, 1e4), (1.9999999, 3e-20), (2.0 ** -63, 2.0 ** 63), (0.0, float("nan"))])
def test_append_tensor_scales(mbd, scales):
    """Scales of any size: blocks that saturate, blocks whose scale rounds to 0, quotients by scales under 2^-60, unusable ones."""
    rng = np.random.default_rng(3)
    usable = [2.0 ** -64 <= s <= 2.0 ** 64 for s in scales]   # the rule of the format (3e-20 is 2^-64.9)
    c = Cache(rng, [300], 2, 128, 16, scales=[s if ok else 1.0 for s, ok in zip(scales, usable)])
    c.device(mbd)
    c.g["ks"].view.fill_(scales[0])
    c.g["vs"].view.fill_(scales[1])
    k, v = (bits(rng, 290, 256, sigma=s) for s in (1.0, 1.0))
    v[:, 128:] = bits(rng, 290, 128, sigma=1e-22)
    cu = np.array([0, 290], np.int32)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 1, 290, up(cu))
    torch.cuda.synchronize()
    c.store(0, np.arange(10, 300), k.reshape(-1, 2, 128), v.reshape(-1, 2, 128))
    p, _, s = c.at(0, np.arange(10, 300))
    for raw, ok in zip((c.k_raw, c.v_raw), usable):
        if not ok:
            c.view(raw)[p, :, s] = c.blocks(raw)[p, :, s] = 0
    c.check_equal("append", skip=("ks", "vs"))


@pytest.mark.parametrize("hkv,d,page", [(8, 128, 16), (1, 64, 8), (2, 256, 4), (3, 64, 1)])
def test_append_prompts(mbd, hkv, d, page):
    rng = np.random.default_rng(page)
    new = np.array([0, 1, 170, 33, 0, 64, 400])
    c = Cache(rng, new + np.array([5, 0, 3, 100, 0, 64, 0]), hkv, d, page)
    c.device(mbd)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = int(cu[-1]) + 3                                    # rows behind the last sequence's are left alone
    k, v = bits(rng, rows, hkv * d), bits(rng, rows, hkv * d)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, len(new), rows, up(cu))
    torch.cuda.synchronize()
    for b, n in enumerate(new):
        if n:
            at = slice(cu[b], cu[b + 1])
            c.store(b, np.arange(c.lens[b] - n, c.lens[b]), k[at].reshape(-1, hkv, d), v[at].reshape(-1, hkv, d))
    c.check_equal("append")


@pytest.mark.parametrize("hkv,d,page,budget,recent", [(2, 64, 1, 40, 8), (2, 128, 16, 100, 0), (1, 256, 8, 64, 64), (3, 64, 64, 7, 3),
                                                      (2, 128, 4, 500, 100)])
def test_evict(mbd, hkv, d, page, budget, recent):
    rng = np.random.default_rng(budget)
    c = Cache(rng, [0, 39, 41, 600, 101, 1, 2000], hkv, d, page)
    c.device(mbd)
    new = torch.full((7,), -5, dtype=torch.int32, device="cuda")
    mbd.kv_cache_evict(c.c, new, c.lens_d, c.table_d, c.width, 7, budget, recent)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(new.cpu().numpy(), c.evict(budget, recent))
    c.check_equal("evict")


def test_decode_with_eviction(mbd):
    """Prompts, then decode steps (append, attention with accumulation) and evictions: the cache follows step by step."""
    rng = np.random.default_rng(20)
    n, hkv, hq, d, page, budget, full = 3, 2, 8, 128, 8, 24, 40
    c = Cache(rng, [full] * n, hkv, d, page, fill=False)
    prompts = np.array([30, 12, 33], np.int32)
    c.lens = prompts.copy()
    c.device(mbd)
    cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    k, v = bits(rng, cu[-1], hkv * d), bits(rng, cu[-1], hkv * d)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, n, int(cu[-1]), up(cu))
    for b in range(n):
        at = slice(cu[b], cu[b + 1])
        c.store(b, np.arange(prompts[b]), k[at].reshape(-1, hkv, d), v[at].reshape(-1, hkv, d))
    torch.cuda.synchronize()
    c.check_equal("append")
    new_lens = torch.empty(n, dtype=torch.int32, device="cuda")
    total = prompts.copy()
    for step in range(14):
        c.lens_d += 1
        c.lens += 1
        k, v = bits(rng, n, hkv * d), bits(rng, n, hkv * d)
        mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, n, n, None, up(total))
        for b in range(n):
            c.store(b, [c.lens[b] - 1], k[b].reshape(1, hkv, d), v[b].reshape(1, hkv, d), [total[b]])
        torch.cuda.synchronize()
        c.check_equal("append")
        check_attend(mbd, c, rng, hq, accumulate=True)
        if int(c.lens.max()) == full:
            mbd.kv_cache_evict(c.c, new_lens, c.lens_d, c.table_d, c.width, n, budget, 6)
            c.lens_d.copy_(new_lens)
            c.lens = c.evict(budget, 6)
        total += 1
        c.check_equal(f"step {step}")
