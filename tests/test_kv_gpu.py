"""The key-value cache on the GPU against the 64-bit reference: appended and evicted caches byte for byte, attention
within the tolerances that oracle/kv_cache.py derives. Everything a call must not touch or use is poisoned: slots
without a token hold NaN, guard bands lie around every tensor, the page table's unused entries name no page."""
import numpy as np
import pytest

import workloads as wl
from oracle import kv_cache as ref
from oracle.kv_cache import check_close
from tests.parity import Guarded

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mbd():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from memory_bound_decoder_gb300 import build
    build.build()
    import memory_bound_decoder_gb300 as m
    m.get_lib()
    m.device_error_flags(clear=True)
    yield m
    torch.cuda.synchronize()


def bits(rng, *shape, sigma=1.0):
    return wl.f32_to_bf16_bits((sigma * rng.standard_normal(shape)).astype(np.float32))


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a).view(np.int16 if a.dtype == np.uint16 else a.dtype)).cuda()


class Cache(ref.Cache):
    """With a copy on the GPU between guard bands."""

    def device(self, mbd):
        it = {"bf16": torch.int16, "fp8": torch.uint8}[self.fmt]
        as_np = lambda a: a.view(np.int16) if a.dtype == np.uint16 else a
        put = lambda a, dt: None if a is None else Guarded(torch, a.size, dt, fill=as_np(a))
        self.g = dict(k=put(self.k_raw, it), v=put(self.v_raw, it), ks=put(self.ks, torch.float32),
                      vs=put(self.vs, torch.float32), weight=put(self.weight, torch.float32),
                      position=put(self.position, torch.int32), table=put(self.table, torch.int32),
                      lens=put(self.lens, torch.int32))
        w = {n: (None if g is None else g.view) for n, g in self.g.items()}
        self.table_d, self.lens_d = w["table"], w["lens"]
        self.c = mbd.kv_cache(w["k"], w["v"], self.n_pages, self.page, self.hkv, self.d, self.fmt, self.mode, w["ks"],
                              w["vs"], w["weight"], w["position"], self.stride if self.gap else 0)
        return self.c

    def check_equal(self, what="", skip=()):
        """Every byte of the GPU's copy, guard bands included, is what the host's says."""
        host = dict(k=self.k_raw, v=self.v_raw, ks=self.ks, vs=self.vs, weight=self.weight, position=self.position,
                    table=self.table, lens=self.lens)
        for name, g in self.g.items():
            if g is None:
                continue
            g.check_guards(f"{what} {name}")
            if name not in skip:
                bits = {1: np.uint8, 2: np.uint16, 4: np.uint32}[host[name].dtype.itemsize]
                np.testing.assert_array_equal(g.numpy(bits), host[name].reshape(-1).view(bits), f"{what}: {name}")


STORES = [("bf16", "static"), ("fp8", "static"), ("fp8", "dynamic")]


def run_attend(mbd, c, rng, hq, window=0, accumulate=False, q_gap=0, scale=None, stream=None, lse=True):
    n, d = len(c.lens), c.d
    scale = d ** -0.5 if scale is None else scale
    q = bits(rng, n, hq * d + q_gap) if q_gap else bits(rng, n, hq * d)
    q[:, :hq * d] = bits(rng, n, hq * d, sigma=2.0)
    out = Guarded(torch, n * hq * d, torch.int16)
    lse_g = Guarded(torch, n * hq, torch.float32)
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, n, hq, accumulate)
    ws = torch.full((nb + 512,), 0xFF, dtype=torch.uint8, device="cuda")   # NaN wherever it is read unwritten
    qd = up(q)
    torch.cuda.synchronize()
    mbd.paged_attention_decode(out.view, qd, q.shape[1], c.c, c.table_d, c.width, c.lens_d, n, hq, scale, window,
                               lse_g.view if lse else None, accumulate, ws, nb, stream)
    torch.cuda.synchronize()
    assert bool((ws[nb:] == 0xFF).all()), "write behind the workspace"
    out.check_guards("out")
    lse_g.check_guards("lse")
    return q[:, :hq * d].copy(), out.numpy(np.uint16).reshape(n, hq, d), lse_g.numpy(np.float32).reshape(n, hq), scale


def check_attend(mbd, c, rng, hq, window=0, accumulate=False, **kw):
    mbd.device_error_flags(clear=True)
    q, out, lse, scale = run_attend(mbd, c, rng, hq, window, accumulate, **kw)
    want = c.attend(q, hq, scale, window, accumulate)
    check_close(wl.bf16_bits_to_f32(out), want[0], want[2], "out")
    if kw.get("lse", True):
        check_close(lse, want[1], want[3], "lse")
    if accumulate:
        w = c.g["weight"].numpy(np.float32).reshape(c.weight.shape)
        dead = np.isnan(c.weight)
        assert np.isnan(w[dead]).all()
        check_close(w[~dead], want[4][~dead], want[5][~dead], "weight")
        c.weight[:] = w
    c.check_equal("attention")
    assert mbd.device_error_flags() == 0


# ------------------------------------------------------------------------------------------------ attention

HEADS = [(12, 2, 128), (32, 8, 128), (8, 1, 128), (16, 1, 128), (5, 5, 64), (16, 1, 64), (6, 2, 256), (9, 1, 256),
         (40, 2, 128), (17, 1, 64), (64, 1, 128)]


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("hq,hkv,d", HEADS)
def test_attention_head_layouts(mbd, hq, hkv, d, fmt, mode):
    rng = np.random.default_rng(hash((hq, hkv, d)) % 1000)
    c = Cache(rng, [37, 0, 1, 200, 129], hkv, d, 16, fmt, mode)
    c.device(mbd)
    check_attend(mbd, c, rng, hq)
    check_attend(mbd, c, rng, hq, accumulate=True)


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("page", [1, 2, 8, 16, 32, 64, 256, 1024])
def test_attention_lengths_and_pages(mbd, page, fmt, mode):
    """Lengths around the sizes that the work is cut into, in every order, pages that end inside a step."""
    rng = np.random.default_rng(page)
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 0, 127, 128, 129, 255, 256, 257, 511, 513, 1000]
    c = Cache(rng, rng.permutation(lens), 2, 128, page, fmt, mode)
    c.device(mbd)
    check_attend(mbd, c, rng, 6, accumulate=True, q_gap=64)


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 5000])
def test_attention_window(mbd, window, fmt, mode):
    rng = np.random.default_rng(window)
    c = Cache(rng, [0, 1, 5, 16, 99, 100, 101, 640, 1500], 1, 64, 32, fmt, mode)
    c.device(mbd)
    check_attend(mbd, c, rng, 4, window=window, accumulate=True)


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("n,length,hq,hkv,d", [(1, 40000, 16, 2, 128), (1, 9000, 32, 8, 128), (2, 20001, 4, 1, 256),
                                               (300, 40, 8, 2, 64), (1, 1, 1, 1, 64), (700, 3, 2, 1, 128)])
def test_attention_shapes(mbd, n, length, hq, hkv, d, fmt, mode):
    """One long sequence split over the card; more sequences than a block scans at once."""
    rng = np.random.default_rng(n)
    lens = np.full(n, length) if n == 1 else rng.integers(0, length + 1, n)
    c = Cache(rng, lens, hkv, d, 16, fmt, mode)
    c.device(mbd)
    check_attend(mbd, c, rng, hq, accumulate=n < 500)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_of_an_empty_batch(mbd, n):
    """Nothing cached at all: zeros and -inf, weights as they were."""
    rng = np.random.default_rng(n)
    c = Cache(rng, [0] * n, 2, 64, 16, "bf16")
    c.device(mbd)
    check_attend(mbd, c, rng, 4, accumulate=True)


def test_attention_offsets_beyond_32_bits(mbd):
    """Pages 2 GiB apart in a pool: byte offsets past 2^32, in the attention and in the append."""
    rng = np.random.default_rng(13)
    c = Cache(rng, [40], 1, 64, 16, "bf16", spare=1, meta=False)
    stride = 1 << 30
    pools = [torch.zeros((c.n_pages - 1) * stride + 16 * 64, dtype=torch.int16, device="cuda") for _ in range(2)]
    for pool, raw in zip(pools, (c.k_raw, c.v_raw)):
        for i in range(c.n_pages):
            pool[i * stride:i * stride + 1024] = up(raw.reshape(c.n_pages, -1)[i])
    c.device(mbd)
    c.c = mbd.kv_cache(pools[0], pools[1], c.n_pages, 16, 1, 64, page_stride=stride)
    assert c.table[0, :3].max() >= 2
    check_attend(mbd, c, rng, 2)
    k, v = bits(rng, 1, 64), bits(rng, 1, 64)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 1, 1)
    c.store(0, [39], k.reshape(1, 1, 64), v.reshape(1, 1, 64))
    for pool, raw in zip(pools, (c.k_raw, c.v_raw)):
        for i in range(c.n_pages):
            got = pool[i * stride:i * stride + 1024].cpu().numpy().view(np.uint16)
            np.testing.assert_array_equal(got, raw.reshape(c.n_pages, -1)[i])


@pytest.mark.parametrize("fmt,mode", STORES)
def test_attention_replayed_with_many_parts(mbd, fmt, mode):
    """A captured call over one long sequence, whose head is cut into parts of parts, replayed over a workspace that
    other calls use between the replays: the same bits every time."""
    rng = np.random.default_rng(14)
    c = Cache(rng, [30011], 1, 128, 64, fmt, mode)
    other = Cache(rng, [5000, 7], 2, 128, 64, fmt, mode)
    c.device(mbd)
    other.device(mbd)
    q, q2 = up(bits(rng, 1, 8 * 128)), up(bits(rng, 2, 4 * 128))
    nb = max(mbd.paged_attention_workspace_bytes(c.c, c.width, 1, 8),
             mbd.paged_attention_workspace_bytes(other.c, other.width, 2, 4))
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


@pytest.mark.parametrize("fmt,mode", STORES)
def test_attention_strides_and_width(mbd, fmt, mode):
    """Pages apart in the pool, a page table wider than any sequence, and no lse."""
    rng = np.random.default_rng(5)
    c = Cache(rng, [70, 3, 200], 2, 128, 16, fmt, mode, width=50, gap=48)
    c.device(mbd)
    check_attend(mbd, c, rng, 8, accumulate=True)
    check_attend(mbd, c, rng, 8, lse=False)


def test_attention_interleaved_pool(mbd):
    """k and v as the halves of one pool's pages."""
    rng = np.random.default_rng(6)
    hkv, d, page, hq = 2, 64, 8, 4
    c = Cache(rng, [33, 7], hkv, d, page, "bf16", gap=hkv * page * d)
    c.device(mbd)
    pool = np.zeros((c.n_pages, 2, hkv, page, d), np.uint16)
    pool[:, 0], pool[:, 1] = c.view(c.k_raw), c.view(c.v_raw)
    p = up(pool)
    c.c = mbd.kv_cache(p, p[:, 1], c.n_pages, page, hkv, d, page_stride=c.stride)
    check_attend(mbd, c, rng, hq)


@pytest.mark.parametrize("fmt,mode", STORES)
def test_attention_peaked_and_rising_logits(mbd, fmt, mode):
    """Logits that rise along the cache by far more than any lazily kept maximum allows, and that fall; scales of the
    values that differ by many powers of two (dynamic)."""
    rng = np.random.default_rng(7)
    hkv, d, L = 2, 128, 1200
    c = Cache(rng, [L, L], hkv, d, 16, fmt, mode)
    for b, slope in ((0, 1.0), (1, -1.0)):
        ramp = np.exp2(slope * np.linspace(-6, 6, L)).astype(np.float32)[:, None, None]
        k = np.abs(rng.standard_normal((L, hkv, d))).astype(np.float32) * ramp
        v = rng.standard_normal((L, hkv, d)).astype(np.float32) * (2.0 ** rng.integers(-20, 20, (L, hkv, 1))
                                                                   if mode == "dynamic" else 1.0)
        c.store(b, np.arange(L), wl.f32_to_bf16_bits(k), wl.f32_to_bf16_bits(v.astype(np.float32)))
    c.device(mbd)
    check_attend(mbd, c, rng, 8, accumulate=True)
    check_attend(mbd, c, rng, 8, scale=-0.01)


def test_attention_extremes_propagate(mbd):
    """A NaN in view reaches its own sequence and head only; +-inf values follow the definition; a key of the type's
    lowest values is given no weight."""
    rng = np.random.default_rng(8)
    c = Cache(rng, [100, 100, 100], 2, 64, 16, "bf16")
    kv, vv = c.view(c.k_raw), c.view(c.v_raw)
    p, _, s = c.at(0, [50])
    vv[p[0], 1, s[0], 3] = 0x7FC0                     # one NaN value: one output element of each of 2 heads
    p, _, s = c.at(1, [10])
    vv[p[0], 0, s[0], 5] = 0x7F80                     # an infinite value
    p, _, s = c.at(2, [20])
    kv[p[0], 0, s[0], :] = 0xFF7F                     # the lowest finite key; queries positive: logit about -3e38
    c.device(mbd)
    q = np.abs(wl.bf16_bits_to_f32(bits(rng, 3, 4 * 64)))
    qb = wl.f32_to_bf16_bits(q)
    out = torch.empty(3 * 4 * 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(12, device="cuda")
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, 3, 4)
    ws = torch.empty(max(1, nb), dtype=torch.uint8, device="cuda")
    mbd.paged_attention_decode(out, up(qb), 0, c.c, c.table_d, c.width, c.lens_d, 3, 4, 0.125, 0, lse, False, ws, nb)
    o = out.view(3, 4, 64).float().cpu().numpy()
    nan = np.isnan(o)
    want = np.zeros_like(nan)
    want[0, 2:, 3] = True
    np.testing.assert_array_equal(nan, want)
    assert np.isposinf(o[1, :2, 5]).all() and np.isfinite(np.delete(o[1, :2], 5, 1)).all()
    c.lens_d.fill_(100)
    assert torch.isfinite(lse).all()
    p, _, s = c.at(2, [20])
    L = c.lens[2]
    k, v = c.rows(2, np.delete(np.arange(L), 20))     # as if that token were not there, for key-value head 0
    x = np.einsum("hd,ld->hl", q[2].reshape(4, 64)[:2].astype(np.float64), k[0]) * 0.125
    pr = np.exp(x - x.max(-1, keepdims=True))
    pr /= pr.sum(-1, keepdims=True)
    np.testing.assert_allclose(o[2, :2], pr @ v[0], rtol=2 ** -8, atol=1e-3)


def test_attention_bad_indices_are_reported_and_masked(mbd):
    """Page numbers outside the pool and lengths outside the table: the error bit, no access, and the rest as if those
    slots were masked."""
    rng = np.random.default_rng(9)
    c = Cache(rng, [64, 50, 30], 2, 64, 16, "bf16")
    c.device(mbd)
    keep = c.table.copy()
    c.table_d.view(3, -1)[0, 1] = c.n_pages            # slots 16..31 of sequence 0
    c.table_d.view(3, -1)[1, 0] = -7                   # slots 0..15 of sequence 1
    c.lens_d[2] = -5
    mbd.device_error_flags(clear=True)
    q, out, lse, scale = run_attend(mbd, c, rng, 4)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    for b, live in ((0, np.r_[0:16, 32:64]), (1, np.arange(16, 50))):
        k, v = c.rows(b, live)
        x = np.einsum("hgd,hld->hgl", wl.bf16_bits_to_f32(q[b]).astype(np.float64).reshape(2, 2, 64), k) * scale
        pr = np.exp(x - x.max(-1, keepdims=True))
        pr /= pr.sum(-1, keepdims=True)
        np.testing.assert_allclose(wl.bf16_bits_to_f32(out[b]), np.einsum("hgl,hld->hgd", pr, v).reshape(4, 64),
                                   rtol=2 ** -7, atol=1e-3)
    assert not out[2].any() and np.isneginf(lse[2]).all()
    c.table_d.copy_(torch.from_numpy(keep.reshape(-1)))
    c.lens_d.copy_(torch.tensor([64, 50, 1 << 30], dtype=torch.int32))
    run_attend(mbd, c, rng, 4)                         # clamped to the table's width; its unused pages are no pages
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX


def test_attention_is_deterministic_and_leaves_no_state(mbd):
    """Equal calls give equal bits, also after the workspace was used by another shape and on another stream."""
    rng = np.random.default_rng(10)
    a = Cache(rng, [3000, 10, 700], 2, 128, 16, "bf16")
    b = Cache(rng, [100] * 40, 4, 64, 8, "fp8", "dynamic")
    a.device(mbd)
    b.device(mbd)
    qa, qb = up(bits(rng, 3, 8 * 128)), up(bits(rng, 40, 4 * 64))
    nb = max(mbd.paged_attention_workspace_bytes(a.c, a.width, 3, 8), mbd.paged_attention_workspace_bytes(b.c, b.width, 40, 4))
    ws = torch.empty(nb + 1, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    outs = []
    torch.cuda.synchronize()
    for i in range(4):
        stream = side if i % 2 else torch.cuda.current_stream()
        out, lse = torch.empty(3, 8 * 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")
        ob = torch.empty(40, 256, dtype=torch.bfloat16, device="cuda")
        torch.cuda.synchronize()
        mbd.paged_attention_decode(ob, qb, 0, b.c, b.table_d, b.width, b.lens_d, 40, 4, 0.1, 0, None, False, ws, nb, stream)
        mbd.paged_attention_decode(out, qa, 0, a.c, a.table_d, a.width, a.lens_d, 3, 8, 0.1, 0, lse, False, ws, nb, stream)
        torch.cuda.synchronize()
        outs.append((out.cpu(), lse.cpu(), ob.cpu()))
    for o in outs[1:]:
        for x, y in zip(o, outs[0]):
            assert torch.equal(x, y)


def test_attention_on_two_streams_at_once(mbd):
    """Calls on two streams over one cache, each with a workspace of its own, and torch's current stream taken up where
    none is given: the bits of the calls made alone."""
    rng = np.random.default_rng(17)
    c = Cache(rng, [6000, 3, 900], 2, 128, 16, "bf16")
    c.device(mbd)
    qs = [up(bits(rng, 3, 8 * 128)) for _ in range(2)]
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, 3, 8)
    spaces = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty(3, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    call = lambda i: mbd.paged_attention_decode(outs[i], qs[i], 0, c.c, c.table_d, c.width, c.lens_d, 3, 8, 0.09, 0, None,
                                                False, spaces[i], nb)
    want = []
    for i in range(2):
        call(i)
        torch.cuda.synchronize()
        want.append(outs[i].clone())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(2):
        assert mbd._stream(streams[i]) == streams[i].cuda_stream
        with torch.cuda.stream(streams[i]):
            assert mbd._stream(None) == streams[i].cuda_stream
    for _ in range(20):
        for i in range(2):
            outs[i].zero_()
        torch.cuda.synchronize()
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i)
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i])


# ------------------------------------------------------------------------------------------------ append

@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("hkv,d,page", [(8, 128, 16), (1, 64, 1), (3, 256, 8), (5, 64, 64)])
def test_append_one_token_each(mbd, hkv, d, page, fmt, mode):
    rng = np.random.default_rng(d + page)
    c = Cache(rng, [1, 2, 17, 16, 64, 65, 100], hkv, d, page, fmt, mode, gap=16)
    c.device(mbd)
    n, wide = 7, 2 * hkv * d + 24
    rows = bits(rng, n, wide)
    rows[2, :hkv * d] = 0                                 # an all-zero key row; the largest finite values
    rows[3, hkv * d:2 * hkv * d] = 0x7F7F
    rd = up(rows)
    mbd.device_error_flags(clear=True)
    for _ in range(2):                                    # a second call stores the same
        mbd.kv_cache_append(c.c, rd, rd[:, hkv * d:], wide, c.table_d, c.width, c.lens_d, n, n)
    torch.cuda.synchronize()
    for b in range(n):
        with np.errstate(over="ignore"):
            c.store(b, [c.lens[b] - 1], rows[b:b + 1, :hkv * d].reshape(1, hkv, d),
                    rows[b:b + 1, hkv * d:2 * hkv * d].reshape(1, hkv, d))
    c.check_equal("append")
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("counts,padding", [([5, 0, 1, 33, 0, 17, 64], 0), ([0, 3], 9), ([700, 1, 900], 3),
                                            ([1] * 300, 20), ([4000], 0)])
def test_append_prompts(mbd, counts, padding, fmt, mode):
    """Uneven prompts behind what is cached already, sequences without new tokens, padding rows behind the last; given
    positions."""
    rng = np.random.default_rng(sum(counts))
    n, hkv, d = len(counts), 2, 128
    lens = [x + int(rng.integers(0, 40)) for x in counts]
    c = Cache(rng, lens, hkv, d, 16, fmt, mode)
    c.device(mbd)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = int(cu[-1]) + padding
    k, v = bits(rng, total, hkv * d), bits(rng, total, hkv * d)
    positions = rng.integers(0, 1 << 30, total).astype(np.int32)
    given = n % 2 == 1
    mbd.device_error_flags(clear=True)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, n, total, up(cu),
                        up(positions) if given else None)
    torch.cuda.synchronize()
    for b, x in enumerate(counts):
        if x:
            at = slice(cu[b], cu[b + 1])
            c.store(b, np.arange(lens[b] - x, lens[b]), k[at].reshape(x, hkv, d), v[at].reshape(x, hkv, d),
                    positions[at] if given else None)
    c.check_equal("append")
    assert mbd.device_error_flags() == 0


def test_append_without_weight_and_position(mbd):
    rng = np.random.default_rng(3)
    c = Cache(rng, [4, 9], 2, 64, 4, "bf16", meta=False)
    c.device(mbd)
    k, v = bits(rng, 2, 128), bits(rng, 2, 128)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 2, 2)
    torch.cuda.synchronize()
    for b in range(2):
        c.store(b, [c.lens[b] - 1], k[b].reshape(1, 2, 64), v[b].reshape(1, 2, 64))
    c.check_equal("append")


def test_append_bad_indices_are_reported_and_dropped(mbd):
    """A page outside the pool, a length past the table or of 0 with a new token: the error bit, and nothing stored."""
    rng = np.random.default_rng(4)
    c = Cache(rng, [20, 20, 20, 20], 2, 64, 16, "bf16")
    c.device(mbd)
    c.table_d.view(4, -1)[0, 1] = c.n_pages
    c.lens_d[1], c.lens_d[2] = 0, c.width * 16 + 1
    k, v = bits(rng, 4, 128), bits(rng, 4, 128)
    mbd.device_error_flags(clear=True)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, 4, 4)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    c.store(3, [19], k[3].reshape(1, 2, 64), v[3].reshape(1, 2, 64))
    c.table[0, 1] = c.n_pages
    c.lens[1], c.lens[2] = 0, c.width * 16 + 1
    c.check_equal("append")


# ------------------------------------------------------------------------------------------------ eviction

def run_evict(mbd, c, budget, recent):
    new = Guarded(torch, len(c.lens), torch.int32)
    mbd.kv_cache_evict(c.c, new.view, c.lens_d, c.table_d, c.width, len(c.lens), budget, recent)
    torch.cuda.synchronize()
    new.check_guards("new lengths")
    return new.numpy(np.int32)


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("budget,recent", [(0, 0), (1, 0), (1, 1), (17, 5), (64, 64), (100, 0), (333, 32), (1000, 10)])
def test_evict(mbd, budget, recent, fmt, mode):
    rng = np.random.default_rng(budget)
    c = Cache(rng, [0, 1, 18, 64, 65, 101, 334, 700], 2, 64, 16, fmt, mode, gap=32)
    for b, length in enumerate(c.lens):                   # positions in any order; weights with ties, NaN, zeros of both
        if length:                                        # signs, infinities
            p, _, s = c.at(b, np.arange(length))
            for h in range(2):
                c.position[p, h, s] = rng.permutation(length) * 3
                w = rng.integers(0, 12, length).astype(np.float32) / 4
                w[rng.random(length) < 0.05] = np.nan
                w[rng.random(length) < 0.05] = -0.0
                w[rng.random(length) < 0.02] = np.inf
                c.weight[p, h, s] = w
    c.device(mbd)
    mbd.device_error_flags(clear=True)
    got = run_evict(mbd, c, budget, recent)
    np.testing.assert_array_equal(got, c.evict(budget, recent))
    c.check_equal("evict")
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("n,length,hkv,d,page,budget", [(1, 70000, 1, 64, 64, 30000), (1, 5000, 2, 128, 16, 4999),
                                                        (40, 900, 8, 64, 32, 300), (3, 3000, 1, 256, 128, 1)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_shapes(mbd, n, length, hkv, d, page, budget, ties):
    """Rows over clusters of every size; all weights equal, where the lowest slots stay."""
    rng = np.random.default_rng(length)
    lens = np.full(n, length) if n == 1 else rng.integers(length // 2, length + 1, n)
    c = Cache(rng, lens, hkv, d, page, "fp8", "dynamic")
    if ties:
        c.weight[~np.isnan(c.weight)] = 0.25
    c.device(mbd)
    np.testing.assert_array_equal(run_evict(mbd, c, budget, budget // 8), c.evict(budget, budget // 8))
    c.check_equal("evict")


@pytest.mark.parametrize("page", [1, 2, 4, 8])
@pytest.mark.parametrize("length", [1, 3, 33, 4501])
def test_evict_small_pages_and_odd_capacities(mbd, page, length):
    """Tables of any width over the smallest pages: a row's capacity may be odd."""
    rng = np.random.default_rng(page + length)
    c = Cache(rng, [length, length // 2], 3, 64, page, "bf16", width=-(-length // page) | 1)
    c.device(mbd)
    budget = length // 3
    np.testing.assert_array_equal(run_evict(mbd, c, budget, budget // 2), c.evict(budget, budget // 2))
    c.check_equal("evict")


def test_evict_the_longest(mbd):
    """As many slots as the entry point takes: the largest shares of the largest cluster."""
    rng = np.random.default_rng(15)
    length = 425984
    c = Cache(rng, [length], 1, 64, 4096, "fp8")
    c.device(mbd)
    np.testing.assert_array_equal(run_evict(mbd, c, 200001, 777), c.evict(200001, 777))
    c.check_equal("evict")


def test_evict_captured(mbd):
    """A captured eviction over a cluster of the largest size, replayed on a fresh cache each time."""
    rng = np.random.default_rng(16)
    c = Cache(rng, [40000], 1, 64, 64, "fp8", "dynamic")
    c.device(mbd)
    start = {n: g.raw.clone() for n, g in c.g.items() if g is not None}
    new = torch.empty(1, dtype=torch.int32, device="cuda")
    call = lambda: mbd.kv_cache_evict(c.c, new, c.lens_d, c.table_d, c.width, 1, 9000, 100)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    c.evict(9000, 100)
    for _ in range(2):
        for n, raw in start.items():
            c.g[n].raw.copy_(raw)
        new.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert int(new) == 9000
        c.check_equal("evict")


def test_evict_bad_pages_are_reported(mbd):
    """Slots on a page outside the pool go first, and nothing is read or written there."""
    rng = np.random.default_rng(12)
    c = Cache(rng, [96, 96], 1, 64, 16, "bf16")
    c.device(mbd)
    c.table_d.view(2, -1)[0, 2] = 1 << 29
    before = {n: g.view.clone() for n, g in c.g.items() if g is not None}
    mbd.device_error_flags(clear=True)
    got = run_evict(mbd, c, 40, 8)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    assert list(got) == [40, 40]
    pages = torch.from_numpy(c.table[0][c.table[0] >= 0].astype(np.int64)).cuda()
    other = torch.ones(c.n_pages, dtype=torch.bool, device="cuda")
    other[pages] = False
    other[torch.from_numpy(c.table[1].astype(np.int64)).cuda()] = False
    for name in ("k", "v", "weight", "position"):          # pages of neither sequence, and the one taken out, as before
        x, y = (t.view(torch.uint8).view(c.n_pages, -1) for t in (c.g[name].view, before[name]))
        assert torch.equal(x[other], y[other]) and torch.equal(x[c.table[0, 2]], y[c.table[0, 2]])


# ------------------------------------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,mode", STORES)
def test_decode_with_eviction(mbd, fmt, mode):
    """A prompt, then decode steps (append, attention with accumulation), an eviction whenever the cache is full: the
    GPU's cache follows the reference step by step, on one stream without a synchronisation inside a step."""
    rng = np.random.default_rng(20)
    n, hkv, hq, d, page, budget, full = 3, 2, 8, 64, 8, 24, 40
    c = Cache(rng, [full] * n, hkv, d, page, fmt, mode, fill=False)
    prompts = np.array([30, 12, 33], np.int32)
    c.lens = prompts.copy()
    c.device(mbd)
    cu = np.concatenate([[0], np.cumsum(prompts)]).astype(np.int32)
    k, v = bits(rng, cu[-1], hkv * d), bits(rng, cu[-1], hkv * d)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, n, int(cu[-1]), up(cu))
    for b in range(n):
        at = slice(cu[b], cu[b + 1])
        c.store(b, np.arange(prompts[b]), k[at].reshape(-1, hkv, d), v[at].reshape(-1, hkv, d))
    position = torch.from_numpy(prompts).cuda()
    new_lens = torch.empty(n, dtype=torch.int32, device="cuda")
    total, evictions = prompts.copy(), 0
    width = (hq + 2 * hkv) * d
    for step in range(24):
        qkv = bits(rng, n, width)
        x = up(qkv)
        c.lens_d += 1
        c.lens += 1
        kn, vn = x[:, hq * d:], x[:, (hq + hkv) * d:]
        nb = mbd.paged_attention_workspace_bytes(c.c, c.width, n, hq, True)
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
        out, lse = torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hq, device="cuda")
        torch.cuda.synchronize()
        mbd.kv_cache_append(c.c, kn, vn, width, c.table_d, c.width, c.lens_d, n, n, None, position)
        mbd.paged_attention_decode(out, x, width, c.c, c.table_d, c.width, c.lens_d, n, hq, d ** -0.5, 0, lse, True, ws, nb)
        for b in range(n):
            c.store(b, [c.lens[b] - 1], qkv[b, hq * d:(hq + hkv) * d].reshape(1, hkv, d),
                    qkv[b, (hq + hkv) * d:].reshape(1, hkv, d), [total[b]])
        want = c.attend(qkv[:, :hq * d].copy(), hq, d ** -0.5, 0, True)
        evict = int(c.lens.max()) == full
        if not evict:
            torch.cuda.synchronize()
        w = c.g["weight"].numpy(np.float32).reshape(c.weight.shape)
        live = ~np.isnan(c.weight)
        check_close(w[live], want[4][live], want[5][live], f"step {step} weight")
        c.weight[live] = w[live]                          # the choice of the eviction is on these very weights
        if evict:
            mbd.kv_cache_evict(c.c, new_lens, c.lens_d, c.table_d, c.width, n, budget, 6)
            c.lens_d.copy_(new_lens)
            c.lens = c.evict(budget, 6)
            evictions += 1
        position += 1
        total += 1
        check_close(out.float().cpu().numpy().reshape(n, hq, d), want[0], want[2], f"step {step} out")
        check_close(lse.cpu().numpy(), want[1], want[3], f"step {step} lse")
        c.check_equal(f"step {step}")
    assert evictions >= 1


def test_captured_steps_share_a_workspace(mbd):
    """Two captured graphs of a step (append, attention with accumulation) over one workspace, replayed in turn while the
    lengths on the device grow: the same bits as the calls made one by one."""
    rng = np.random.default_rng(30)
    n, hkv, hq, d, page, steps = 4, 2, 8, 128, 16, 12
    width = (hq + 2 * hkv) * d
    rows = [up(bits(rng, n, width)) for _ in range(steps)]
    seed = rng.integers(1 << 30)

    def fresh():
        r = np.random.default_rng(seed)
        c = Cache(r, [100, 1, 64, 333], hkv, d, page, "fp8", "dynamic", width=25, spare=30)
        for b in range(n):                                # pages for the tokens to come
            used = -(-int(c.lens[b]) // page)
            free = [p for p in range(c.n_pages) if p not in set(c.table[c.table >= 0]) and p < c.n_pages]
            c.table[b, used:used + 1] = free[0]
        c.table[(c.table < 0) | (c.table >= c.n_pages)] = -1
        c.device(mbd)
        return c

    def call(c, x, out, ws, nb):
        mbd.kv_cache_append(c.c, x[:, hq * d:], x[:, (hq + hkv) * d:], width, c.table_d, c.width, c.lens_d, n, n)
        mbd.paged_attention_decode(out, x, width, c.c, c.table_d, c.width, c.lens_d, n, hq, d ** -0.5, 0, None, True, ws, nb)

    a, b = fresh(), fresh()
    nb = mbd.paged_attention_workspace_bytes(a.c, a.width, n, hq, True)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    outs = [torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    want = []
    for x in rows:
        a.lens_d += 1
        call(a, x, outs[0], ws, nb)
        want.append(outs[0].clone())
    torch.cuda.synchronize()
    ins, graphs = [torch.empty_like(rows[0]) for _ in range(2)], []
    ws.fill_(0xFF)
    torch.cuda.synchronize()
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(b, ins[i], outs[i], ws, nb)
        graphs.append(g)
    for s, x in enumerate(rows):
        b.lens_d += 1
        ins[s % 2].copy_(x)
        graphs[s % 2].replay()
        assert torch.equal(outs[s % 2], want[s]), f"step {s}"
    torch.cuda.synchronize()
    for name in ("k", "v", "ks", "vs", "weight", "position"):
        assert torch.equal(a.g[name].raw, b.g[name].raw), name
