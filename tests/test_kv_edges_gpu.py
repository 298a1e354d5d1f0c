"""The key-value cache's entry points on the GPU at the edges of what their documentation allows: values that are not
finite, calls from several host threads, pages outside the pool, the largest sizes. Tolerances are those that
oracle/kv_cache.py derives, on the inputs without the planted values."""
import numpy as np
import pytest

import workloads as wl
from oracle import kv_cache as ref
from oracle.kv_cache import check_close
from tests.test_kv_gpu import STORES, Cache, bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN16, INF16 = 0x7FC0, 0x7F80


def attend(mbd, c, q, hq, scale, accumulate=True):
    """out [n, hq, d], lse [n, hq] and the weights after the call."""
    n = len(c.lens)
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, n, hq, accumulate)
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.zeros(n, hq * c.d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, hq, device="cuda")
    mbd.device_error_flags(clear=True)
    mbd.paged_attention_decode(out, up(q), 0, c.c, c.table_d, c.width, c.lens_d, n, hq, scale, 0, lse, accumulate, ws, nb)
    torch.cuda.synchronize()
    assert mbd.device_error_flags() == 0
    w = c.g["weight"].numpy(np.float32).reshape(c.weight.shape)
    return out.float().cpu().numpy().reshape(n, hq, c.d), lse.cpu().numpy(), w


# Lengths whose last key is alone in its warp's step, whatever the step (16, 32 or 64 keys); a single key; a sequence
# that is cut into many parts.
LONELY = [1, 49, 65, 129, 20033]


def check_planted(c, want, got, heads, hq, nan_lse=True):
    """The query heads in `heads` are NaN in out (and lse); the rest is as the reference without the plant."""
    out, lse, w = got
    sick = np.zeros(hq, bool)
    sick[heads] = True
    assert np.isnan(out[:, sick]).all()
    check_close(out[:, ~sick], want[0][:, ~sick], want[2][:, ~sick], "out of the other heads")
    if nan_lse:
        assert np.isnan(lse[:, sick]).all()
    whole = ~sick if nan_lse else np.ones(hq, bool)
    check_close(lse[:, whole], want[1][:, whole], want[3][:, whole], "lse")
    group = hq // c.hkv
    for h in range(c.hkv):
        live = ~np.isnan(c.weight[:, h])
        if sick[h * group:(h + 1) * group].any():
            if nan_lse:
                assert np.isnan(w[:, h]).all()
                continue
        check_close(w[:, h][live], want[4][:, h][live], want[5][:, h][live], "weights")


@pytest.mark.parametrize("fmt,mode,where", [(*store, where) for store in STORES
                                            for where in ("query", "key", "k_scale", "v_scale")
                                            if store[1] == "dynamic" or "scale" not in where])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 2, 128), (18, 2, 128), (2, 2, 256)])
def test_attention_nan_reaches_its_heads(mbd, fmt, mode, hq, hkv, d, where):
    """A NaN in one head's query, in the last key, or in a scale of the last token gives NaN to the query heads that read
    it, wherever that key lies, and to no others."""
    rng = np.random.default_rng(d + hq)
    c = Cache(rng, LONELY, hkv, d, 16, fmt, mode)
    q = bits(rng, len(LONELY), hq * d)
    want = c.attend(q, hq, d ** -0.5, 0, True)
    group, bad = hq // hkv, hkv - 1
    heads = list(range(bad * group, hq))
    for b, length in enumerate(c.lens):
        p, _, s = c.at(b, [length - 1])
        if where == "query":
            heads = [hq - 1]
            q[b, (hq - 1) * d + 5] = NAN16
        elif where == "key":
            c.view(c.k_raw)[p[0], bad, s[0], 7] = NAN16 if fmt == "bf16" else 0x7F
        else:
            (c.ks if where == "k_scale" else c.vs)[p[0], bad, s[0]] = np.nan
    c.device(mbd)
    check_planted(c, want, attend(mbd, c, q, hq, d ** -0.5), heads, hq, nan_lse=where != "v_scale")


def test_attention_nan_value_under_a_scale_of_zero(mbd):
    """A NaN code whose token has a zero scale: NaN in that element of the output, nothing in the others."""
    rng = np.random.default_rng(3)
    hq = hkv = 2
    c = Cache(rng, LONELY, hkv, 64, 16, "fp8", "dynamic")
    for b, length in enumerate(c.lens):
        p, _, s = c.at(b, [length - 1])
        c.vs[p[0], :, s[0]] = 0
        c.view(c.v_raw)[p[0], :, s[0]] = 0
    q = bits(rng, len(LONELY), hq * 64)
    want = c.attend(q, hq, 0.125, 0, True)
    for b, length in enumerate(c.lens):
        p, _, s = c.at(b, [length - 1])
        c.view(c.v_raw)[p[0], 1, s[0], 9] = 0x7F
    c.device(mbd)
    out, lse, _ = attend(mbd, c, q, hq, 0.125)
    nan = np.zeros(out.shape, bool)
    nan[:, 1, 9] = True
    np.testing.assert_array_equal(np.isnan(out), nan)
    check_close(np.where(nan, 0, out), np.where(nan, 0, want[0]), want[2], "out")
    check_close(lse, want[1], want[3], "lse")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (4, 2, 128), (18, 2, 128), (2, 2, 256)])
def test_attention_infinite_values(mbd, hq, hkv, d, accumulate):
    """An infinite value comes out as the infinity of its sign, whatever its probability (of a single key: exactly 1, of
    equal keys: a power of two), and leaves the other elements alone."""
    rng = np.random.default_rng(d)
    c = Cache(rng, [1, 2, 64, 100, 4096, 20033], hkv, d, 16, "bf16")
    for b in (1, 2, 4):                                   # equal keys: probabilities 1/2, 1/64, 1/4096
        p, _, s = c.at(b, np.arange(c.lens[b]))
        c.view(c.k_raw)[p, :, s] = wl.f32_to_bf16_bits(np.ones(d, np.float32))
    at = [(b, int(rng.integers(0, n))) for b, n in enumerate(c.lens)]
    for b, slot in at:                                    # (the reference sees zeros there)
        p, _, s = c.at(b, [slot])
        c.view(c.v_raw)[p[0], :, s[0], 3] = c.view(c.v_raw)[p[0], :, s[0], d - 2] = 0
    q = bits(rng, len(c.lens), hq * d)
    want = c.attend(q, hq, d ** -0.5, 0, True)
    for b, slot in at:
        p, _, s = c.at(b, [slot])
        c.view(c.v_raw)[p[0], :, s[0], 3], c.view(c.v_raw)[p[0], :, s[0], d - 2] = INF16, INF16 | 0x8000
    c.device(mbd)
    out, lse, w = attend(mbd, c, q, hq, d ** -0.5, accumulate)
    assert np.isposinf(out[..., 3]).all() and np.isneginf(out[..., d - 2]).all()
    keep = np.delete(np.arange(d), [3, d - 2])
    check_close(out[..., keep], want[0][..., keep], want[2][..., keep], "out")
    check_close(lse, want[1], want[3], "lse")
    if accumulate:
        live = ~np.isnan(c.weight)
        check_close(w[live], want[4][live], want[5][live], "weights")


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (18, 2, 128), (2, 2, 256)])
def test_attention_with_a_logit_of_infinity(mbd, hq, hkv, d):
    """An infinite key under positive queries leaves no softmax: NaN for the heads that read it, and no others."""
    rng = np.random.default_rng(hq)
    c = Cache(rng, LONELY, hkv, d, 16, "bf16")
    q = wl.f32_to_bf16_bits(np.abs(wl.bf16_bits_to_f32(bits(rng, len(LONELY), hq * d))) + np.float32(2 ** -10))
    want = c.attend(q, hq, d ** -0.5, 0, True)
    for b, length in enumerate(c.lens):
        p, _, s = c.at(b, [length // 2])
        c.view(c.k_raw)[p[0], 1, s[0], 3] = INF16
    c.device(mbd)
    check_planted(c, want, attend(mbd, c, q, hq, d ** -0.5), list(range(hq // hkv, hq)), hq)


@pytest.mark.parametrize("where", ["last", "first", "all"])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (18, 2, 128), (2, 2, 256)])
def test_attention_infinite_values_without_weight(mbd, hq, hkv, d, where):
    """An infinite value whose logit is -inf: zero times infinity, NaN in that element wherever the key lies (alone in
    its warp, or with every logit -inf), and nothing in the others."""
    rng = np.random.default_rng(hq)
    c = Cache(rng, LONELY, hkv, d, 16, "bf16")
    q = wl.f32_to_bf16_bits(np.abs(wl.bf16_bits_to_f32(bits(rng, len(LONELY), hq * d))) + np.float32(2 ** -10))
    slots = [np.arange(n) if where == "all" else np.array([n - 1 if where == "last" else 0]) for n in c.lens]
    alone = np.array([len(at) == n for at, n in zip(slots, c.lens)])
    for b, at in enumerate(slots):
        p, _, s = c.at(b, at)
        c.view(c.k_raw)[p, :, s, 3] = INF16 | 0x8000
        c.view(c.v_raw)[p[-1], :, s[-1], 5] = INF16
    c.device(mbd)
    out, lse, w = attend(mbd, c, q, hq, d ** -0.5)
    assert np.isnan(out[..., 5]).all()
    keep = np.delete(np.arange(d), 5)
    assert not out[alone][..., keep].any() and np.isneginf(lse[alone]).all()
    group = hq // hkv
    for b in np.flatnonzero(~alone):
        k, v = c.rows(b, np.setdiff1d(np.arange(c.lens[b]), slots[b]))
        x = np.einsum("hgd,hld->hgl", wl.bf16_bits_to_f32(q[b]).astype(np.float64).reshape(hkv, group, d), k) * d ** -0.5
        pr = np.exp(x - x.max(-1, keepdims=True))
        pr /= pr.sum(-1, keepdims=True)
        a = np.einsum("hgl,hld->hgd", pr, np.abs(v)).reshape(hq, d)
        o = np.einsum("hgl,hld->hgd", pr, v).reshape(hq, d)
        size = np.abs(wl.bf16_bits_to_f32(q[b])).reshape(hq, d).sum(-1).max() * np.abs(k).max() * d ** -0.5
        tol = a * (2 * (d * 2.0 ** -23 + 2.0 ** -22) * size + 2.0 ** -16 + 2 * (k.shape[1] / 32 + 64) * 2.0 ** -23) + 2.0 ** -8 * np.abs(o)
        check_close(out[b][:, keep], o[:, keep], tol[:, keep], "out")


@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (18, 2, 128), (2, 2, 256), (260, 2, 64)])
def test_attention_with_logits_of_minus_infinity(mbd, hq, hkv, d):
    """Keys of -inf under positive queries have no weight; where all of a head's keys are such, it gives zeros and -inf
    and adds nothing to the weights."""
    rng = np.random.default_rng(d)
    c = Cache(rng, [1, 50, 20033, 300], hkv, d, 16, "bf16")
    q = wl.f32_to_bf16_bits(np.abs(wl.bf16_bits_to_f32(bits(rng, 4, hq * d))) + np.float32(2 ** -10))
    want = [x.copy() for x in c.attend(q, hq, d ** -0.5, 0, True)]
    group = hq // hkv
    for b in range(3):                                    # key-value head 0 of the first three
        p, _, s = c.at(b, np.arange(c.lens[b]))
        c.view(c.k_raw)[p, 0, s, 11] = INF16 | 0x8000
        want[0][b, :group], want[1][b, :group] = 0, -np.inf
        want[4][p, 0, s] = c.weight[p, 0, s]
    half = Cache.at(c, 3, np.arange(0, 300, 2))           # every other key of the last: the reference on the others
    c.view(c.k_raw)[half[0], 0, half[2], 11] = INF16 | 0x8000
    k, v = (x[0] for x in c.rows(3, np.arange(1, 300, 2)))
    qd = wl.bf16_bits_to_f32(q[3]).astype(np.float64).reshape(hq, d)[:group]
    x = qd @ k.T * d ** -0.5
    m = x.max(-1, keepdims=True)
    pr = np.exp(x - m) / np.exp(x - m).sum(-1, keepdims=True)
    want[0][3, :group], want[1][3, :group] = pr @ v, (m + np.log(np.exp(x - m).sum(-1, keepdims=True)))[:, 0]
    dx = (d * 2.0 ** -23 + 2.0 ** -22) * (np.abs(qd) @ np.abs(k).T * d ** -0.5).max()
    dp = 2 * dx + (150 / 32 + 8) * 2.0 ** -23             # as oracle/kv_cache.py derives them, over all of the group
    want[2][3, :group] = pr @ np.abs(v) * (dp + 2.0 ** -16 + (150 / 32 + 64) * 2.0 ** -23) + 2.0 ** -8 * np.abs(pr @ v)
    want[3][3, :group] = dp + 2.0 ** -22 * np.abs(want[1][3, :group])
    p, _, s = c.at(3, np.arange(1, 300, 2))
    want[4][p, 0, s] = c.weight[p, 0, s] + pr.sum(0)
    want[5][p, 0, s] = pr.sum(0) * dp + 2.0 ** -23 * want[4][p, 0, s]
    want[4][half[0], 0, half[2]] = c.weight[half[0], 0, half[2]]
    c.device(mbd)
    out, lse, w = attend(mbd, c, q, hq, d ** -0.5)
    check_close(out, want[0], want[2], "out")
    check_close(lse, want[1], want[3], "lse")
    live = ~np.isnan(c.weight)
    check_close(w[live], want[4][live], want[5][live], "weights")


@pytest.mark.parametrize("hq,d", [(1 << 23, 256), (1 << 24, 128), ((1 << 23) + 8, 256)])
def test_attention_of_an_empty_sequence_with_the_most_heads(mbd, hq, d):
    """Rows of 2^31 elements and more, all of which have to become zero."""
    rng = np.random.default_rng(1)
    c = Cache(rng, [0], 1, d, 16, "bf16")
    c.device(mbd)
    out = torch.full((hq * d,), 0x3F80, dtype=torch.int16, device="cuda")
    q, lse = torch.empty(hq * d, dtype=torch.int16, device="cuda"), torch.zeros(hq, device="cuda")
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, 1, hq)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    mbd.paged_attention_decode(out, q, 0, c.c, c.table_d, c.width, c.lens_d, 1, hq, 0.1, 0, lse, False, ws, nb)
    assert not bool(out.view(torch.int64).any()) and bool(torch.isneginf(lse).all())


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("budget,recent,bad", [(40, 8, {2}), (40, 8, {0, 1, 2}), (40, 40, {1}), (70, 5, {1, 3, 5}),
                                               (40, 0, {3, 4, 5}), (20, 3, {0, 1, 2, 3, 4, 5}), (90, 0, {0, 2, 4, 5})])
def test_evict_around_bad_pages(mbd, fmt, mode, budget, recent, bad):
    """Slots on pages outside the pool take up their places before the budget; every row that is kept arrives, the best
    ones, and the other sequence is evicted as ever."""
    rng = np.random.default_rng(budget + len(bad))
    c = Cache(rng, [96, 96], 2, 64, 16, fmt, mode)
    for b in range(2):
        p, _, s = c.at(b, np.arange(96))
        for h in range(2):
            c.position[p, h, s] = rng.permutation(96)
            c.weight[p, h, s] = rng.integers(0, 8, 96).astype(np.float32) / 4
            c.weight[p[rng.integers(0, 96)], h, s[3]] = np.nan
    for i in bad:
        c.table[0, i] = (-1, c.n_pages, 1 << 29)[i % 3]
    c.device(mbd)
    new = torch.zeros(2, dtype=torch.int32, device="cuda")
    mbd.device_error_flags(clear=True)
    mbd.kv_cache_evict(c.c, new, c.lens_d, c.table_d, c.width, 2, budget, recent)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    np.testing.assert_array_equal(new.cpu().numpy(), c.evict(budget, recent))
    c.check_equal("evict")


def test_window_counts_slots_also_after_an_eviction(mbd):
    """The window is the last slots as they lie, whatever positions an eviction left there; without one, the order of
    the slots decides nothing."""
    rng = np.random.default_rng(21)
    hq, hkv, d, n = 4, 2, 64, 3
    c = Cache(rng, [300, 200, 64], hkv, d, 16, "bf16")
    for b, length in enumerate(c.lens):
        p, _, s = c.at(b, np.arange(length))
        c.position[p, :, s] = np.arange(length)[:, None]
    c.device(mbd)
    new = torch.zeros(n, dtype=torch.int32, device="cuda")
    mbd.kv_cache_evict(c.c, new, c.lens_d, c.table_d, c.width, n, 100, 20)
    c.lens = c.evict(100, 20)
    c.lens_d.copy_(new)
    c.check_equal("evict")
    p, _, s = c.at(0, np.arange(100))
    assert (np.diff(c.position[p, 0, s].astype(np.int64)) < 0).any()
    q = bits(rng, n, hq * d)
    nb = mbd.paged_attention_workspace_bytes(c.c, c.width, n, hq)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    for window in (0, 20):
        out, lse = torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, hq, device="cuda")
        mbd.paged_attention_decode(out, up(q), 0, c.c, c.table_d, c.width, c.lens_d, n, hq, 0.125, window, lse, False, ws, nb)
        want = c.attend(q, hq, 0.125, window)
        check_close(out.float().cpu().numpy().reshape(n, hq, d), want[0], want[2], "out")
        check_close(lse.cpu().numpy(), want[1], want[3], "lse")


@pytest.mark.parametrize("fmt,mode", STORES)
@pytest.mark.parametrize("hkv,d", [(3, 64), (5, 128), (7, 64), (3, 256), (1, 64), (11, 128), (17, 256)])
def test_append_prompts_of_any_layout(mbd, hkv, d, fmt, mode):
    """Many tokens of head layouts whose rows are no power of two of vectors, several tokens to a CTA, the last CTA with
    fewer: the quotients that find a vector's token and head."""
    rng = np.random.default_rng(hkv * d)
    counts = [708, 0, 2, 40]
    lens = [x + 5 * i for i, x in enumerate(counts)]
    c = Cache(rng, lens, hkv, d, 8, fmt, mode)
    c.device(mbd)
    cu = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    total = int(cu[-1]) + 1                               # 751, a prime; one row is padding
    k, v = bits(rng, total, hkv * d), bits(rng, total, hkv * d)
    mbd.device_error_flags(clear=True)
    mbd.kv_cache_append(c.c, up(k), up(v), 0, c.table_d, c.width, c.lens_d, len(counts), total, up(cu))
    torch.cuda.synchronize()
    for b, x in enumerate(counts):
        if x:
            at = slice(cu[b], cu[b + 1])
            c.store(b, np.arange(lens[b] - x, lens[b]), k[at].reshape(x, hkv, d), v[at].reshape(x, hkv, d))
    c.check_equal("append")
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("fmt,mode", STORES)
def test_attention_of_small_probabilities(mbd, fmt, mode):
    """Probabilities of 2^-16 to 2^-36 beside one of 1, each with a value in an element of its own: off by half a bf16 step
    (2^-8), by the rounding before the product (2^-16, 2^-11 in FP8) and by the fp32 sums and exponentials (a hundred times
    2^-23), in FP8 besides by 2^-31 of the largest value."""
    powers = np.array([0, 16, 18, 20, 22, 24, 26, 28, 30, 32, 36])
    d, n = 64, len(powers)
    c = Cache(np.random.default_rng(0), [n], 1, d, 16, fmt, mode, fill=False)
    kx, vx = np.zeros((n, 1, d)), np.zeros((n, 1, d))
    kx[:, 0, 0] = -powers                                 # exact in E4M3
    vx[1:, 0, 1:n] = 448 * np.eye(n - 1)
    p, _, s = c.at(0, np.arange(n))
    for raw, scales, x in ((c.k_raw, c.ks, kx), (c.v_raw, c.vs, vx)):
        if fmt == "fp8":
            c.view(raw)[p, :, s] = ref.e4m3_codes(x)
            scales[(p, slice(None), s) if mode == "dynamic" else 0] = 1
        else:
            c.view(raw)[p, :, s] = wl.f32_to_bf16_bits(x.astype(np.float32))
    c.weight[p, :, s] = 0
    q = np.zeros((1, d), np.uint16)
    q[0, 0] = 0x3F80
    scale = float(np.float32(np.log(2)))
    c.device(mbd)
    out, lse, w = attend(mbd, c, q, 1, scale)
    pr = np.exp(-powers * scale)
    pr /= pr.sum()
    want = np.zeros(d)
    want[1:n] = pr[1:] * 448
    tol = want * (2.0 ** -8 + (2.0 ** -11 if fmt == "fp8" else 2.0 ** -16) + 100 * 2.0 ** -23)
    check_close(out[0, 0], want, tol + (448 * 2.0 ** -31 if fmt == "fp8" else 0), "out")
    check_close(w[p, 0, s], pr, pr * 100 * 2.0 ** -23, "weights")
