"""The attention of whole prompts on the GPU against the NumPy reference, within the tolerances that oracle/step.py derives. Rows of
the stacked projection that no sequence owns hold NaN, guard bands lie around the outputs."""
import numpy as np
import pytest

import workloads as wl
from oracle import step as ref
from oracle.kv_cache import check_close
from tests.parity import Guarded
from tests.test_kv_gpu import bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NAN = 0x7FC1


def make(rng, lens, hq, hkv, d, pad=0, gap=0, sigma=2.0):
    """(stacked projection as bits, offsets): `pad` rows behind the last sequence hold NaN."""
    rows = int(np.sum(lens))
    width = (hq + 2 * hkv) * d + gap
    qkv = np.full((rows + pad, width), NAN, np.uint16)
    qkv[:rows, :hq * d] = bits(rng, rows, hq * d, sigma=sigma)
    qkv[:rows, hq * d:(hq + 2 * hkv) * d] = bits(rng, rows, 2 * hkv * d)
    return qkv, np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def run(mbd, qkv, cu, hq, hkv, d, scale, window=0, lse=True, stream=None):
    n = len(qkv)
    out, lse_g = Guarded(torch, n * hq * d, torch.int16), Guarded(torch, n * hq, torch.float32)
    x = up(qkv)
    cu_d = up(cu)
    torch.cuda.synchronize()
    mbd.prompt_attention(out.view, x, qkv.shape[1], x[:, hq * d:], x[:, (hq + hkv) * d:], qkv.shape[1], cu_d, len(cu) - 1, n, hq,
                         hkv, d, scale, window, lse_g.view if lse else None, stream)
    torch.cuda.synchronize()
    out.check_guards("out")
    lse_g.check_guards("lse")
    return out.numpy(np.uint16).reshape(n, hq, d), lse_g.numpy(np.float32).reshape(n, hq)


def check(mbd, qkv, cu, hq, hkv, d, scale=None, window=0, lse=True, **kw):
    scale = d ** -0.5 if scale is None else scale
    mbd.device_error_flags(clear=True)
    out, got_lse = run(mbd, qkv, cu, hq, hkv, d, scale, window, lse, **kw)
    rows = int(cu[-1])
    parts = [np.ascontiguousarray(qkv[:rows, a:b]) for a, b in ((0, hq * d), (hq * d, (hq + hkv) * d), ((hq + hkv) * d, (hq + 2 * hkv) * d))]
    want = ref.prompt(*parts, cu, hq, hkv, d, scale, window)
    check_close(wl.bf16_bits_to_f32(out[:rows]), want[0], want[2], "out")
    if lse:
        check_close(got_lse[:rows], want[1], want[3], "lse")
    else:
        assert (got_lse.view(np.uint32) == 0x5A5A5A5A).all()
    assert (out[rows:] == 0x5A5A).all(), "rows behind the last sequence"
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("d", [128, 64, 256])
@pytest.mark.parametrize("length", [1, 2, 127, 128, 129, 256, 300])
def test_one_prompt(mbd, length, d):
    rng = np.random.default_rng(length)
    check(mbd, *make(rng, [length], 2, 1, d), 2, 1, d)


@pytest.mark.parametrize("hq,hkv,d", [(12, 2, 128), (8, 8, 128), (4, 4, 64), (16, 1, 64), (9, 1, 128), (6, 2, 64), (64, 1, 128),
                                      (3, 3, 256), (8, 2, 256), (1, 1, 128), (1, 1, 64), (10, 2, 128)])
def test_head_layouts(mbd, hq, hkv, d):
    rng = np.random.default_rng(hq)
    check(mbd, *make(rng, [37, 0, 1, 200, 129], hq, hkv, d, pad=70, gap=64), hq, hkv, d)


@pytest.mark.parametrize("d,hq,hkv", [(128, 2, 1), (64, 3, 3), (256, 2, 1)])
def test_many_lengths(mbd, d, hq, hkv):
    """Lengths around the tiles' and blocks' sizes, in any order, empty sequences first, last and between."""
    rng = np.random.default_rng(d)
    lens = [0, 1, 2, 63, 64, 65, 0, 0, 127, 128, 129, 255, 256, 257, 383, 384, 385, 700, 3, 0]
    check(mbd, *make(rng, rng.permutation(lens), hq, hkv, d, pad=3), hq, hkv, d)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 2, 2), (256, 1, 1)])
@pytest.mark.parametrize("window", [1, 2, 64, 100, 127, 128, 129, 130, 255, 256, 257, 500, 5000])
def test_window(mbd, window, d, hq, hkv):
    rng = np.random.default_rng(window)
    check(mbd, *make(rng, [1, 90, 700, 128, 400], hq, hkv, d), hq, hkv, d, window=window)


@pytest.mark.parametrize("n,hi,hq,hkv,d", [(300, 40, 2, 2, 64), (1100, 3, 2, 1, 128), (40, 300, 8, 2, 128), (1, 2500, 2, 1, 128),
                                           (2, 1500, 2, 2, 64)])
def test_shapes(mbd, n, hi, hq, hkv, d):
    rng = np.random.default_rng(n)
    check(mbd, *make(rng, rng.integers(0, hi + 1, n) if n > 2 else np.full(n, hi), hq, hkv, d), hq, hkv, d)


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-30, 3.0, -2.0])
@pytest.mark.parametrize("d", [64, 128])
def test_scales(mbd, scale, d):
    """Also of 0 (equal weights), negative, and so large that one key takes all."""
    rng = np.random.default_rng(5)
    check(mbd, *make(rng, [300, 60], 4, 2, d), 4, 2, d, scale=scale)
    check(mbd, *make(rng, [300, 60], 4, 2, d), 4, 2, d, scale=scale, window=40)


@pytest.mark.parametrize("rising", [True, False])
def test_rising_and_falling_logits(mbd, rising):
    """Logits that grow along the keys, so that every block raises the maximum, or fall, so that it stays."""
    rng = np.random.default_rng(6)
    qkv, cu = make(rng, [900], 2, 1, 128)
    step = np.linspace(0, 40, 900, dtype=np.float32)[::1 if rising else -1]
    qkv[:, :128 * 2] = wl.f32_to_bf16_bits(np.ones((900, 256), np.float32))
    qkv[:, 256:384] = wl.f32_to_bf16_bits(np.repeat(step[:, None], 128, 1))
    check(mbd, qkv, cu, 2, 1, 128)


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 3), (256, 1, 1)])
def test_masked_places_hold_anything(mbd, d, hq, hkv):
    """NaN and infinite keys and values after a row, before its window, and in other sequences change nothing."""
    rng = np.random.default_rng(7)
    lens = [150, 40, 513, 129]
    qkv, cu = make(rng, lens, hq, hkv, d, pad=20)
    odd = qkv.copy()
    kv = slice(hq * d, (hq + 2 * hkv) * d)
    for b, at in ((0, 140), (2, 300), (2, 505)):             # seen by the rows from there on (to the window's end)
        odd[cu[b] + at, kv] = rng.choice([NAN, 0x7F80, 0xFF80], odd[0, kv].shape)
    for window in (0, 50, 128):
        a, la = run(mbd, qkv, cu, hq, hkv, d, d ** -0.5, window)
        o, lo = run(mbd, odd, cu, hq, hkv, d, d ** -0.5, window)
        clean = np.ones(len(qkv), bool)
        clean[cu[-1]:] = False
        for b, at in ((0, 140), (2, 300), (2, 505)):
            clean[cu[b] + at:min(cu[b + 1], cu[b] + at + window) if window else cu[b + 1]] = False
        # the same rows; a block's product that is added by hand is summed in another order
        fa, fo = wl.bf16_bits_to_f32(a[clean]).astype(np.float64), wl.bf16_bits_to_f32(o[clean]).astype(np.float64)
        assert np.isfinite(fo).all()
        assert (np.abs(fa - fo) <= 2.0 ** -7 * np.abs(fa) + 2.0 ** -12).all()
        np.testing.assert_array_equal(la[clean], lo[clean])
        dirty = ~clean
        dirty[cu[-1]:] = False
        assert np.isnan(lo[dirty]).all()                      # a NaN or infinite key among 2 d * hkv random ones: NaN logits


@pytest.mark.parametrize("d,hq,hkv", [(128, 4, 2), (64, 3, 3), (256, 2, 1)])
@pytest.mark.parametrize("window", [0, 70])
def test_other_rows_change_no_bit(mbd, d, hq, hkv, window):
    """What lies behind a sequence's end, in padding or in the next sequence, changes no bit of its rows."""
    rng = np.random.default_rng(13)
    qkv, cu = make(rng, [300, 5, 129, 0, 200], hq, hkv, d, pad=90)
    want = None
    for fill in (0, NAN, 0x7F80, 0x4640):
        x = qkv.copy()
        x[cu[-1]:] = fill
        x[cu[1]:cu[2]] = fill                                # the second sequence
        out, lse = run(mbd, x, cu, hq, hkv, d, d ** -0.5, window)
        keep = np.ones(len(x), bool)
        keep[cu[-1]:] = keep[cu[1]:cu[2]] = False
        if want is None:
            want = out[keep], lse[keep]
        np.testing.assert_array_equal(out[keep], want[0])
        np.testing.assert_array_equal(lse[keep], want[1])
        alone, alone_lse = run(mbd, np.ascontiguousarray(x[:300]), cu[:2], hq, hkv, d, d ** -0.5, window)
        np.testing.assert_array_equal(alone, out[:300])
        np.testing.assert_array_equal(alone_lse, lse[:300])


def test_infinite_values_in_view(mbd):
    """An infinity where one sign is in view, NaN where both are or a NaN is, in the columns concerned alone."""
    rng = np.random.default_rng(8)
    hq, hkv, d = 4, 2, 128
    qkv, cu = make(rng, [200, 300], hq, hkv, d, sigma=0.5)
    v0 = (hq + hkv) * d
    qkv[30, v0 + 5] = 0x7F80
    qkv[60, v0 + 5] = 0xFF80
    qkv[200 + 10, v0 + 128 + 7] = NAN
    qkv[200 + 140, v0 + 128 + 100] = 0xFF80
    out, _ = run(mbd, qkv, cu, hq, hkv, d, 0.05)
    f = wl.bf16_bits_to_f32(out)
    assert np.isfinite(f[:30]).all() and (f[30:60, :2, 5] == np.inf).all() and np.isnan(f[60:200, :2, 5]).all()
    assert np.isnan(f[210:, 2:, 7]).all() and (f[340:, 2:, 100] == -np.inf).all()
    f[30:200, :2, 5] = f[210:, 2:, 7] = f[340:, 2:, 100] = 0
    assert np.isfinite(f).all()


def test_infinite_logits(mbd):
    """Rows whose logits are all -inf: zeros and -inf; +inf or NaN among them: NaN."""
    qkv, cu = make(np.random.default_rng(9), [140], 2, 1, 128)
    q, k = slice(0, 256), slice(256, 384)
    qkv[:, q] = wl.f32_to_bf16_bits(np.ones((140, 256), np.float32))
    qkv[:, 256] = 0xFF80
    out, lse = run(mbd, qkv, cu, 2, 1, 128, 0.1)
    assert not (out & 0x7FFF).any() and (lse == -np.inf).all()
    qkv[50, k] = 0x3F80                                       # one finite logit, then a +inf
    qkv[100, 256] = 0x7F80
    out, lse = run(mbd, qkv, cu, 2, 1, 128, 0.1)
    v = wl.bf16_bits_to_f32(qkv[50, 384:])
    assert (wl.bf16_bits_to_f32(out[50:100]) == v).all() and np.allclose(lse[50:100], 12.8)
    assert np.isnan(wl.bf16_bits_to_f32(out[100:])).all() and np.isnan(lse[100:]).all()
    assert not (out[:50] & 0x7FFF).any() and (lse[:50] == -np.inf).all()


def test_without_lse_and_apart(mbd):
    """No lse; q, k and v in tensors of their own; another stream."""
    rng = np.random.default_rng(10)
    qkv, cu = make(rng, [100, 200], 4, 2, 64)
    check(mbd, qkv, cu, 4, 2, 64, lse=False)
    check(mbd, qkv, cu, 4, 2, 64, stream=torch.cuda.Stream())
    a, _ = run(mbd, qkv, cu, 4, 2, 64, 0.125)
    q, k, v = (up(np.ascontiguousarray(qkv[:, x:y])) for x, y in ((0, 256), (256, 384), (384, 512)))
    out = torch.empty(300, 256, dtype=torch.int16, device="cuda")
    mbd.prompt_attention(out, q, 0, k, v, 0, up(cu), 2, 300, 4, 2, 64, 0.125)
    assert torch.equal(out.cpu(), torch.from_numpy(a.reshape(300, 256).view(np.int16)))


def test_bad_offsets(mbd):
    """Sequences whose bounds are out of order or out of the rows are left out and flagged, the others are served."""
    rng = np.random.default_rng(11)
    qkv, _ = make(rng, [300], 2, 1, 128)
    mbd.device_error_flags(clear=True)
    for cu in ([0, 100, 400], [-5, 100, 200], [0, 200, 100]):
        out, _ = run(mbd, qkv, np.array(cu, np.int32), 2, 1, 128, 0.1)
        assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
        assert (out[200:] == 0x5A5A).all()
    good, _ = run(mbd, qkv, np.array([0, 100], np.int32), 2, 1, 128, 0.1)
    out, _ = run(mbd, qkv, np.array([0, 100, 400], np.int32), 2, 1, 128, 0.1)
    np.testing.assert_array_equal(out[:100], good[:100])
    mbd.device_error_flags(clear=True)


def test_equal_calls_and_replays(mbd):
    """Equal bits from call to call, from a captured call, and beside another call on a second stream."""
    rng = np.random.default_rng(12)
    hq, hkv, d = 8, 2, 128
    qkv, cu = make(rng, [700, 31, 257, 1200], hq, hkv, d)
    x, cu_d, n = up(qkv), up(cu), len(qkv)
    outs = [torch.zeros(n, hq * d, dtype=torch.int16, device="cuda") for _ in range(3)]
    call = lambda o, s=None: mbd.prompt_attention(o, x, qkv.shape[1], x[:, hq * d:], x[:, (hq + hkv) * d:], qkv.shape[1], cu_d, 4,
                                                  n, hq, hkv, d, 0.09, 0, None, s)
    call(outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(outs[1])
    other = torch.cuda.Stream()
    for _ in range(10):
        outs[1].zero_()
        outs[2].zero_()
        torch.cuda.synchronize()
        g.replay()
        call(outs[2], other)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    assert mbd.device_error_flags() == 0


def test_large_against_torch(mbd):
    """Thousands of tokens and all heads of a large layer, against fp32 products in chunks: relative to the sum of p |v|, the
    rounding of p and of the output, 2^-8 each, and 2^-12 for everything in fp32."""
    g = torch.Generator("cuda").manual_seed(3)
    lens, hq, hkv, d = [4001, 1, 2050, 130], 16, 2, 128
    n, width = sum(lens), (16 + 4) * 128
    qkv = torch.randn(n, width, device="cuda", generator=g).bfloat16()
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")
    out = torch.empty(n, hq * d, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(n, hq, device="cuda")
    mbd.prompt_attention(out, qkv, width, qkv[:, hq * d:], qkv[:, (hq + hkv) * d:], width, cu, 4, n, hq, hkv, d, d ** -0.5, 0, lse)
    start = 0
    for length in lens:
        x = qkv[start:start + length].double()
        for h in range(hq):
            q, k, v = x[:, h * d:(h + 1) * d], x[:, (hq + h // 8) * d:][:, :d], x[:, (hq + hkv + h // 8) * d:][:, :d]
            logits = (q @ k.t() * d ** -0.5).masked_fill_(torch.ones(length, length, device="cuda", dtype=torch.bool).triu_(1), -np.inf)
            want_lse = torch.logsumexp(logits, -1)
            p = torch.exp(logits - want_lse[:, None])
            want, size = p @ v, p @ v.abs()
            got = out[start:start + length, h * d:(h + 1) * d].double()
            assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all()
            assert (lse[start:start + length, h].double() - want_lse).abs().max() < 1e-4
        start += length
