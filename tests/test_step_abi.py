"""Host-side checks of the serving step's entry points (no GPU: all of them fail before any CUDA call), the frequencies of
rotary positions, and pins of the NumPy reference that the GPU tests compare with."""
import ctypes
import math
import re
from fractions import Fraction

import numpy as np
import pytest

import memory_bound_decoder_gb300 as mbd
import workloads as wl
from memory_bound_decoder_gb300 import build as mbd_build
from oracle import step as ref

A = 1 << 28   # fake device pointers, A apart: never dereferenced


@pytest.fixture(scope="module")
def lib():
    mbd_build.build()
    return mbd.get_lib()


def _rc(fn, *args, **kw):
    n0 = mbd.kernel_launches()
    with pytest.raises(mbd.MbdError) as e:
        fn(*args, **kw)
    assert mbd.kernel_launches() == n0
    return e.value.status


def resize(**kw):
    a = dict(page_table=A, pages_per_seq=4, page_size=16, n_pages=8, free_pages=2 * A, free_ends=3 * A, seq_lens=4 * A,
             want_lens=5 * A, n_seqs=3, cu_tokens=6 * A, positions=7 * A, slots=8 * A, n_tokens=5, tokens_seen=9 * A,
             stream=None)
    a.update(kw)
    return lambda: mbd.kv_cache_resize(*a.values())


def rotary(**kw):
    a = dict(out=A, out_stride=0, x=2 * A, x_stride=0, turns=3 * A, amplitude=1.0, positions=4 * A, n_tokens=5, n_heads=3,
             head_dim=64, rotary_dim=32, layout="half", stream=None)
    a.update(kw)
    return lambda: mbd.rotary(*a.values())


def test_version(lib):
    hdr = open(mbd.HEADER_PATH).read()
    assert mbd.step_abi_version() == int(re.search(r"#define MBD_STEP_ABI_VERSION (\d+)", hdr).group(1)) == 1
    assert ctypes.sizeof(mbd.RotaryScaling) == 8 + 8 * 8 + 8


@pytest.mark.parametrize("kw,status", [
    (dict(pages_per_seq=0), mbd.ERR_INVALID_ARG), (dict(page_size=0), mbd.ERR_INVALID_ARG),
    (dict(n_pages=0), mbd.ERR_INVALID_ARG), (dict(n_seqs=-1), mbd.ERR_INVALID_ARG), (dict(n_tokens=-1), mbd.ERR_INVALID_ARG),
    (dict(page_table=None), mbd.ERR_INVALID_ARG), (dict(free_pages=None), mbd.ERR_INVALID_ARG),
    (dict(free_ends=None), mbd.ERR_INVALID_ARG), (dict(seq_lens=None), mbd.ERR_INVALID_ARG),
    (dict(want_lens=None), mbd.ERR_INVALID_ARG), (dict(cu_tokens=None), mbd.ERR_INVALID_ARG),
    (dict(want_lens=4 * A), mbd.ERR_INVALID_ARG), (dict(free_ends=2 * A + 28), mbd.ERR_INVALID_ARG),
    (dict(cu_tokens=A + 44), mbd.ERR_INVALID_ARG), (dict(slots=7 * A + 16), mbd.ERR_INVALID_ARG),
    (dict(page_table=A + 2), mbd.ERR_MISALIGNED), (dict(slots=8 * A + 4), mbd.ERR_MISALIGNED),
    (dict(positions=7 * A + 1), mbd.ERR_MISALIGNED), (dict(tokens_seen=9 * A + 2), mbd.ERR_MISALIGNED),
    (dict(page_size=24), mbd.ERR_UNSUPPORTED), (dict(page_size=1 << 17), mbd.ERR_UNSUPPORTED),
    (dict(n_seqs=8193), mbd.ERR_UNSUPPORTED), (dict(n_pages=1 << 31), mbd.ERR_UNSUPPORTED),
    (dict(pages_per_seq=1 << 27), mbd.ERR_UNSUPPORTED), (dict(pages_per_seq=1 << 26, n_seqs=32), mbd.ERR_UNSUPPORTED),
    (dict(n_tokens=(1 << 24) + 1), mbd.ERR_UNSUPPORTED),
])
def test_resize_arguments(lib, kw, status):
    assert _rc(resize(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(n_tokens=-1), mbd.ERR_INVALID_ARG), (dict(n_heads=0), mbd.ERR_INVALID_ARG), (dict(rotary_dim=0), mbd.ERR_INVALID_ARG),
    (dict(rotary_dim=80), mbd.ERR_INVALID_ARG), (dict(layout=2), mbd.ERR_INVALID_ARG),
    (dict(amplitude=math.inf), mbd.ERR_INVALID_ARG), (dict(amplitude=math.nan), mbd.ERR_INVALID_ARG),
    (dict(out=None), mbd.ERR_INVALID_ARG), (dict(x=None), mbd.ERR_INVALID_ARG), (dict(turns=None), mbd.ERR_INVALID_ARG),
    (dict(x_stride=184), mbd.ERR_INVALID_ARG), (dict(out_stride=-8), mbd.ERR_INVALID_ARG),
    (dict(x=A + 64), mbd.ERR_INVALID_ARG), (dict(x=A, x_stride=200), mbd.ERR_INVALID_ARG),
    (dict(turns=A + 8), mbd.ERR_INVALID_ARG), (dict(positions=A + 4), mbd.ERR_INVALID_ARG),
    (dict(x_stride=196), mbd.ERR_MISALIGNED), (dict(out=A + 8), mbd.ERR_MISALIGNED), (dict(x=2 * A + 4), mbd.ERR_MISALIGNED),
    (dict(turns=3 * A + 4), mbd.ERR_MISALIGNED), (dict(positions=4 * A + 2), mbd.ERR_MISALIGNED),
    (dict(head_dim=72), mbd.ERR_UNSUPPORTED), (dict(rotary_dim=24), mbd.ERR_UNSUPPORTED),
    (dict(head_dim=4112), mbd.ERR_UNSUPPORTED), (dict(n_tokens=(1 << 24) + 1), mbd.ERR_UNSUPPORTED),
])
def test_rotary_arguments(lib, kw, status):
    assert _rc(rotary(**kw)) == status


def test_empty_calls(lib):
    n0 = mbd.kernel_launches()
    mbd.kv_cache_resize(None, 4, 16, 8, None, None, None, None, 0, None, None, None, 5)
    mbd.rotary(None, 0, None, 0, None, 1.0, None, 0, 3, 64, 32)
    assert mbd.kernel_launches() == n0


# ------------------------------------------------------------------------------------------------ frequencies

# A table's unit is 2^-64 of a turn, 3.4e-19 radians, and it is rounded to nearest: 1.7e-19, which is more than 1e-13 of the
# slowest frequencies. 2^-60 is 8.7e-19.
UNIT = 2.0 ** -60


def freqs(table):
    return np.array([x * 2.0 ** -64 * 2 * math.pi for x in table])


@pytest.mark.parametrize("dim", [16, 64, 128])
def test_plain_and_stretched_frequencies(lib, dim):
    g = 10000.0 ** (-np.arange(0, dim, 2) / dim)
    # 2^-50: a few roundings of fp64 (pow, the division by 2 pi) of frequencies up to 1
    close = lambda table, want: np.testing.assert_allclose(freqs(table), want, rtol=2.0 ** -50, atol=UNIT)
    table, amp = mbd.rotary_table(dim)
    assert amp == 1.0
    close(table, g)
    close(mbd.rotary_table(dim, scaling="linear", factor=4.0)[0], g / 4)
    close(mbd.rotary_table(dim, scaling="ntk", factor=8.0)[0], (10000.0 * 8 ** (dim / (dim - 2))) ** (-np.arange(0, dim, 2) / dim))
    f = 1.0 + np.arange(dim // 2) / 7
    table, amp = mbd.rotary_table(dim, scaling="factors", factors=f, amplitude=1.25)
    assert amp == 1.25
    close(table, g / f)


def test_frequencies_in_bands(lib):
    """The fastest pairs stay, the slowest are divided by the factor, those between lie between."""
    dim = 128
    g = 500000.0 ** (-np.arange(0, dim, 2) / dim)
    f = freqs(mbd.rotary_table(dim, 500000.0, "llama3", 8.0, 8192, 1.0, 4.0)[0])
    turns = 8192 * g / (2 * math.pi)
    np.testing.assert_allclose(f[turns > 4], g[turns > 4], rtol=1e-13, atol=UNIT)
    np.testing.assert_allclose(f[turns < 1], g[turns < 1] / 8, rtol=1e-13, atol=UNIT)
    mid = (turns > 1) & (turns < 4)
    assert mid.any()
    s = (turns[mid] - 1) / 3
    np.testing.assert_allclose(f[mid], (1 - s) * g[mid] / 8 + s * g[mid], rtol=1e-13, atol=UNIT)


def test_frequencies_ramped(lib):
    dim, base = 128, 1e6
    g = base ** (-np.arange(0, dim, 2) / dim)
    table, amp = mbd.rotary_table(dim, base, "yarn", 4.0, 32768)
    assert amp == np.float32(0.1 * math.log(4.0) + 1)
    f = freqs(table)
    d = lambda b: dim * math.log(32768 / (2 * math.pi * b)) / (2 * math.log(base))
    first, last = math.floor(d(32)), math.ceil(d(1))
    assert 0 < first < last < dim // 2
    np.testing.assert_allclose(f[:first + 1], g[:first + 1], rtol=1e-13, atol=UNIT)
    np.testing.assert_allclose(f[last:], g[last:] / 4, rtol=1e-13, atol=UNIT)
    i = np.arange(first, last)
    r = (i - first) / (last - first)
    np.testing.assert_allclose(f[i], r * g[i] / 4 + (1 - r) * g[i], rtol=1e-13, atol=UNIT)
    assert mbd.rotary_table(dim, base, "yarn", 0.5, 32768)[1] == 1.0


def test_table_refusals(lib):
    for args in [(0,), (7,), (-2,), (64, 0.0), (64, math.inf), (64, math.nan), (64, 1e4, 9), (64, 1e4, "linear", 0.0),
                 (64, 1e4, "linear", math.inf), (2, 1e4, "ntk", 2.0), (64, 1e4, "llama3", 8.0, 0.0),
                 (64, 1e4, "llama3", 8.0, 8192, 4.0, 4.0), (64, 1.0, "yarn", 4.0, 32768), (64, 1e4, "yarn", 4.0, 0.0),
                 (64, 1e4, "factors")]:
        assert _rc(mbd.rotary_table, *args) == mbd.ERR_INVALID_ARG, args
    assert _rc(mbd.rotary_table, 64, amplitude=-1.0) == mbd.ERR_INVALID_ARG
    assert _rc(mbd.rotary_table, 4, scaling="factors", factors=[1.0, 0.0]) == mbd.ERR_INVALID_ARG
    with pytest.raises(ValueError):
        mbd.rotary_table(64, scaling="factors", factors=[1.0])


def test_whole_turns_count_as_none(lib):
    """A frequency of many turns a position keeps its fraction."""
    table, _ = mbd.rotary_table(2, scaling="factors", factors=[2.0 ** -10 / (2 * math.pi) / 1.25])
    assert abs(table[0] - 0) < 2 ** 24 or abs(table[0] - 2 ** 64) < 2 ** 24   # 1280 turns


# ------------------------------------------------------------------------------------------------ the reference itself

def test_reference_rotary_against_rational_turns():
    """A quarter turn a position: the pair (a, b) goes to (-b, a), (-a, -b), (b, -a), and back; far positions too."""
    x = wl.f32_to_bf16_bits(np.array([[3.0, 5.0]], np.float32).repeat(6, 0))
    out, _ = ref.rotary(x, [0, 1, 2, 3, 2 ** 31 - 4, -1], [2 ** 62], 1.0, 1, 2, 2, "interleaved")
    np.testing.assert_allclose(out[:, 0], [[3, 5], [-5, 3], [-3, -5], [5, -3], [3, 5], [5, -3]], atol=1e-14)
    assert float(Fraction(2 ** 62, 2 ** 64)) == 0.25


def test_reference_resize_by_hand():
    rng = np.random.default_rng(0)
    p = ref.Pages(rng, [5, 4, 0, 9], 4, 4, 2)
    p.table[:] = [[0, 1, -1, -1], [2, -1, -1, -1], [-1] * 4, [3, 4, 5, -1]]
    p.ring[:] = [-7] * 6 + [6, 7]
    p.ends[:], p.seen[:] = (6, 2), (5, 104, 0, 9)
    # 0 ends (its pages 0, 1 go behind 6, 7), 1 takes page 6, 2 wants 12 tokens (pages 7, 0, 1), 3 has nothing left to take
    cu, positions, slots = p.resize([0, 5, 12, 13], 20)
    assert list(cu) == [0, 0, 1, 13, 13] and list(p.lens) == [0, 5, 12, 9] and list(p.seen) == [0, 105, 12, 9]
    assert p.table.tolist() == [[-1] * 4, [2, 6, -1, -1], [7, 0, 1, -1], [3, 4, 5, -1]]
    assert list(p.ends) == [2, 0] and list(slots[:3]) == [24, 28, 29] and list(slots[12:]) == [7] + [-1] * 7
    assert list(positions[:3]) == [104, 0, 1] and not positions[13:].any()


def test_reference_prompt_closed_forms():
    """Equal keys: the mean of the values seen so far, lse the logit and the logarithm of their number."""
    rng = np.random.default_rng(1)
    one = lambda *s: wl.f32_to_bf16_bits(np.ones(s, np.float32))
    v = wl.f32_to_bf16_bits(rng.standard_normal((7, 64)).astype(np.float32))
    out, lse, *_ = ref.prompt(one(7, 64), one(7, 64), v, [0, 3, 3, 7], 1, 1, 64, 0.125, 2)
    f = wl.bf16_bits_to_f32(v).astype(np.float64)
    np.testing.assert_allclose(out[:, 0], [f[0], f[0:2].mean(0), f[1:3].mean(0), f[3], f[3:5].mean(0), f[4:6].mean(0), f[5:7].mean(0)])
    np.testing.assert_allclose(lse[:, 0] - 8, np.log([1, 2, 2, 1, 2, 2, 2]), atol=1e-12)


# ------------------------------------------------------------------------------------------------ prompts

def prompt(**kw):
    a = dict(out=A, q=2 * A, q_stride=0, k=3 * A, v=4 * A, kv_stride=0, cu_tokens=5 * A, n_seqs=3, n_tokens=50, n_q_heads=4,
             n_kv_heads=2, head_dim=64, scale=0.125, window=0, lse=6 * A, stream=None)
    a.update(kw)
    return lambda: mbd.prompt_attention(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(n_seqs=-1), mbd.ERR_INVALID_ARG), (dict(n_tokens=-1), mbd.ERR_INVALID_ARG), (dict(n_q_heads=0), mbd.ERR_INVALID_ARG),
    (dict(n_kv_heads=0), mbd.ERR_INVALID_ARG), (dict(n_q_heads=3), mbd.ERR_INVALID_ARG), (dict(head_dim=0), mbd.ERR_INVALID_ARG),
    (dict(window=-1), mbd.ERR_INVALID_ARG), (dict(scale=math.inf), mbd.ERR_INVALID_ARG),
    (dict(scale=math.nan), mbd.ERR_INVALID_ARG), (dict(scale=3e38), mbd.ERR_INVALID_ARG),
    (dict(out=None), mbd.ERR_INVALID_ARG), (dict(q=None), mbd.ERR_INVALID_ARG), (dict(k=None), mbd.ERR_INVALID_ARG),
    (dict(v=None), mbd.ERR_INVALID_ARG), (dict(cu_tokens=None), mbd.ERR_INVALID_ARG),
    (dict(q_stride=248), mbd.ERR_INVALID_ARG), (dict(kv_stride=120), mbd.ERR_INVALID_ARG),
    (dict(out=2 * A + 512), mbd.ERR_INVALID_ARG), (dict(out=3 * A), mbd.ERR_INVALID_ARG), (dict(out=4 * A + 16), mbd.ERR_INVALID_ARG),
    (dict(lse=A + 64), mbd.ERR_INVALID_ARG), (dict(lse=2 * A + 64), mbd.ERR_INVALID_ARG), (dict(cu_tokens=A + 64), mbd.ERR_INVALID_ARG),
    (dict(out=A + 8), mbd.ERR_MISALIGNED), (dict(q=2 * A + 2), mbd.ERR_MISALIGNED), (dict(k=3 * A + 8), mbd.ERR_MISALIGNED),
    (dict(v=4 * A + 4), mbd.ERR_MISALIGNED), (dict(q_stride=260), mbd.ERR_MISALIGNED), (dict(kv_stride=132), mbd.ERR_MISALIGNED),
    (dict(cu_tokens=5 * A + 2), mbd.ERR_MISALIGNED), (dict(lse=6 * A + 2), mbd.ERR_MISALIGNED),
    (dict(head_dim=80), mbd.ERR_UNSUPPORTED), (dict(head_dim=512), mbd.ERR_UNSUPPORTED),
    (dict(n_q_heads=8192), mbd.ERR_UNSUPPORTED), (dict(n_tokens=(1 << 24) + 1), mbd.ERR_UNSUPPORTED),
    (dict(n_seqs=(1 << 24) + 1), mbd.ERR_UNSUPPORTED),
])
def test_prompt_arguments(lib, kw, status):
    assert _rc(prompt(**kw)) == status


def test_empty_prompts(lib):
    n0 = mbd.kernel_launches()
    for kw in (dict(n_seqs=0), dict(n_tokens=0)):
        prompt(**{**dict(out=None, q=None, k=None, v=None, cu_tokens=None), **kw})()
    assert mbd.kernel_launches() == n0
