"""Host-side checks of the key-value cache's entry points (no GPU: all of them fail before any CUDA call) and pins of
the NumPy reference that the GPU tests compare with."""
import ctypes
import re

import numpy as np
import pytest

import memory_bound_decoder_gb300 as mbd
import workloads as wl
from memory_bound_decoder_gb300 import build as mbd_build
from oracle import kv_cache as ref

A = 1 << 24   # fake device pointers, A apart: never dereferenced


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


def cache(**kw):
    a = dict(k=A, v=2 * A, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, fmt="bf16", mode="static", k_scale=3 * A,
             v_scale=4 * A, weight=5 * A, position=6 * A, page_stride=0)
    a.update(kw)
    return mbd.kv_cache(**a)


def append(c, **kw):
    a = dict(k=7 * A, v=8 * A, row_stride=0, page_table=9 * A, pages_per_seq=4, seq_lens=10 * A, n_seqs=3, n_tokens=3,
             cu_tokens=None, positions=None, stream=None)
    a.update(kw)
    return lambda: mbd.kv_cache_append(c, *a.values())


def attend(c, **kw):
    a = dict(page_table=9 * A, pages_per_seq=4, seq_lens=10 * A, n_seqs=3, n_q_heads=4, scale=0.125, window=0,
             lse=11 * A, accumulate=False, workspace=12 * A, workspace_bytes=1 << 22, stream=None)
    out, q, q_stride = kw.pop("out", 13 * A), kw.pop("q", 14 * A), kw.pop("q_stride", 0)
    a.update(kw)
    return lambda: mbd.paged_attention_decode(out, q, q_stride, c, *a.values())


def evict(c, **kw):
    a = dict(new_lens=15 * A, seq_lens=10 * A, page_table=9 * A, pages_per_seq=4, n_seqs=3, budget=16, recent=4,
             stream=None)
    a.update(kw)
    return lambda: mbd.kv_cache_evict(c, *a.values())


CALLS = [append, attend, evict]


def test_version(lib):
    hdr = open(mbd.HEADER_PATH).read()
    assert mbd.kv_abi_version() == int(re.search(r"#define MBD_KV_ABI_VERSION (\d+)", hdr).group(1)) == 1
    assert ctypes.sizeof(mbd.KVCache) == 8 * 8 + 4 * 6


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,status", [
    (dict(n_pages=0), mbd.ERR_INVALID_ARG), (dict(page_size=0), mbd.ERR_INVALID_ARG),
    (dict(n_kv_heads=0), mbd.ERR_INVALID_ARG), (dict(head_dim=0), mbd.ERR_INVALID_ARG),
    (dict(page_stride=-1), mbd.ERR_INVALID_ARG), (dict(page_stride=2 * 16 * 64 - 8), mbd.ERR_INVALID_ARG),
    (dict(fmt=2), mbd.ERR_INVALID_ARG), (dict(fmt="fp8", mode=2), mbd.ERR_INVALID_ARG),
    (dict(k=None), mbd.ERR_INVALID_ARG), (dict(v=None), mbd.ERR_INVALID_ARG),
    (dict(fmt="fp8", k_scale=None), mbd.ERR_INVALID_ARG), (dict(fmt="fp8", v_scale=None), mbd.ERR_INVALID_ARG),
    (dict(v=A), mbd.ERR_INVALID_ARG), (dict(v=A + 64), mbd.ERR_INVALID_ARG),
    (dict(v=A + 4080, page_stride=6144), mbd.ERR_INVALID_ARG),   # pages of 4096 bytes, 12288 apart: 16 bytes into
    (dict(v=A + 8208, page_stride=6144), mbd.ERR_INVALID_ARG),   # the same page, 16 bytes into the next
    (dict(weight=A + 64), mbd.ERR_INVALID_ARG), (dict(position=5 * A + 4), mbd.ERR_INVALID_ARG),
    (dict(fmt="fp8", mode="dynamic", k_scale=4 * A + 4), mbd.ERR_INVALID_ARG),
    (dict(k=A + 8), mbd.ERR_MISALIGNED), (dict(v=2 * A + 2), mbd.ERR_MISALIGNED),
    (dict(page_stride=2 * 16 * 64 + 4), mbd.ERR_MISALIGNED), (dict(fmt="fp8", k_scale=3 * A + 2), mbd.ERR_MISALIGNED),
    (dict(weight=5 * A + 1), mbd.ERR_MISALIGNED), (dict(position=6 * A + 2), mbd.ERR_MISALIGNED),
    (dict(head_dim=80), mbd.ERR_UNSUPPORTED), (dict(page_size=24), mbd.ERR_UNSUPPORTED),
    (dict(page_size=1 << 17), mbd.ERR_UNSUPPORTED), (dict(n_pages=1 << 31), mbd.ERR_UNSUPPORTED),
    (dict(n_kv_heads=8192), mbd.ERR_UNSUPPORTED),
])
def test_cache_descriptions(lib, call, kw, status):
    assert _rc(call(cache(**kw))) == status


@pytest.mark.parametrize("call", CALLS)
def test_common_arguments(lib, call):
    c = cache()
    bad = cache()
    bad.reserved = 1
    assert _rc(call(bad)) == mbd.ERR_INVALID_ARG
    assert _rc(call(c, pages_per_seq=0)) == mbd.ERR_INVALID_ARG
    assert _rc(call(c, n_seqs=-1)) == mbd.ERR_INVALID_ARG
    assert _rc(call(c, page_table=None)) == mbd.ERR_INVALID_ARG
    assert _rc(call(c, seq_lens=None)) == mbd.ERR_INVALID_ARG
    assert _rc(call(c, page_table=9 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(call(c, seq_lens=10 * A + 1)) == mbd.ERR_MISALIGNED
    assert _rc(call(c, pages_per_seq=1 << 27)) == mbd.ERR_UNSUPPORTED
    kw = dict(n_tokens=(1 << 24) + 1) if call is append else {}
    assert _rc(call(c, n_seqs=(1 << 24) + 1, **kw)) == mbd.ERR_UNSUPPORTED


def test_append_arguments(lib):
    c = cache()
    assert _rc(append(c, k=None)) == mbd.ERR_INVALID_ARG
    assert _rc(append(c, v=None)) == mbd.ERR_INVALID_ARG
    assert _rc(append(c, n_tokens=-1)) == mbd.ERR_INVALID_ARG
    assert _rc(append(c, n_tokens=4)) == mbd.ERR_INVALID_ARG            # one row per sequence without offsets
    assert _rc(append(c, n_seqs=0, cu_tokens=16 * A)) == mbd.ERR_INVALID_ARG
    assert _rc(append(c, row_stride=127)) == mbd.ERR_INVALID_ARG
    assert _rc(append(c, row_stride=132)) == mbd.ERR_MISALIGNED
    assert _rc(append(c, k=7 * A + 8)) == mbd.ERR_MISALIGNED
    assert _rc(append(c, cu_tokens=16 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(append(c, positions=16 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(append(c, k=A + 4096)) == mbd.ERR_INVALID_ARG            # reads what it writes
    assert _rc(append(c, seq_lens=5 * A + 64)) == mbd.ERR_INVALID_ARG
    mbd.kv_cache_append(c, None, None, 0, None, 4, None, 0, 0)           # nothing to do
    mbd.kv_cache_append(c, None, None, 0, None, 4, None, 3, 0)


def test_attention_arguments(lib):
    c = cache()
    assert _rc(attend(c, n_q_heads=3)) == mbd.ERR_INVALID_ARG           # not a multiple of the key-value heads
    assert _rc(attend(c, n_q_heads=0)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, scale=float("nan"))) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, scale=float("inf"))) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, scale=3e38)) == mbd.ERR_INVALID_ARG            # not finite in units of log2
    assert _rc(attend(c, window=-1)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, out=None)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, q=None)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, q_stride=255)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, q_stride=260)) == mbd.ERR_MISALIGNED
    assert _rc(attend(c, out=13 * A + 8)) == mbd.ERR_MISALIGNED
    assert _rc(attend(c, q=14 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(attend(c, lse=11 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(attend(c, out=14 * A)) == mbd.ERR_INVALID_ARG            # overlaps q
    assert _rc(attend(c, out=A + 256)) == mbd.ERR_INVALID_ARG           # inside the cache
    assert _rc(attend(c, lse=13 * A + 64)) == mbd.ERR_INVALID_ARG       # inside out
    assert _rc(attend(cache(weight=None), accumulate=True)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, accumulate=True, workspace=None)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, accumulate=True, workspace_bytes=16)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, accumulate=True, workspace=12 * A + 128)) == mbd.ERR_MISALIGNED
    assert _rc(attend(c, accumulate=True, workspace=A)) == mbd.ERR_INVALID_ARG
    assert _rc(attend(c, n_seqs=1 << 20, n_q_heads=32)) == mbd.ERR_UNSUPPORTED
    mbd.paged_attention_decode(None, None, 0, c, None, 4, None, 0, 4, 0.125)
    size = mbd.paged_attention_workspace_bytes
    assert size(c, 4, 0, 4, True) == 0 and size(c, 0, 3, 4, True) == 0 and size(c, 4, 3, 3, True) == 0
    assert size(cache(head_dim=80), 4, 3, 4, True) == 0
    assert size(c, 4, 3, 4, True) >= size(c, 4, 3, 4, False) + 3 * 4 * 4 * 16 * 4


def test_evict_arguments(lib):
    c = cache()
    assert _rc(evict(c, new_lens=None)) == mbd.ERR_INVALID_ARG
    assert _rc(evict(c, new_lens=10 * A)) == mbd.ERR_INVALID_ARG        # read by some heads while others write it
    assert _rc(evict(c, new_lens=15 * A + 2)) == mbd.ERR_MISALIGNED
    assert _rc(evict(c, budget=-1)) == mbd.ERR_INVALID_ARG
    assert _rc(evict(c, recent=-1)) == mbd.ERR_INVALID_ARG
    assert _rc(evict(c, recent=17)) == mbd.ERR_INVALID_ARG
    assert _rc(evict(cache(weight=None))) == mbd.ERR_INVALID_ARG
    assert _rc(evict(cache(position=None))) == mbd.ERR_INVALID_ARG
    assert _rc(evict(c, pages_per_seq=425984 // 16 + 1)) == mbd.ERR_UNSUPPORTED
    assert _rc(evict(c, budget=(1 << 30) + 1)) == mbd.ERR_UNSUPPORTED
    assert _rc(evict(cache(n_pages=(1 << 27) + 1, k=1 << 40, v=1 << 42, weight=1 << 44, position=1 << 45))) == mbd.ERR_UNSUPPORTED
    assert _rc(evict(c, n_seqs=(1 << 23) + 1)) == mbd.ERR_UNSUPPORTED
    mbd.kv_cache_evict(c, None, None, None, 4, 0, 16, 4)


def test_interleaved_pools_are_accepted(lib):
    """k and v as the two halves of one pool's pages: the description passes, and an empty call does nothing."""
    c = cache(v=A + 4096, page_stride=4096)
    assert _rc(attend(c, q=None)) == mbd.ERR_INVALID_ARG      # (q is checked before the pointers of the cache)
    assert _rc(attend(c, out=A + 64)) == mbd.ERR_INVALID_ARG
    assert _rc(evict(c, new_lens=2 * A, seq_lens=2 * A)) == mbd.ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------------ the reference itself

def test_e4m3_codes():
    finite = np.array([c for c in range(256) if c & 0x7F != 0x7F])
    np.testing.assert_array_equal(ref.e4m3_codes(ref.E4M3[finite]), finite)
    # ties go to the even code: half the least step, 17 and 19 between 16, 18 and 20, 432 between 416 and 448
    x = np.array([2.0 ** -10, 3 * 2.0 ** -10, 17.0, 19.0, 432.0, 464.0, 1e9, -0.0, -1e-9])
    assert list(ref.E4M3[ref.e4m3_codes(x)]) == [0.0, 2.0 ** -8, 16.0, 20.0, 448.0, 448.0, 448.0, 0.0, 0.0]
    assert list(ref.e4m3_codes(x)[-2:]) == [0x80, 0x80]


def test_reference_attention_closed_forms():
    """One token: the output is its value, lse its logit. Equal keys: the mean of the values."""
    rng = np.random.default_rng(0)
    c = ref.Cache(rng, [1, 5, 0], 1, 64, 4, "bf16")
    c.view(c.k_raw)[:] = wl.f32_to_bf16_bits(np.ones(64, np.float32))
    q = wl.f32_to_bf16_bits(np.full((3, 1, 64), 0.5, np.float32))
    out, lse, *_ = c.attend(q, 1, 0.25)
    np.testing.assert_allclose(out[0, 0], c.rows(0, [0])[1][0, 0])
    np.testing.assert_allclose(out[1, 0], c.rows(1, np.arange(5))[1][0].mean(0))
    assert lse[0, 0] == 8.0 and abs(lse[1, 0] - 8.0 - np.log(5)) < 1e-12 and lse[2, 0] == -np.inf
    assert not out[2].any()


def test_reference_eviction_by_hand():
    rng = np.random.default_rng(1)
    c = ref.Cache(rng, [6], 1, 64, 2, "bf16")
    p, _, s = c.at(0, np.arange(6))
    c.weight[p, 0, s] = [0.1, 0.5, 0.1, 0.5, 0.0, 0.9]
    c.position[p, 0, s] = [5, 0, 1, 2, 4, 3]
    before = c.rows(0, np.arange(6))[0][0].copy()
    # newest: slot 0 (position 5); then 5 (0.9) and 1 (0.5, before slot 3): slots 0, 1 stay, slot 2 takes slot 5's row
    assert list(c.evict(3, 1)) == [3]
    np.testing.assert_array_equal(c.rows(0, np.arange(3))[0][0], before[[0, 1, 5]])
    assert list(c.position[p, 0, s][:3]) == [5, 0, 3]
