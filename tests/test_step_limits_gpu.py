"""The serving step's operators at the largest sizes that the header allows, as far as memory and seconds go: results are those of small
calls over the same rows."""
import numpy as np
import pytest

from oracle import step as ref
from tests.test_kv_gpu import mbd, up  # noqa: F401  (mbd is the fixture)
from tests.test_prompt_gpu import check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

MOST = 1 << 24


def i32(*values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def test_a_prompt_of_the_most_tokens(mbd):
    """2^24 rows in a window: a row depends on the window's rows alone, whose bits a cut of the prompt has from a block's border on."""
    window, d, tail = 100, 64, 1000
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(1 << 16, 3 * d, device="cuda", generator=g).bfloat16().repeat(MOST >> 16, 1)
    out, lse = torch.zeros(MOST, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(MOST, 1, device="cuda")
    mbd.device_error_flags(clear=True)
    call = lambda o, l, y, n: mbd.prompt_attention(o, y, 3 * d, y[:, d:], y[:, 2 * d:], 3 * d, i32(0, n), 1, n, 1, 1, d, 0.125, window, l)
    call(out, lse, x, MOST)
    n = 1 << 17                                              # two periods of the rows
    small, small_lse = torch.zeros(n, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, 1, device="cuda")
    call(small, small_lse, x[:n], n)
    torch.cuda.synchronize()
    assert mbd.device_error_flags() == 0
    assert torch.equal(out[:n], small) and torch.equal(lse[:n], small_lse)
    for period in (2, 100, (MOST >> 16) - 1):
        at = period << 16
        assert torch.equal(out[at:at + (1 << 16)], small[1 << 16:]) and torch.equal(lse[at:at + (1 << 16)], small_lse[1 << 16:])
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("hq,hkv,d", [(4096, 1, 64), (4096, 4096, 64), (4095, 1365, 64)])
def test_prompts_of_the_most_heads(mbd, hq, hkv, d):
    rng = np.random.default_rng(hkv)
    check(mbd, *make(rng, [3, 0, 130 if hkv == 1 else 9], hq, hkv, d, pad=2), hq, hkv, d)


def test_the_widest_strides(mbd):
    """One row, whose stride is never used."""
    x = torch.randn(1, 384, device="cuda").bfloat16()
    out, a = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda"), x.clone()
    far = 1 << 34
    mbd.prompt_attention(out, x, far, x[:, 128:], x[:, 256:], far, i32(0, 1), 1, 1, 1, 1, 128, 0.1)
    turns, amp = mbd.rotary_table(128)
    t = torch.frombuffer(turns, dtype=torch.int64).cuda()
    mbd.rotary(a, far, a, far, t, amp, i32(0), 1, 3, 128, 128)
    torch.cuda.synchronize()
    assert torch.equal(out, x[:, 256:]) and torch.equal(a, x)
    assert mbd.device_error_flags() == 0


def test_rotary_of_the_most_rows_and_heads(mbd):
    turns, amp = mbd.rotary_table(16)
    t = torch.frombuffer(turns, dtype=torch.int64).cuda()
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(MOST, 16, device="cuda", generator=g).bfloat16()
    out, want = torch.empty_like(x), torch.empty(1000, 16, dtype=torch.bfloat16, device="cuda")
    mbd.rotary(out, 0, x, 0, t, amp, None, MOST, 1, 16, 16)
    mbd.rotary(want, 0, x[-1000:], 0, t, amp, torch.arange(MOST - 1000, MOST, dtype=torch.int32, device="cuda"), 1000, 1, 16, 16)
    torch.cuda.synchronize()
    assert torch.equal(out[-1000:], want)
    heads = 1 << 20                                          # one row of 2^20 heads is 2^20 rows of one head at its position
    mbd.rotary(out, 0, x, 0, t, amp, i32(77), 1, heads, 16, 16)
    mbd.rotary(x[heads:], 0, x[:heads], 0, t, amp, torch.full((heads,), 77, dtype=torch.int32, device="cuda"), heads, 1, 16, 16)
    torch.cuda.synchronize()
    assert torch.equal(out[:heads], x[heads:2 * heads])


@pytest.mark.parametrize("page", [1, 1 << 16])
def test_resize_by_the_most_rows(mbd, page):
    """One sequence takes 2^24 tokens at once, and one of 8192 the last page."""
    rng = np.random.default_rng(3)
    n = 8192 if page > 1 else 2
    width = MOST // page
    p = ref.Pages(rng, [0] * n, page, width, width + 1)
    want = np.zeros(n, np.int32)
    want[[n // 2 - 1, n - 1]] = MOST - 1, 1
    d = {f: up(getattr(p, f)) for f in ("table", "ring", "ends", "lens", "seen")}
    cu, pos, slots = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(MOST, dtype=torch.int32, device="cuda"), \
        torch.zeros(MOST, dtype=torch.int64, device="cuda")
    mbd.device_error_flags(clear=True)
    mbd.kv_cache_resize(d["table"], width, page, p.n_pages, d["ring"], d["ends"], d["lens"], up(want), n, cu, pos, slots, MOST, d["seen"])
    torch.cuda.synchronize()
    assert mbd.device_error_flags() == 0
    long = int(np.argmax(want))
    ring = np.roll(p.ring, -p.ends[0])
    pages = ring[:-(-(MOST - 1) // page)]
    at = np.arange(MOST - 1)
    np.testing.assert_array_equal(d["table"].cpu().numpy()[long, :len(pages)], pages)
    np.testing.assert_array_equal(slots.cpu().numpy()[:-1], pages[at // page].astype(np.int64) * page + at % page)
    np.testing.assert_array_equal(pos.cpu().numpy(), np.append(at, 0))
    assert slots[-1].item() == int(ring[len(pages)]) * page
    np.testing.assert_array_equal(d["lens"].cpu().numpy(), want)
    np.testing.assert_array_equal(cu.cpu().numpy(), np.concatenate([[0], np.cumsum(want)]))
    assert d["ends"].cpu()[1].item() == p.n_pages - len(pages) - 1
