"""The serving step's operators where offsets pass 32 bits and where numbers of sequences change the order of the work: results are
those of the small call, bit for bit."""
import numpy as np
import pytest

from tests.test_kv_gpu import mbd  # noqa: F401  (mbd is the fixture)
from tests.test_prompt_gpu import check, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [32, 33, 256, 257])
@pytest.mark.parametrize("hq,hkv", [(2, 1), (1, 1)])
def test_prompts_of_many_sequences(mbd, n, hq, hkv):
    """Sequences of any length in every order, some empty: found by place up to 256 of them, one behind the other from there on."""
    rng = np.random.default_rng(n)
    lens = rng.integers(0, 40, n)
    lens[rng.integers(0, n, 4)] = [0, 130, 300, 129]
    check(mbd, *make(rng, lens, hq, hkv, 64, pad=5), hq, hkv, 64)


def test_prompts_beyond_32_bits(mbd):
    """Rows whose inputs and outputs lie more than 4 GiB behind the first."""
    n, length, hq, hkv, d = 140000, 500, 128, 8, 128
    width = (hq + 2 * hkv) * d
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(n, width, dtype=torch.bfloat16, device="cuda")
    x[-length:] = torch.randn(length, width, device="cuda", generator=g).bfloat16()
    out = torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(n, hq, device="cuda")
    assert out.numel() * 2 > 1 << 32 and x.numel() * 2 > 1 << 32
    x[:length] = x[-length:]
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    small, small_lse = torch.zeros(length, hq * d, dtype=torch.bfloat16, device="cuda"), torch.zeros(length, hq, device="cuda")
    part = lambda t: (t[:, :hq * d], width, t[:, hq * d:], t[:, (hq + hkv) * d:], width)
    x[length:-length] = 1.0                                  # one long sequence in the middle, within a window
    mbd.prompt_attention(out, *part(x), i32(0, length, n - length, n), 3, n, hq, hkv, d, 0.09, 300, lse)
    mbd.prompt_attention(small, *part(x), i32(0, length), 1, length, hq, hkv, d, 0.09, 300, small_lse)
    torch.cuda.synchronize()
    assert torch.equal(out[-length:], small) and torch.equal(lse[-length:], small_lse)
    assert torch.equal(out[:length], small) and torch.isfinite(small.float()).all()


def test_rotary_beyond_32_bits(mbd):
    """Rows 64 MiB apart."""
    n, stride, heads, d = 80, 1 << 25, 3, 128
    g = torch.Generator("cuda").manual_seed(2)
    rows = torch.randn(n, heads * d, device="cuda", generator=g).bfloat16()
    pool = torch.empty(n * stride, dtype=torch.bfloat16, device="cuda")
    assert pool.numel() * 2 > 1 << 32
    view = pool.view(n, stride)
    view[:, :heads * d] = rows
    turns, amp = mbd.rotary_table(d, scaling="linear", factor=2.0)
    t = torch.frombuffer(turns, dtype=torch.int64).cuda()
    at = torch.arange(n, dtype=torch.int32, device="cuda") * 12345
    want = torch.empty_like(rows)
    mbd.rotary(want, 0, rows, 0, t, amp, at, n, heads, d, d)
    mbd.rotary(pool, stride, pool, stride, t, amp, at, n, heads, d, d)
    torch.cuda.synchronize()
    assert torch.equal(view[:, :heads * d], want)
