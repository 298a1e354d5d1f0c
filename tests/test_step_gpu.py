"""Pages and slots, and rotary positions on the GPU against the NumPy reference, between guard bands."""
import numpy as np
import pytest

import workloads as wl
from oracle import step as ref
from oracle.kv_cache import check_close
from tests.parity import Guarded
from tests.test_kv_gpu import bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ pages

class Pages(ref.Pages):
    """With a copy on the GPU between guard bands."""

    FIELDS = ("table", "ring", "ends", "lens", "seen")

    def device(self):
        self.g = {f: Guarded(torch, getattr(self, f).size, torch.int32, fill=getattr(self, f)) for f in self.FIELDS}
        return self

    def call(self, mbd, want, n_tokens, outputs=True, seen=True, stream=None):
        n = len(self.lens)
        out = dict(cu=Guarded(torch, n + 1, torch.int32), positions=Guarded(torch, n_tokens, torch.int32),
                   slots=Guarded(torch, n_tokens, torch.int64))
        want_d = up(np.asarray(want, np.int32))
        d = {f: g.view for f, g in self.g.items()}
        torch.cuda.synchronize()
        mbd.kv_cache_resize(d["table"], self.width, self.page, self.n_pages, d["ring"], d["ends"], d["lens"], want_d, n,
                            out["cu"].view, out["positions"].view if outputs else None, out["slots"].view if outputs else None,
                            n_tokens, d["seen"] if seen else None, stream)
        torch.cuda.synchronize()
        for f, g in list(out.items()) + list(self.g.items()):
            g.check_guards(f)
        return out["cu"].numpy(np.int32), out["positions"].numpy(np.int32), out["slots"].numpy(np.int64)

    def check(self):
        for f in self.FIELDS:
            np.testing.assert_array_equal(self.g[f].numpy(np.int32), getattr(self, f).reshape(-1), f)

    def step(self, mbd, want, n_tokens):
        got = self.call(mbd, want, n_tokens)
        for g, w, what in zip(got, self.resize(want, n_tokens), ("cu", "positions", "slots")):
            np.testing.assert_array_equal(g, w, what)
        self.check()


@pytest.mark.parametrize("n,page,hi", [(1, 1, 40), (3, 16, 100), (40, 8, 300), (1000, 4, 60), (1025, 16, 200), (3000, 2, 9),
                                       (8192, 1, 3)])
@pytest.mark.parametrize("room", ["ample", "few pages", "few rows"])
def test_resize(mbd, n, page, hi, room):
    """Several steps of growing, ending and starting sequences over one ring, which goes round; where pages or rows are
    few, some are refused."""
    rng = np.random.default_rng(n + page)
    lens = rng.integers(0, hi + 1, n) * (rng.random(n) < 0.7)
    width = -(-hi // page)
    spare = n * width if room == "ample" else n * width // 8 + 1
    p = Pages(rng, lens, page, width, spare).device()
    mbd.device_error_flags(clear=True)
    for step in range(6):
        kind = rng.random(n)
        want = np.where(kind < 0.2, 0, np.where(kind < 0.7, np.minimum(p.lens + 1, hi), rng.integers(0, hi + 1, n)))
        rows = int(np.maximum(0, want - p.lens).sum())
        p.step(mbd, want, rows // 2 if room == "few rows" else rows + (step % 3) * 7)
    assert mbd.device_error_flags() == 0


def test_resize_of_nothing(mbd):
    """Lengths that stay: no rows, nothing changed; no room for rows at all."""
    rng = np.random.default_rng(0)
    p = Pages(rng, [5, 0, 64], 16, 4, 3).device()
    p.step(mbd, [5, 0, 64], 4)
    p.step(mbd, [6, 1, 30], 0)
    assert list(p.lens) == [5, 0, 30]


def test_resize_of_a_long_prompt(mbd):
    """One sequence of a hundred thousand tokens comes and goes."""
    rng = np.random.default_rng(1)
    p = Pages(rng, [0, 3], 16, 8192, 9000).device()
    p.step(mbd, [100001, 4], 100002)
    p.step(mbd, [0, 5], 1)
    p.step(mbd, [131072, 0], 131072)


def test_resize_out_of_range(mbd):
    """Lengths out of range, ends outside the ring, pages outside the pool, a page given up twice: flagged, nothing outside
    the tensors written, other sequences served."""
    rng = np.random.default_rng(2)
    p = Pages(rng, [5, 7, 9, 0], 4, 4, 6).device()
    mbd.device_error_flags(clear=True)
    p.step(mbd, [6, 17, -1, 3], 30)
    assert list(p.lens) == [6, 7, 9, 3]
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    for bad in ([-1, 2], [p.n_pages, 2], [0, -1], [0, p.n_pages + 1]):
        before = {f: p.g[f].view.clone() for f in p.FIELDS}
        p.g["ends"].view.copy_(torch.tensor(bad))
        cu, _, slots = p.call(mbd, [0, 8, 12, 3], 30)
        assert not cu.any() and (slots == -1).all()
        for f in ("table", "ring", "lens", "seen"):
            assert torch.equal(p.g[f].view, before[f]), f
        assert p.g["ends"].view.tolist() == bad
        p.g["ends"].view.copy_(before["ends"])
        assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    p = Pages(rng, [8, 8, 8], 4, 3, 1).device()      # every sequence names the same two pages, and all give them up
    p.g["table"].view.view(3, 3)[:, :2] = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    p.g["ends"].view.copy_(torch.tensor([6, 4]))
    cu, _, _ = p.call(mbd, [0, 0, 0], 0)
    assert p.g["ends"].view.tolist() == [6, 7] and p.g["lens"].view.tolist() == [0, 0, 0]
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    p = Pages(rng, [3, 0], 4, 3, 4).device()         # a free page that is none of the pool's
    p.g["ring"].view.fill_(1 << 30)
    _, _, slots = p.call(mbd, [3, 4], 6)
    assert list(slots) == [-1] * 6 and mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX


def test_resize_without_optional_outputs(mbd):
    rng = np.random.default_rng(3)
    p = Pages(rng, [5, 70, 0], 16, 8, 9).device()
    seen = p.g["seen"].view.clone()
    got = p.call(mbd, [6, 0, 33], 40, outputs=False, seen=False)
    cu, _, _ = p.resize([6, 0, 33], 40)
    np.testing.assert_array_equal(got[0], cu)
    assert torch.equal(p.g["seen"].view, seen)
    for f in ("table", "ring", "ends", "lens"):
        np.testing.assert_array_equal(p.g[f].numpy(np.int32), getattr(p, f).reshape(-1), f)


def test_resize_positions_are_slots_where_nothing_was_evicted(mbd):
    rng = np.random.default_rng(4)
    p = Pages(rng, [5, 70], 16, 8, 9).device()
    _, positions, _ = p.call(mbd, [7, 72], 4, seen=False)
    assert list(positions) == [5, 6, 70, 71]


def test_resize_captured(mbd):
    """A captured step replayed while the wanted lengths on the device change."""
    rng = np.random.default_rng(5)
    n, rows = 50, 400
    p = Pages(rng, rng.integers(0, 90, n), 8, 12, 700).device()
    want = torch.zeros(n, dtype=torch.int32, device="cuda")
    cu, pos = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(rows, dtype=torch.int32, device="cuda")
    slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
    d = {f: g.view for f, g in p.g.items()}
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mbd.kv_cache_resize(d["table"], p.width, p.page, p.n_pages, d["ring"], d["ends"], d["lens"], want, n, cu, pos, slots,
                            rows, d["seen"])
    for _ in range(5):
        w = np.where(rng.random(n) < 0.3, rng.integers(0, 97, n), np.minimum(p.lens + 1, 96)).astype(np.int32)
        want.copy_(torch.from_numpy(w))
        g.replay()
        torch.cuda.synchronize()
        for got, e in zip((cu, pos, slots), p.resize(w, rows)):
            np.testing.assert_array_equal(got.cpu().numpy(), e)
        p.check()


# ------------------------------------------------------------------------------------------------ rotary positions

def run_rotary(mbd, rng, n, heads, d, dim, layout, scaling="none", far=5000, gap=0, in_place=True, positions="random", **kw):
    turns, amp = mbd.rotary_table(dim, scaling=scaling, **kw)
    width = heads * d + gap
    x = bits(rng, n, width)
    pos = np.arange(n) if positions is None else rng.integers(-far if positions == "negative" else 0, far + 1, n).astype(np.int32)
    xg = Guarded(torch, x.size, torch.int16, fill=x.view(np.int16))
    og = xg if in_place else Guarded(torch, n * heads * d, torch.int16)
    mbd.rotary(og.view, width if in_place else 0, xg.view, width, torch.frombuffer(turns, dtype=torch.int64).cuda(), amp,
               None if positions is None else up(pos), n, heads, d, dim, layout)
    torch.cuda.synchronize()
    xg.check_guards("x")
    og.check_guards("out")
    got = og.numpy(np.uint16)
    if in_place:
        got = got.reshape(n, width)
        np.testing.assert_array_equal(got[:, heads * d:], x[:, heads * d:])
        got = got[:, :heads * d]
    else:
        np.testing.assert_array_equal(xg.numpy(np.uint16), x.reshape(-1))
    got = np.ascontiguousarray(got).reshape(n, heads, d)
    rows = np.ascontiguousarray(x[:, :heads * d])
    np.testing.assert_array_equal(got[..., dim:], rows.reshape(n, heads, d)[..., dim:])
    want, tol = ref.rotary(rows, pos, list(turns), amp, heads, d, dim, layout)
    check_close(wl.bf16_bits_to_f32(got), want, tol, "rotary")


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("n,heads,d,dim", [(1, 1, 16, 16), (3, 14, 128, 128), (128, 40, 128, 128), (5, 32, 64, 32),
                                           (700, 3, 96, 48), (2, 5, 80, 16), (9, 2, 256, 256), (4, 130, 112, 96),
                                           (1, 2, 4096, 4096), (2, 3, 4096, 16), (2000, 17, 64, 64)])
def test_rotary(mbd, n, heads, d, dim, layout, in_place):
    run_rotary(mbd, np.random.default_rng(n), n, heads, d, dim, layout, gap=64 if n % 2 else 0, in_place=in_place)


@pytest.mark.parametrize("scaling,kw", [("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
                                        ("llama3", dict(base=5e5, factor=8.0, original=8192)),
                                        ("yarn", dict(base=1e6, factor=4.0, original=32768)),
                                        ("factors", dict(factors=1 + np.arange(64) / 9, amplitude=1.19))])
@pytest.mark.parametrize("far", [100, 131071, (1 << 31) - 1])
def test_rotary_scaled_and_far(mbd, scaling, kw, far):
    """Angles of far positions are as good as those of near ones."""
    run_rotary(mbd, np.random.default_rng(far % 1000), 50, 10, 128, 128, "half", scaling, far, **kw)


def test_rotary_positions(mbd):
    """Rows as positions where none are given; positions before 0 turn back."""
    rng = np.random.default_rng(6)
    run_rotary(mbd, rng, 300, 4, 64, 64, "half", positions=None)
    run_rotary(mbd, rng, 300, 4, 64, 64, "interleaved", positions="negative", far=1 << 30)


def test_rotary_of_infinite_and_nan_elements(mbd):
    """They stay with their pair: nothing else of the row changes."""
    turns, amp = mbd.rotary_table(64)
    x = torch.randn(2, 128, device="cuda").bfloat16()
    y = x.clone()
    y[0, 3], y[1, 64 + 40] = float("inf"), float("nan")
    t = torch.frombuffer(turns, dtype=torch.int64).cuda()
    pos = torch.tensor([7, 9], dtype=torch.int32, device="cuda")
    for z in (x, y):
        mbd.rotary(z, 128, z, 128, t, amp, pos, 2, 2, 64, 64)
    torch.cuda.synchronize()
    same = x == y
    assert int((~same).sum()) == 4 and not same[0, 3] and not same[0, 35] and not same[1, 104] and not same[1, 72]


def test_rotary_keeps_lengths_and_inner_products(mbd):
    """A pair's length stays, and the product of a query and a key depends on the distance of their positions alone."""
    turns, amp = mbd.rotary_table(128)
    t = torch.frombuffer(turns, dtype=torch.int64).cuda()
    g = torch.Generator("cuda").manual_seed(1)
    q, k = (torch.randn(1, 128, device="cuda", generator=g).bfloat16().repeat(4, 1) for _ in range(2))
    at = torch.tensor([3, 1000, 100000, 2000000000], dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(q), torch.empty_like(k)
    mbd.rotary(a, 0, q, 0, t, amp, at, 4, 1, 128, 128)
    mbd.rotary(b, 0, k, 0, t, amp, at + 77, 4, 1, 128, 128)
    dots = (a.double() * b.double()).sum(1)
    # each of the 256 factors is rounded to bf16 once: 2^-8 of |q||k| together with Cauchy-Schwarz, twice
    assert (dots - dots[0]).abs().max() <= 4 * 2.0 ** -8 * q[0].double().norm() * k[0].double().norm()
    torch.testing.assert_close(a.double().norm(dim=1), q.double().norm(dim=1), rtol=2.0 ** -8, atol=0)
