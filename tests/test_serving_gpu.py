"""A serving step's operators together, as a program calls them: pages and slots, rotary positions, the attention of whole prompts,
append, decode attention with the accumulation of weights, and eviction, on one stream without a synchronisation inside a step,
against the NumPy references step by step. Also the entry points from several host threads and streams."""
import numpy as np
import pytest

import workloads as wl
from oracle import kv_cache as kvref
from oracle import kv_nvfp4 as nvref
from oracle import step as ref
from oracle.kv_cache import check_close
from tests.test_host_threads_gpu import in_threads
from tests.test_kv_gpu import bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def as_bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


class Server:
    """The GPU's side of a cache and its pages, and the references of both, over the same page numbers."""

    def __init__(self, mbd, rng, n, width, page, hkv, d, fmt, mode):
        self.mbd, self.n, self.width, self.page, self.hkv, self.d = mbd, n, width, page, hkv, d
        self.pages = ref.Pages(rng, [0] * n, page, width, n * width // 2)
        n_pages = self.pages.n_pages
        make = (lambda *a, **k: nvref.Cache(*a, **k)) if fmt == "nvfp4" else (lambda *a, **k: kvref.Cache(*a, fmt, mode, **k))
        self.cache = make(rng, [0] * n, hkv, d, page, spare=n_pages, width=width, fill=False)
        self.cache.table = self.pages.table                # one table for both
        c = self.cache
        dev = lambda a: None if a is None else up(a)
        self.t = dict(k=dev(c.k_raw), v=dev(c.v_raw), ks=dev(c.ks), vs=dev(c.vs), weight=dev(c.weight), position=dev(c.position))
        self.p = {f: up(getattr(self.pages, f)) for f in ("table", "ring", "ends", "lens", "seen")}
        self.c = mbd.kv_cache(self.t["k"], self.t["v"], n_pages, page, hkv, d, fmt, mode, self.t["ks"], self.t["vs"],
                              self.t["weight"], self.t["position"])

    def resize(self, want, rows, cu, positions, slots):
        self.mbd.kv_cache_resize(self.p["table"], self.width, self.page, self.pages.n_pages, self.p["ring"], self.p["ends"],
                                 self.p["lens"], want, self.n, cu, positions, slots, rows, self.p["seen"])

    def check(self, what):
        for f, t in self.p.items():
            np.testing.assert_array_equal(t.cpu().numpy().reshape(-1), getattr(self.pages, f).reshape(-1), f"{what}: {f}")
        for name, a in dict(k=self.cache.k_raw, v=self.cache.v_raw, ks=self.cache.ks, position=self.cache.position).items():
            if a is not None:
                got = self.t[name].cpu().numpy()
                assert got.reshape(-1).view(a.dtype).tobytes() == np.ascontiguousarray(a).tobytes(), f"{what}: {name}"


@pytest.mark.parametrize("fmt,mode", [("bf16", "static"), ("fp8", "dynamic"), ("nvfp4", "static")])
@pytest.mark.parametrize("hq,hkv,d,dim,layout", [(8, 2, 64, 32, "interleaved"), (6, 2, 128, 128, "half")])
def test_serving(mbd, fmt, mode, hq, hkv, d, dim, layout):
    """Prompts come in, all sequences are decoded, some end and others take their rows, full ones are evicted from."""
    rng = np.random.default_rng(21)
    n, page, width, budget, recent = 5, 8, 12, 48, 8
    room, cap = 160, page * width
    s = Server(mbd, rng, n, width, page, hkv, d, fmt, mode)
    turns, amp = mbd.rotary_table(dim, 1e4, "yarn", 4.0, 64)
    turns_d = torch.frombuffer(turns, dtype=torch.int64).cuda()
    w = (hq + 2 * hkv) * d
    i32 = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")
    cu, positions, slots, new_lens = i32(n + 1), i32(room), torch.zeros(room, dtype=torch.int64, device="cuda"), i32(n)
    nb = mbd.paged_attention_workspace_bytes(s.c, width, n, hq, True)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    mbd.device_error_flags(clear=True)
    ended = evicted = prompts = 0
    for step in range(40):
        lens = s.pages.lens.copy()
        # Prompts only into empty rows, in steps of their own: their attention is over their own rows.
        fresh = [b for b in range(n) if lens[b] == 0]
        is_prompt = bool(fresh) and step % 5 == 0
        if is_prompt:
            want = lens.copy()
            for b in fresh:
                want[b] = rng.integers(1, 40)
            prompts += 1
        else:
            want = np.where(lens > 0, lens + 1, 0)
            if step % 9 == 8 and lens.any():
                want[int(rng.choice(np.flatnonzero(lens)))] = 0
                ended += 1
        qkv = bits(rng, room, w, sigma=1.5)
        x, want_d = up(qkv), up(want.astype(np.int32))
        out, lse = torch.zeros(room, hq * d, dtype=torch.bfloat16, device="cuda"), torch.zeros(room, hq, device="cuda")
        decode_out, decode_lse = torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, hq, device="cuda")
        torch.cuda.synchronize()
        s.resize(want_d, room, cu, positions, slots)
        mbd.rotary(x, w, x, w, turns_d, amp, positions, room, hq + hkv, d, dim, layout)
        mbd.kv_cache_append(s.c, x[:, hq * d:], x[:, (hq + hkv) * d:], w, s.p["table"], width, s.p["lens"], n, room, cu, positions)
        if is_prompt:
            mbd.prompt_attention(out, x, w, x[:, hq * d:], x[:, (hq + hkv) * d:], w, cu, n, room, hq, hkv, d, d ** -0.5, 0, lse)
        cu_r, pos_r, slots_r = s.pages.resize(want, room)
        rows = int(cu_r[-1])
        if not is_prompt:
            # One row a sequence: the rows of those that are decoded, and any row for those that are empty (nothing in view).
            pick = torch.from_numpy(np.minimum(cu_r[:-1], room - 1).astype(np.int64)).cuda()
            q = x[pick].contiguous()
            mbd.paged_attention_decode(decode_out, q, w, s.c, s.p["table"], width, s.p["lens"], n, hq, d ** -0.5, 0, decode_lse, True, ws, nb)
        # ---- the references
        got = [t.cpu().numpy() for t in (cu, positions, slots)]
        for g, e, what in zip(got, (cu_r, pos_r, slots_r), ("cu", "positions", "slots")):
            np.testing.assert_array_equal(g, e, f"step {step} {what}")
        rot, tol = ref.rotary(np.ascontiguousarray(qkv[:rows, :(hq + hkv) * d]), pos_r[:rows], list(turns), amp, hq + hkv, d, dim, layout)
        xb = as_bits(x)                                     # what the other operators were given: the GPU's own rounding
        check_close(wl.bf16_bits_to_f32(xb[:rows, :(hq + hkv) * d]).reshape(rows, hq + hkv, d), rot, tol, f"step {step} rotary")
        np.testing.assert_array_equal(xb[:, (hq + hkv) * d:], qkv[:, (hq + hkv) * d:])
        s.cache.lens = s.pages.lens
        for b in range(n):
            a, e = cu_r[b], cu_r[b + 1]
            if e > a:
                at = np.arange(s.pages.lens[b] - (e - a), s.pages.lens[b])
                s.cache.store(b, at, xb[a:e, hq * d:(hq + hkv) * d].reshape(-1, hkv, d), xb[a:e, (hq + hkv) * d:].reshape(-1, hkv, d),
                              pos_r[a:e])
        if is_prompt:
            part = lambda lo, hi: np.ascontiguousarray(xb[:rows, lo * d:hi * d])
            e = ref.prompt(part(0, hq), part(hq, hq + hkv), part(hq + hkv, hq + 2 * hkv), cu_r, hq, hkv, d, d ** -0.5)
            check_close(wl.bf16_bits_to_f32(as_bits(out)[:rows]).reshape(rows, hq, d), e[0], e[2], f"step {step} prompts")
            check_close(lse.cpu().numpy()[:rows], e[1], e[3], f"step {step} prompts' lse")
            assert not out[rows:].any()
        else:
            e = s.cache.attend(as_bits(q)[:, :hq * d].copy(), hq, d ** -0.5, 0, True)
            check_close(wl.bf16_bits_to_f32(as_bits(decode_out)).reshape(n, hq, d), e[0], e[2], f"step {step} decode")
            check_close(decode_lse.cpu().numpy(), e[1], e[3], f"step {step} decode lse")
            got = s.t["weight"].cpu().numpy().reshape(s.cache.weight.shape)
            live = ~np.isnan(s.cache.weight)
            check_close(got[live], e[4][live], e[5][live], f"step {step} weights")
            s.cache.weight[live] = got[live]                # the choice of the eviction is on these very weights
        s.check(f"step {step}")
        if int(s.pages.lens.max()) > budget + 8:
            mbd.kv_cache_evict(s.c, new_lens, s.p["lens"], s.p["table"], width, n, budget, recent)
            s.resize(new_lens, 0, cu, None, None)           # the pages behind the budget go back to the ring
            left = s.cache.evict(budget, recent)
            s.pages.resize(left, 0)
            torch.cuda.synchronize()
            s.check(f"step {step} eviction")
            evicted += 1
    assert ended >= 2 and evicted >= 2 and prompts >= 2 and mbd.device_error_flags() == 0
    assert (s.pages.seen[s.pages.lens > 0] >= s.pages.lens[s.pages.lens > 0]).all()


def test_captured_decode_step(mbd):
    """One captured graph of a decode step (resize, rotary, append, attention), replayed while the cache grows, gives the bits of
    the calls made one by one."""
    rng = np.random.default_rng(22)
    n, page, width, hq, hkv, d = 6, 16, 6, 8, 2, 128
    w = (hq + 2 * hkv) * d
    seed = int(rng.integers(1 << 30))
    turns, amp = mbd.rotary_table(d)
    turns_d = torch.frombuffer(turns, dtype=torch.int64).cuda()
    rows = [up(bits(rng, n, w)) for _ in range(40)]

    def fresh():
        s = Server(mbd, np.random.default_rng(seed), n, width, page, hkv, d, "nvfp4", "static")
        i32 = lambda k: torch.zeros(k, dtype=torch.int32, device="cuda")
        return s, dict(cu=i32(n + 1), pos=i32(n), slots=torch.zeros(n, dtype=torch.int64, device="cuda"), want=i32(n),
                       x=torch.zeros(n, w, dtype=torch.int16, device="cuda"), out=torch.zeros(n, hq * d, dtype=torch.bfloat16, device="cuda"))

    def call(s, b, ws, nb):
        s.resize(b["want"], n, b["cu"], b["pos"], b["slots"])
        mbd.rotary(b["x"], w, b["x"], w, turns_d, amp, b["pos"], n, hq + hkv, d, d)
        mbd.kv_cache_append(s.c, b["x"][:, hq * d:], b["x"][:, (hq + hkv) * d:], w, s.p["table"], width, s.p["lens"], n, n, b["cu"], b["pos"])
        mbd.paged_attention_decode(b["out"], b["x"], w, s.c, s.p["table"], width, s.p["lens"], n, hq, d ** -0.5, 0, None, False, ws, nb)

    (a, ab), (g, gb) = fresh(), fresh()
    nb = mbd.paged_attention_workspace_bytes(a.c, width, n, hq)
    ws = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(g, gb, ws[1], nb)
    for step, x in enumerate(rows):
        for s, b in ((a, ab), (g, gb)):
            b["x"].copy_(x)
            b["want"].copy_(s.p["lens"] + 1)
        call(a, ab, ws[0], nb)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ab["out"], gb["out"]) and torch.equal(ab["slots"], gb["slots"]), f"step {step}"
    assert a.p["lens"].tolist() == [40] * n and torch.equal(a.t["k"], g.t["k"])


def test_from_host_threads(mbd):
    """Prompts of every head size, resizes of few and of many sequences and NVFP4 attention from host threads on streams of their
    own, where launches depend on attributes of the kernels: each gives the bits of the call made alone."""
    rng = np.random.default_rng(23)
    jobs, checks = [], []
    for d in (64, 128, 256):
        n = 300
        x = up(bits(rng, n, 4 * d))
        cu, out = up(np.array([0, 100, n], np.int32)), torch.zeros(n, 2 * d, dtype=torch.int16, device="cuda")
        call = lambda s=None, x=x, cu=cu, out=out, d=d, n=n: mbd.prompt_attention(out, x, 4 * d, x[:, 2 * d:], x[:, 3 * d:], 4 * d, cu, 2, n, 2, 1,
                                                                                  d, 0.1, 0, None, s)
        jobs.append((call, out))
    for n in (4, 8192):
        p = ref.Pages(rng, [3] * n, 4, 2, n)
        t = {f: up(getattr(p, f)) for f in ("table", "ring", "ends", "lens", "seen")}
        want, cu, slots = up(p.lens), torch.zeros(n + 1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int64, device="cuda")
        call = lambda s=None, p=p, t=t, want=want, cu=cu, slots=slots, n=n: mbd.kv_cache_resize(
            t["table"], 2, 4, p.n_pages, t["ring"], t["ends"], t["lens"], want, n, cu, None, slots, n, t["seen"], s)
        jobs.append((call, cu))
    c = nvref.Cache(rng, [200, 77], 2, 128, 16)
    t = [up(a) for a in (c.k_raw, c.v_raw, c.ks, c.vs, c.table, c.lens)]
    cache = mbd.kv_cache(t[0], t[1], c.n_pages, 16, 2, 128, "nvfp4", "static", t[2], t[3])
    q, out = up(bits(rng, 2, 512)), torch.zeros(2, 512, dtype=torch.int16, device="cuda")
    nb = mbd.paged_attention_workspace_bytes(cache, c.width, 2, 4)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    jobs.append((lambda s=None: mbd.paged_attention_decode(out, q, 0, cache, t[4], c.width, t[5], 2, 4, 0.1, 0, None, False, ws, nb, s), out))
    for call, result in jobs:
        call()
        torch.cuda.synchronize()
        checks.append(result.clone())

    def body(call):
        stream = torch.cuda.Stream()

        def run():
            for i in range(300):
                call(stream)
            stream.synchronize()
        return run

    in_threads(*[body(call) for call, _ in jobs])
    torch.cuda.synchronize()
    for (_, result), want in zip(jobs, checks):
        assert torch.equal(result, want)
    assert mbd.device_error_flags() == 0
