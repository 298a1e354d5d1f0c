"""README's step that decodes some sequences and starts others, run as it stands there."""
import re

import numpy as np
import pytest

import workloads as wl
from oracle import step as ref
from oracle.kv_cache import check_close
from tests.test_kv_gpu import bits, mbd, up  # noqa: F401  (mbd is the fixture)
from tests.test_readme_step_gpu import README
from tests.test_serving_gpu import Server, as_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,mode", [("bf16", "static"), ("fp8", "dynamic"), ("nvfp4", "static")])
def test_readme_mixed_step(mbd, fmt, mode):
    blocks = re.findall(r"```python\n(.*?)```", open(README).read(), re.S)
    front, = (b for b in blocks if "kv_cache_resize" in b)
    append, = (b for b in blocks if "kv_cache_append" in b)
    append = re.search(r"mbd\.kv_cache_append\(.*?\)\n", append, re.S).group(0)
    mixed, = (b for b in blocks if "newest" in b)
    rng = np.random.default_rng(3)
    hq, hkv, d, B, rows = 4, 2, 128, 5, 300
    s = Server(mbd, rng, B, 12, 16, hkv, d, fmt, mode)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    w = (hq + 2 * hkv) * d
    names = dict(mbd=mbd, torch=torch, table=s.p["table"], pages_per_seq=12, n_pages=s.pages.n_pages, free_pages=s.p["ring"],
                 free_ends=s.p["ends"], lens=s.p["lens"], B=B, cu_tokens=i32(B + 1), positions=i32(rows), cache=s.c, hq=hq, hkv=hkv,
                 slots=torch.zeros(rows, dtype=torch.int64, device="cuda"), rows=rows, tokens_seen=s.p["seen"],
                 step_out=torch.zeros(B, hq * d, dtype=torch.bfloat16, device="cuda"))
    nb = mbd.paged_attention_workspace_bytes(s.c, 12, B, hq)
    names.update(workspace=torch.empty(nb, dtype=torch.uint8, device="cuda"), nbytes=nb)
    # the append's rows are a step's, with their offsets: as README says of the front of a step
    append = append.replace("lens, B, B,", "lens, B, rows, cu_tokens,")
    assert "rows, cu_tokens" in append
    mbd.device_error_flags(clear=True)
    for want, decoded in (([90, 0, 37, 0, 0], []), ([91, 50, 38, 0, 0], [0, 2]), ([92, 51, 0, 129, 0], [0, 1]), ([93, 52, 3, 130, 1], [0, 1, 3])):
        names.update(qkv=up(bits(rng, rows, w)), want_lens=up(np.array(want, np.int32)), decoded=decoded,
                     out=torch.zeros(rows, hq * d, dtype=torch.bfloat16, device="cuda"))
        for code in (front, append, mixed):
            exec(code, names)
        torch.cuda.synchronize()
        cu, positions, _ = s.pages.resize(want, rows)
        n = int(cu[-1])
        x = as_bits(names["qkv"])
        k, v = (x[:, a * d:b * d].reshape(rows, hkv, d) for a, b in ((hq, hq + hkv), (hq + hkv, hq + 2 * hkv)))
        s.cache.lens = s.pages.lens
        for b in range(B):
            a, e = cu[b], cu[b + 1]
            if e > a:
                s.cache.store(b, np.arange(s.pages.lens[b] - (e - a), s.pages.lens[b]), k[a:e], v[a:e], positions[a:e])
        part = lambda a, b: np.ascontiguousarray(x[:n, a * d:b * d])
        e, _, tol, _ = ref.prompt(part(0, hq), part(hq, hq + hkv), part(hq + hkv, hq + 2 * hkv), cu, hq, hkv, d, d ** -0.5)
        last = np.maximum(cu[1:] - 1, 0)
        f = s.cache.attend(x[last, :hq * d].copy(), hq, d ** -0.5)
        e, tol = e.copy(), tol.copy()
        for b in decoded:
            assert cu[b + 1] - cu[b] == 1
            e[cu[b]], tol[cu[b]] = f[0][b], f[2][b]
        got = wl.bf16_bits_to_f32(as_bits(names["out"])[:n]).reshape(n, hq, d)
        check_close(got, e, tol, f"{want}")
    assert mbd.device_error_flags() == 0
