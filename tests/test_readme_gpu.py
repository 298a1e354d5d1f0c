"""README's example of a decode step over the key-value cache, run as it stands there."""
import os
import re

import numpy as np
import pytest

from tests.test_kv_gpu import Cache, bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_decode_step(mbd):
    """Steps on both sides of evictions: each new token is stored under its own position, and the newest 256 stay."""
    block = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "kv_cache_append" in b]
    assert len(block) == 1
    rng = np.random.default_rng(1)
    hq, hkv, d, lens = 4, 1, 128, np.array([2047, 2046, 100], np.int32)
    c = Cache(rng, [2064] * 3, hkv, d, 16, "fp8", "dynamic", fill=False)
    c.lens = lens
    c.device(mbd)
    B = len(lens)
    names = dict(mbd=mbd, n_pages=c.n_pages, n_kv_heads=hkv, hq=hq, hkv=hkv, B=B, pages_per_seq=c.width, table=c.table_d,
                 lens=c.lens_d, k_pool=c.g["k"].view, v_pool=c.g["v"].view, k_scale=c.g["ks"].view,
                 v_scale=c.g["vs"].view, weight=c.g["weight"].view, position=c.g["position"].view,
                 new_lens=torch.zeros(B, dtype=torch.int32, device="cuda"), positions=c.lens_d.clone(),
                 out=torch.empty(B, hq * d, dtype=torch.bfloat16, device="cuda"),
                 workspace=torch.empty(1 << 26, dtype=torch.uint8, device="cuda"))
    # What was there before the first step: slots in the order of the tokens, the older ones with the more weight.
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    rows = up(bits(rng, int(cu[-1]), hkv * d))
    mbd.kv_cache_append(c.c, rows, rows, 0, c.table_d, c.width, c.lens_d, B, int(cu[-1]), up(cu))
    w = names["weight"].view(c.n_pages, -1)
    w.copy_(torch.where(torch.isnan(w), w, 9.0))
    for step in range(20):
        c.lens_d += 1
        names["qkv"] = up(bits(rng, B, (hq + 2 * hkv) * d))
        exec(block[0], names)
        torch.cuda.synchronize()
        at = names["position"].view(c.n_pages, hkv, 16).cpu().numpy()
        for b in range(B):
            n, newest = int(names["new_lens"][b]), int(names["positions"][b])
            assert newest == lens[b] + step and n == min(lens[b] + step + 1, 2048)
            p, _, s = c.at(b, np.arange(n))
            held = at[p, 0, s]
            assert len(set(held)) == n and set(range(max(0, newest - 255), newest + 1)) <= set(held.tolist())
        c.lens_d.copy_(names["new_lens"])
        names["positions"] += 1
