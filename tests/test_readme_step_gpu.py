"""README's example of the front of a serving step, run as it stands there."""
import os
import re

import numpy as np
import pytest

import workloads as wl
from oracle import step as ref
from oracle.kv_cache import check_close
from tests.test_kv_gpu import bits, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_serving_step(mbd):
    block = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "kv_cache_resize" in b]
    assert len(block) == 1
    rng = np.random.default_rng(2)
    hq, hkv, B, rows = 4, 2, 3, 400
    p = ref.Pages(rng, [0] * B, 16, 20, 60)
    qkv = bits(rng, rows, (hq + 2 * hkv) * 128)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    want = np.array([200, 0, 77], np.int32)
    names = dict(mbd=mbd, torch=torch, table=up(p.table), pages_per_seq=20, n_pages=p.n_pages, free_pages=up(p.ring), free_ends=up(p.ends),
                 lens=up(p.lens), want_lens=up(want), B=B, cu_tokens=i32(B + 1), positions=i32(rows),
                 slots=torch.zeros(rows, dtype=torch.int64, device="cuda"), rows=rows, tokens_seen=up(p.seen), qkv=up(qkv), hq=hq,
                 hkv=hkv, out=torch.zeros(rows, hq * 128, dtype=torch.bfloat16, device="cuda"))
    exec(block[0], names)
    torch.cuda.synchronize()
    cu, positions, slots = p.resize(want, rows)
    for got, e in (("cu_tokens", cu), ("positions", positions), ("slots", slots), ("table", p.table), ("lens", p.lens)):
        np.testing.assert_array_equal(names[got].cpu().numpy(), e)
    x = names["qkv"].cpu().numpy().view(np.uint16)
    part = lambda a, b: np.ascontiguousarray(x[:277, a * 128:b * 128])
    e = ref.prompt(part(0, 4), part(4, 6), part(6, 8), cu, hq, hkv, 128, 128 ** -0.5)
    got = wl.bf16_bits_to_f32(names["out"].cpu().view(torch.int16).numpy().view(np.uint16)[:277]).reshape(277, hq, 128)
    check_close(got, e[0], e[2], "prompts")
