"""Entry points called from several host threads at once, where a launch depends on an attribute of the kernel: every
call succeeds, and its results are those of the call made alone."""
import threading

import numpy as np
import pytest

import workloads as wl
from tests.test_kv_gpu import Cache, mbd, up  # noqa: F401  (mbd is the fixture)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def in_threads(*jobs):
    """Run the jobs at the same time, each on a host thread of its own; the first exception of any is raised here."""
    gate, failed = threading.Barrier(len(jobs)), []

    def body(job):
        try:
            gate.wait()
            job()
        except Exception as e:                            # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=body, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if failed:
        raise failed[0]


def test_evict_from_two_host_threads(mbd):
    """Evictions of two caches of very different width from two threads, on a stream each: every launch is accepted."""
    rng = np.random.default_rng(40)
    calls, caches = [], []
    for page, width in ((1024, 100), (1, 425984)):        # 50 KB and 208 KB of shared memory a CTA
        c = Cache(rng, [90] * 2, 1, 64, page, "bf16", width=width)
        c.device(mbd)
        new = torch.zeros(2, dtype=torch.int32, device="cuda")
        stream = torch.cuda.Stream()
        caches.append((c, new))

        def run(c=c, new=new, stream=stream):
            for i in range(4000):
                mbd.kv_cache_evict(c.c, new, c.lens_d, c.table_d, c.width, 2, 40, 8, stream)
                if i % 500 == 499:
                    stream.synchronize()
        calls.append(run)
    torch.cuda.synchronize()
    in_threads(*calls)
    torch.cuda.synchronize()
    assert mbd.device_error_flags() == 0
    for c, new in caches:                                 # each further call on the same lengths does the first's again
        assert new.tolist() == [40, 40]


def test_partial_norms_from_two_host_threads(mbd):
    """Norms over eight partials in rows of different width, which take 52 and 64 KB of shared memory a CTA."""
    calls, checks = [], []
    for hidden in (26000, 32768):
        parts = [up(wl.normal_bf16((2, hidden), 7, "x", salt=j)) for j in range(8)]
        start, weight = up(wl.normal_bf16((2, hidden), 8, "residual")), up(wl.weight_bf16(hidden, 9))
        residual, stream = torch.empty_like(start), torch.cuda.Stream()
        out = torch.empty(2, hidden, dtype=torch.bfloat16, device="cuda")

        def norm(out=out, residual=residual, parts=parts, weight=weight, hidden=hidden, stream=stream):
            mbd.fused_allreduce_add_rmsnorm(out, residual, parts, weight, 2, hidden, 1e-6, stream)

        def once(norm=norm, residual=residual, start=start, stream=stream):
            with torch.cuda.stream(stream):
                residual.copy_(start)
            norm()

        torch.cuda.synchronize()
        once()
        torch.cuda.synchronize()
        checks.append((out, out.clone(), residual, residual.clone()))

        def run(norm=norm, once=once, stream=stream):
            for i in range(60000):
                norm()
                if i % 500 == 499:
                    stream.synchronize()
            once()
        calls.append(run)
    in_threads(*calls)
    torch.cuda.synchronize()
    for out, want, residual, sums in checks:
        assert torch.equal(out, want) and torch.equal(residual, sums)
