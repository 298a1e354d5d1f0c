"""Pages and slots where a call is refused or its input is bad: what the call must leave as it is."""
import numpy as np
import pytest

from tests.test_kv_gpu import mbd  # noqa: F401  (mbd is the fixture)
from tests.test_step_gpu import Pages

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def emptied(rng, spare):
    """Two rows without a token whose tokens were all evicted, so that they have seen some, a fresh one, and one in use."""
    p = Pages(rng, [0, 0, 0, 5], 4, 8, spare)
    p.seen[:] = [4000, 77, 0, 9]
    return p.device()


@pytest.mark.parametrize("room", [6, 3000])   # one CTA, and a cluster of them
def test_tokens_seen_of_empty_rows(mbd, room):
    """They stay through a refusal for want of pages or rows, a length out of range and bad ends, the next grant counts on from
    them, and a wanted length of 0 resets them."""
    rng = np.random.default_rng(0)
    mbd.device_error_flags(clear=True)
    p = emptied(rng, 0)
    p.step(mbd, [1, 2, 3, 6], room)                  # no page is free (and seven rows are asked for)
    assert list(p.seen) == [4000, 77, 0, 10 if room >= 7 else 9] and list(p.lens) == [0, 0, 0, 6 if room >= 7 else 5]
    p = emptied(rng, 9)
    p.step(mbd, [1, 2, 3, 5], 0)                     # no rows
    assert list(p.seen) == [4000, 77, 0, 9]
    assert mbd.device_error_flags() == 0
    p = emptied(rng, 9)
    p.step(mbd, [33, -1, 1, 5], room)                # lengths out of range
    assert list(p.seen) == [4000, 77, 1, 9] and list(p.lens) == [0, 0, 1, 5]
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    p = emptied(rng, 9)
    p.g["ends"].view.copy_(torch.tensor([-1, 2]))
    p.call(mbd, [1, 0, 3, 6], room)
    assert p.g["seen"].view.tolist() == [4000, 77, 0, 9]
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    p = emptied(rng, 9)
    _, positions, _ = p.resize([2, 0, 0, 0], room)   # (the reference)
    assert list(positions[:2]) == [4000, 4001] and list(p.seen) == [4002, 0, 0, 0]
    p = emptied(rng, 9)
    p.step(mbd, [2, 0, 0, 0], room)
    assert mbd.device_error_flags() == 0


@pytest.mark.parametrize("room", [6, 3000])
@pytest.mark.parametrize("page", [-1, -7, 11, 1 << 30])
def test_given_up_pages_outside_the_pool(mbd, page, room):
    """Flagged in the call that gives them up, which hands them on to the ring as they are; so is the call that takes one."""
    rng = np.random.default_rng(1)
    p = Pages(rng, [20, 5], 4, 5, 4)
    assert p.n_pages == 11
    p.table[0, 3] = page
    p.device()
    mbd.device_error_flags(clear=True)
    p.step(mbd, [4, 5], room)
    assert mbd.device_error_flags(clear=True) == mbd.DEVERR_BAD_INDEX
    assert page in p.ring
    p.step(mbd, [4, 6], room)                        # nothing bad is touched
    assert mbd.device_error_flags() == 0
