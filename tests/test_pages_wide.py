"""Page tables and slot maps of many tokens (more than 65536 entries in the map, which threads write eight at a time),
against the walk over the requests.  Whole numbers: equal or wrong."""
import random

import pytest

from deepseek_sparse_attention_lightning_gb300 import build
from test_pages import _check, _state

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def _wave(batch, longest, add, ended, seed):
    """Changes of a wave, the tokens it brings, and a state that has pages enough for it."""
    rng = random.Random(seed)
    change = [-1 - rng.randint(0, 5) if rng.random() < ended else rng.choice((0, rng.randint(0, add), add)) for _ in range(batch)]
    change[0] = add
    new = sum(max(0, n) for n in change)
    max_pages = -(-(longest + add) // 64) + 1
    return change, new, _state(rng, batch, max_pages, new // 64 + batch + 3, longest)


# The last three: more than 4096 requests, whose offsets and lengths are read from memory.
@pytest.mark.parametrize("batch,longest,add,ended", [
    (1, 100, 70001, 0.0), (300, 200, 2000, 0.2), (1500, 90, 150, 0.3), (4096, 64, 60, 0.1), (4097, 64, 60, 0.1), (6000, 65, 40, 0.2),
    (20001, 70, 13, 0.4),
])
@pytest.mark.parametrize("apart", [False, True])
def test_waves(batch, longest, add, ended, apart):
    change, new, state = _wave(batch, longest, add, ended, batch + add)
    assert new > 65536
    _check(change, state, new, apart)
    _check(change, state, new + 37, apart, offset=3)       # slots off 32 bytes, and some behind the last token
    _check(change, state, new + 5, apart, offset=4)        # ... 16-byte aligned
    _check(change, state, 2 * new + 1, apart)              # whole runs behind the last token


@pytest.mark.parametrize("batch,add", [(128, 1), (5000, 2), (17, 300)])
def test_a_step_in_a_map_made_for_waves(batch, add):
    change, new, state = _wave(batch, 3000 if batch < 1000 else 70, add, 0.1, batch)
    for tokens in (65537, 200003):
        _check(change, state, tokens, False)
        _check(change, state, tokens, True, offset=1)


@pytest.mark.parametrize("batch,longest,add", [(300, 200, 2000), (6000, 65, 40)])
@pytest.mark.parametrize("edit", ["free ids", "table ids", "ended ids", "count", "too few pages", "too few slots", "long"])
def test_bad_state_and_refusals(batch, longest, add, edit):
    change, new, (lens, table, free, count, pages) = _wave(batch, longest, add, 0.2, 7 + batch)
    rng, tokens = random.Random(3), new
    if edit == "free ids":
        for i in range(0, count, 13):
            free[i] = rng.choice((-7, pages, 2 ** 31 - 1, -2 ** 31))
    elif edit == "table ids":       # of the pages that new tokens begin in: a run of slots with one good page
        for r in range(0, batch, 5):
            if lens[r] % 64 and change[r] > 0:
                table[r][lens[r] // 64] = rng.choice((-1, pages, pages + 9))
    elif edit == "ended ids":
        for r in range(batch):
            if change[r] < 0 and lens[r] and r % 2:
                table[r][0] = rng.choice((-1, pages))
    elif edit == "count":
        count = pages + 1
        free = [i % pages for i in range(pages)]
    elif edit == "too few pages":
        count //= 3
    elif edit == "too few slots":
        tokens = max(65537, new * 2 // 3)
    else:
        for r in range(0, batch, 11):
            lens[r] = len(table[r]) * 64 + 1
    assert tokens > 65536
    for apart in (False, True):
        _check(change, (lens, table, free, count, pages), tokens, apart, offset=3 if apart else 0)
