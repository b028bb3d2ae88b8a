"""Page tables and slot maps from request lengths, against a walk over the requests on the host.  Whole numbers:
equal or wrong."""
import random

import pytest
import torch

from deepseek_sparse_attention_lightning_gb300 import api, build

FAKE = 0x7f0000000000


@pytest.fixture(scope="module")
def L():
    build.build()
    return api.lib()


def test_refusals_on_the_host(L):
    ok = dict(batch=2, max_pages=4, num_pages=9, change=FAKE, seq=FAKE, seq_out=FAKE, table=FAKE, free=FAKE, count=FAKE,
              count_out=FAKE, max_tokens=8, cu=FAKE, slots=FAKE)
    call = lambda **over: L.dsa_pages_update(*{**ok, **over}.values(), None)
    for bad in (dict(batch=0), dict(max_pages=0), dict(num_pages=0), dict(max_tokens=-1), dict(slots=None),
                dict(slots=FAKE + 2), *({k: v} for k in ("change", "seq", "seq_out", "table", "free", "count",
                                                         "count_out", "cu") for v in (None, FAKE + 1))):
        assert call(**bad) == 1, bad
    for bad in (dict(batch=65536), dict(num_pages=1 << 25), dict(max_pages=1 << 25)):
        assert call(**bad) == 2, bad


def walk(change, lens, table, free, count, max_tokens, num_pages):
    """What a call does, request by request: (lens, table, free, count, cu, slots, bad)."""
    lens, table, free = list(lens), [list(r) for r in table], list(free)
    cap, bad = len(table[0]) * 64, False
    cu, slots, asked, tokens, taken = [0], [-1] * max_tokens, 0, 0, 0
    if not 0 <= count <= num_pages:
        bad, count = True, min(max(count, 0), num_pages)
    back = []
    for r, n in enumerate(change):
        ln = max(0, lens[r])
        if n < 0:
            for i in range(min(-(-ln // 64), len(table[r]))):
                if 0 <= table[r][i] < num_pages:
                    back.append(table[r][i])
                else:
                    bad = True
                table[r][i] = -1
            lens[r] = 0
            cu.append(cu[-1])
            continue
        fits = ln + n <= cap
        need = -(-(ln + n) // 64) - -(-ln // 64) if fits else 0
        begin = tokens
        asked, tokens = asked + need, tokens + n
        cu.append(min(tokens, max_tokens))
        if not fits or (need and asked > count) or (n and tokens > max_tokens):
            bad, lens[r] = True, ln
            continue
        for j in range(need):
            page = free[count - 1 - (asked - need + j)]
            if not 0 <= page < num_pages:
                page, bad = -1, True
            table[r][-(-ln // 64) + j] = page
        taken = asked if need else taken
        for i in range(n):
            page = table[r][(ln + i) // 64]
            slots[begin + i] = page * 64 + (ln + i) % 64 if 0 <= page < num_pages else -1
            bad |= not 0 <= page < num_pages
        lens[r] = ln + n
    count -= taken
    for page in back:
        if count < num_pages:
            free[count] = page
            count += 1
        else:
            bad = True
    return lens, table, free, count, cu, slots, bad


def _state(rng, batch, max_pages, spare, longest):
    lens = [rng.randint(0, longest) for _ in range(batch)]
    held = [-(-n // 64) for n in lens]
    num_pages = sum(held) + spare
    ids = list(range(num_pages))
    rng.shuffle(ids)
    table, at = [], 0
    for n in held:
        table.append(ids[at:at + n] + [-1] * (max_pages - n))
        at += n
    return lens, table, ids[at:] + [-1] * at, spare, num_pages


def _call(change, state, max_tokens, apart, offset=0):
    lens, table, free, count, _ = state
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    seq, tab, fr, cnt = i32(lens), i32(table), i32(free), i32([count])
    cu = torch.full((len(lens) + 1,), 77, dtype=torch.int32, device="cuda")
    buf = torch.full((max_tokens + 8,), 77, dtype=torch.int32, device="cuda")
    slots = buf[offset:offset + max_tokens]
    so, co = (torch.full_like(seq, 77), torch.full_like(cnt, 77)) if apart else (None, None)
    api.dsa_pages_update(i32(change), seq, tab, fr, cnt, cu, slots, seqlens_out=so, free_count_out=co)
    err = api.dsa_get_device_error()
    assert (buf[:offset] == 77).all() and (buf[offset + max_tokens:] == 77).all()
    if apart:
        assert seq.tolist() == list(lens) and cnt.item() == count
    return ((so if apart else seq).tolist(), tab.tolist(), fr.tolist(), (co if apart else cnt).item(), cu.tolist(),
            slots.tolist(), err)


def _check(change, state, max_tokens, apart, offset=0):
    want = walk(change, *state[:4], max_tokens, state[4])
    got = _call(change, state, max_tokens, apart, offset)
    for name, a, b in zip(("lengths", "table", "free", "count", "offsets", "slots"), got, want):
        assert a == b, name
    assert got[6] == (5 if want[6] else 0)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,longest,add,ended", [
    (1, 0, 1, 0.0), (1, 64, 1, 0.0), (1, 130, 20000, 0.0), (3, 64, 64, 0.0), (33, 200, 3, 0.3), (128, 5000, 1, 0.1),
    (1024, 70, 1, 0.2), (1025, 70, 2, 0.2), (700, 3, 90, 0.5), (40, 1000, 900, 0.2), (5000, 64, 5, 0.3), (17000, 65, 2, 0.1),
])
@pytest.mark.parametrize("apart", [False, True])
def test_steps_and_prompts(L, batch, longest, add, ended, apart):
    rng = random.Random(batch * 31 + add)
    change = [-1 - rng.randint(0, 5) if rng.random() < ended else rng.randint(0, add) for _ in range(batch)]
    max_pages = -(-(longest + add) // 64) + 1
    new = sum(max(0, n) for n in change)
    state = _state(rng, batch, max_pages, new // 64 + batch + 3, longest)
    _check(change, state, new, apart)
    _check(change, state, new + 37, apart, offset=3)      # slots off 16 bytes, and some behind the last token


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [7, 300, 2000])
def test_what_does_not_fit_is_refused(L, batch):
    rng = random.Random(batch)
    change = [rng.choice((-1, 0, 1, 40, 64, 129)) for _ in range(batch)]
    new = sum(max(0, n) for n in change)
    for spare, tokens, max_pages in ((batch // 3, new, 6), (0, new, 6), (2 * batch + 64, new // 2, 6), (2 * batch + 64, 0, 6),
                                     (2 * batch + 64, new, 4)):
        state = _state(rng, batch, max_pages, spare, 200)
        for apart in (False, True):
            _check(change, state, tokens, apart)


@pytest.mark.gpu
def test_bad_state_is_reported(L):
    rng = random.Random(5)
    lens, table, free, count, pages = _state(rng, 40, 5, 30, 200)
    change = [-1 if r % 4 == 0 else 40 for r in range(40)]
    new = sum(max(0, n) for n in change)
    for edit in ("negative length", "long", "count", "count below", "free id", "table id", "ended id"):
        l2, t2, f2, c2 = list(lens), [list(r) for r in table], list(free), count
        if edit == "negative length":
            l2[1] = l2[4] = -9
        elif edit == "long":
            l2[2], l2[8] = 5 * 64 + 1, 5 * 64 + 1
        elif edit == "count":
            c2 = pages + 1
            f2 = [i % pages for i in range(pages)]
        elif edit == "count below":
            c2 = -3
        elif edit == "free id":
            f2[count - 2], f2[count - 5] = -7, pages
        elif edit == "table id":
            l2[3], t2[3][0] = 30, pages + 5
        else:
            l2[4], t2[4][:3] = 130, [-2, 1, pages]
        _check(change, (l2, t2, f2, c2, pages), new, False)


@pytest.mark.gpu
def test_no_tokens_and_a_step_of_none(L):
    state = _state(random.Random(3), 9, 3, 4, 100)
    _check([0] * 9, state, 0, False)
    _check([-1] * 9, state, 5, False)


@pytest.mark.gpu
def test_a_captured_step_walks_on(L):
    """Replays of a captured call update lengths, table and stack in place, and cross pages as a walk does."""
    rng = random.Random(11)
    state = _state(rng, 21, 9, 80, 100)
    lens, table, free, count, pages = state
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    change = i32([1] * 20 + [3])
    seq, tab, fr, cnt = i32(lens), i32(table), i32(free), i32([count])
    cu, slots = torch.empty(22, dtype=torch.int32, device="cuda"), torch.empty(23, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.dsa_pages_update(change, seq, tab, fr, cnt, cu, slots)
    step = change.tolist()
    for i in range(90):
        if i == 50:
            step = [-1 if r % 3 == 0 else 2 for r in range(20)] + [0]
            change.copy_(i32(step))
        if i == 51:
            step = [r % 2 for r in range(21)]
            change.copy_(i32(step))
        graph.replay()
        lens, table, free, count, offs, sl, bad = walk(step, lens, table, free, count, 23, pages)
        if sum(max(0, n) for n in step) > 23:
            assert bad
        assert (seq.tolist(), tab.tolist(), cnt.item(), cu.tolist(), slots.tolist()) == (lens, table, count, offs, sl), i
        assert fr.tolist()[:count] == free[:count]
        assert api.dsa_get_device_error() == (5 if bad else 0)


@pytest.mark.gpu
def test_binding_checks(L):
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
    ok = dict(change=i32(3), seqlens=i32(3), page_table=i32(3, 2), free_pages=i32(5), free_count=i32(1), cu_new=i32(4),
              slots=i32(6))
    api.dsa_pages_update(**ok)
    for name, t in (("change", i32(2)), ("seqlens", i32(4)), ("free_count", i32(2)), ("cu_new", i32(3)),
                    ("seqlens_out", i32(2)), ("free_count_out", i32(0)), ("page_table", i32(2, 3).t())):
        with pytest.raises(ValueError, match=name):
            api.dsa_pages_update(**{**ok, name: t})
    for name in ("change", "slots", "page_table"):
        with pytest.raises(TypeError, match=name):
            api.dsa_pages_update(**{**ok, name: ok[name].long()})
    with pytest.raises(ValueError, match="slots"):
        api.dsa_pages_update(**{**ok, "slots": i32(12)[::2]})
