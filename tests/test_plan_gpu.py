"""The cache's planning against its definition on the host, number for number."""
import random

import pytest
import torch

import prompt_reference as R

pytestmark = pytest.mark.gpu


def _pool(held, extra, cols, seed):
    """A table of the held tokens over shuffled pages, -1 or nonsense behind them, and the number of pages."""
    rng = random.Random(seed)
    live = [R.up(m) for m in held]
    pages = sum(live) + extra
    order = list(range(pages))
    rng.shuffle(order)
    table, at = [], 0
    for c in live:
        table.append(order[at:at + c] + [rng.choice((-1, 0, 1 << 29, pages)) for _ in range(cols - c)])
        at += c
    return table, pages


def _cache(V, table, pages, length):
    codes = torch.zeros((1, 1, 1, 1), dtype=torch.uint8, device="cuda").expand(pages, 1, 128, 128)
    scales = torch.zeros((1, 1), device="cuda").expand(pages, 1)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    return V.Cache(codes, codes, scales, scales, ints(table), ints(length))


def _check(V, held, news, table, pages, T, in_place=True):
    cache = _cache(V, table, pages, held if in_place else [5] * len(held))
    before = None if in_place else torch.tensor(held, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, slot, position = V.cache_plan(cache, torch.tensor(news, dtype=torch.int32, device="cuda"), T, held=before, dev_status=status)
    torch.cuda.synchronize()
    t, length, s, sl, pos, code = R.plan(table, held, news, pages, T)
    pad = [-1] * (T - len(sl))
    assert int(status) == code
    assert start.tolist() == s
    assert cache.length.tolist() == (length if code == 0 else held if in_place else [5] * len(held))
    assert cache.table.tolist() == t
    assert slot.tolist() == sl + pad and position.tolist() == pos + pad
    assert in_place or before.tolist() == held


CASES = {
    "one": ([0], [1], 3),
    "page borders": ([0, 127, 128, 129, 1], [128, 1, 1, 127, 0], 9),
    "a token each": ([300, 5, 255, 256, 0], [1, 1, 1, 1, 1], 2),
    "no new page": ([300, 5, 130], [1, 2, 3], 0),
    "nothing": ([300, 5], [0, 0], 4),
    "a chunk": ([1000], [5000], 50),
    "prompts among tokens": ([0, 900, 0, 70, 128], [700, 1, 33, 1, 1], 20),
    "exactly enough": ([100, 0], [500, 200], 6),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_plans(V, name, in_place):
    held, news, extra = CASES[name]
    cols = max(R.up(m + n) for m, n in zip(held, news)) + 2
    table, pages = _pool(held, extra, cols, seed=len(name))
    for more in (0, 5):
        _check(V, held, news, table, pages, sum(news) + more, in_place)


@pytest.mark.parametrize("B", [33, 513, 4096, 4097, 9001, 65535])
def test_many_sequences(V, B):
    rng = random.Random(B)
    held = [rng.randrange(0, 300) for _ in range(B)]
    news = [rng.choice((0, 1, 1, 1, 130)) if B < 10000 else rng.choice((0, 0, 1)) for _ in range(B)]
    table, pages = _pool(held, 3 * B, 5, seed=B)
    _check(V, held, news, table, pages, sum(news))


def test_long_tables(V):
    rng = random.Random(2)
    held = [400000, 3, 90001, 128 * 700]
    news = [1, 40000, 128, 129]
    table, pages = _pool(held, 400, 4000, seed=3)
    _check(V, held, news, table, pages, sum(news))


def test_more_pages_than_one_bitmap_holds(V):
    """Two million pages, of which the first 1.9 million are named."""
    named, pages = 1_900_000, 2_000_000
    table = torch.full((2, named + 9), -1, dtype=torch.int32, device="cuda")
    table[0, :named] = torch.randperm(named, device="cuda").to(torch.int32)
    table[1, 0] = named + 1
    codes = torch.zeros((1, 1, 1, 1), dtype=torch.uint8, device="cuda").expand(pages, 1, 128, 128)
    cache = V.Cache(codes, codes, None, None, table, torch.tensor([named * 128, 100], dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    news = torch.tensor([3, 300], dtype=torch.int32, device="cuda")
    start, slot, _ = V.cache_plan(cache, news, 303, dev_status=status)
    assert int(status) == 0 and cache.table[0, named:named + 2].tolist() == [named, -1]
    assert cache.table[1, :5].tolist() == [named + 1, named + 2, named + 3, named + 4, -1]
    assert slot[:4].tolist() == [named * 128, named * 128 + 1, named * 128 + 2, (named + 1) * 128 + 100]
    # one more than the rest, then the rest: 99,995 pages
    for pages_more, code in ((99996, V.VCA_ERR_FULL), (99995, 0)):
        n = pages_more * 128 + 512 - 400
        news = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        start = V.cache_plan(cache, news, n, dev_status=status)[0]
        assert int(status) == code
        if code:
            assert start.tolist() == [0, 0, 0] and cache.length.tolist() == [named * 128 + 3, 400]
        status.zero_()
    assert torch.equal(cache.table[1, 4:99999].cpu(), torch.arange(named + 5, pages, dtype=torch.int32))


REFUSED = {
    "too few pages": ([100, 0], [500, 200], 5, 0),
    "no page": ([128], [1], 0, 0),
    "negative held": ([100, -1, 3], [1, 1, 1], 9, 0),
    "negative news": ([100, 1, 3], [1, -1, 1], 9, 0),
    "behind the table": ([100, 1, 3], [1, 129 + 1000 * 128, 1], 2000, 0),
    "huge": ([2 ** 31 - 1, 1], [2 ** 31 - 1, 1], 9, 0),
    "more rows than T": ([100, 1], [5, 6], 9, -1),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", REFUSED)
def test_a_plan_is_made_whole_or_not_at_all(V, name, in_place):
    held, news, extra, rows = REFUSED[name]
    T = min(sum(max(0, n) for n in news), 2000) + rows
    sane = [m if 0 <= m < 10000 else 0 for m in held]
    table, pages = _pool(sane, extra, 9, seed=5)
    _check(V, held, news, table, pages, T, in_place)


def test_shared_and_released_pages(V):
    """A page that two sequences name is free when both are gone; a length of 0 gives pages back."""
    table = [[4, 2, -1], [4, 3, -1], [1, -1, -1]]
    _check(V, [256, 200, 128], [1, 100, 1], table, 8, 102)
    _check(V, [0, 200, 128], [300, 0, 0], table, 8, 300)      # 2 is free, 4 is not
    _check(V, [0, 0, 128], [300, 1, 0], table, 8, 301)


def test_pages_that_do_not_exist(V):
    """They name nothing and have no slots; the call says so, and the plan is made."""
    table = [[9999, 1, -1], [-3, -1, -1], [0, -1, -1]]
    cache = _cache(V, table, 6, [200, 100, 128])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, slot, position = V.cache_plan(cache, torch.tensor([2, 30, 1], dtype=torch.int32, device="cuda"), 33, dev_status=status)
    assert int(status) == V.VCA_ERR_INVALID_ARG and start.tolist() == [0, 2, 32, 33] and cache.length.tolist() == [202, 130, 129]
    assert cache.table.tolist() == [[9999, 1, -1], [-3, 2, -1], [0, 3, -1]]
    assert slot.tolist() == [128 + 72, 128 + 73] + [-1] * 28 + [2 * 128, 2 * 128 + 1] + [3 * 128]


def test_without_slots_and_positions(V):
    cache = _cache(V, [[0, -1], [1, -1]], 5, [100, 128])
    start = torch.empty(3, dtype=torch.int32, device="cuda")
    V.vca_cache_plan(cache, cache.length, torch.tensor([1, 1], dtype=torch.int32, device="cuda"), 2, start, None, None)
    assert start.tolist() == [0, 1, 2] and cache.length.tolist() == [101, 129] and cache.table.tolist() == [[0, -1], [1, 2]]


@pytest.mark.parametrize("budget", [1, 128, 129, 300, 100000])
def test_fresh_pages(V, budget):
    held = [1000, 0, 77, 128, 300]
    table, pages = _pool(held, 5 * 9 + 2, 9, seed=7)
    cache = _cache(V, table, pages, held)
    cols = min(R.up(budget), 12)
    if cols * 128 < budget:
        with pytest.raises(V.VCAError):
            V.cache_fresh(cache, budget, out=torch.zeros((5, cols), dtype=torch.int32, device="cuda"))
        return
    dst = torch.full((5, cols + 1), 77, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.cache_fresh(cache, budget, out=dst, dev_status=status)
    assert int(status) == 0 and dst.tolist() == R.fresh(table, held, pages, budget, [[77] * (cols + 1)] * 5)
    assert cache.table.tolist() == table and cache.length.tolist() == held


def test_fresh_pages_that_are_too_few_or_lengths_out_of_range(V):
    for held, extra, code in (([1000, 300], 10, V.VCA_ERR_FULL), ([1000, 9 * 128 + 1], 30, V.VCA_ERR_INVALID_ARG),
                              ([1000, -4], 30, V.VCA_ERR_INVALID_ARG)):
        table, pages = _pool([m if 0 < m <= 1152 else 0 for m in held], extra, 9, seed=8)
        cache = _cache(V, table, pages, held)
        dst = torch.full((2, 9), 77, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        V.cache_fresh(cache, 1100, out=dst, dev_status=status)
        assert int(status) == code and bool((dst == 77).all())


def test_captured(V):
    """A captured decode step replayed until the pages are used up, and told so."""
    held = [126, 254, 0]
    table, pages = _pool(held, 3, 4, seed=9)
    cache = _cache(V, table, pages, held)
    news = torch.ones(3, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start, slot, position = (torch.full((n,), -1, dtype=torch.int32, device="cuda") for n in (4, 3, 3))
    V.cache_plan(_cache(V, table, pages, held), news, 3, start=start, slot=slot, position=position)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.cache_plan(cache, news, 3, start=start, slot=slot, position=position, dev_status=status)
    for _ in range(140):
        t, length, s, sl, pos, code = R.plan(table, held, [1, 1, 1], pages, 3)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status) == code and cache.table.tolist() == t and start.tolist() == s
        if code:
            assert cache.length.tolist() == held
            break
        assert cache.length.tolist() == length and slot.tolist() == sl and position.tolist() == pos
        table, held = t, length
    assert code == V.VCA_ERR_FULL


def test_on_a_named_stream(V):
    table, pages = _pool([100, 200], 9, 4, seed=10)
    cache = _cache(V, table, pages, [100, 200])
    news, start = torch.tensor([100, 1], dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    dst = torch.full((2, 2), -1, dtype=torch.int32, device="cuda")
    busy, side = torch.randn((4096, 4096), device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-2      # the calls must wait for this on `side`
        cache.length.copy_(torch.tensor([100, 130], dtype=torch.int32))
    V.vca_cache_plan(cache, cache.length, news, 101, start, None, None, stream=side)
    V.vca_cache_fresh(cache, 200, dst, stream=side)
    side.synchronize()
    t, length, s, _, _, _ = R.plan(table, [100, 130], [100, 1], pages, 101)
    assert cache.table.tolist() == t and cache.length.tolist() == length and start.tolist() == s
    assert dst.tolist() == R.fresh(t, length, pages, 200, [[-1, -1]] * 2)
