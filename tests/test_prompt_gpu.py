"""Prompt attention against its definition in 64 bits, within bounds that its
arithmetic gives (prompt_reference.py)."""
import math

import pytest
import torch

import prompt_reference as R

pytestmark = pytest.mark.gpu


def _inputs(lens, Hq, H, seed=1, extra=0):
    T = sum(lens) + extra
    return R.rows(T, Hq, seed), R.rows(T, H, seed + 1), R.rows(T, H, seed + 2, outliers=False), R.starts(lens)


def _check(V, lens, Q, K, Val, start, **kw):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.prompt_attention(Q, K, Val, start, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    kw.pop("out", None)
    kw["scale"] = kw.pop("softmax_scale", None)
    o, z, eo, el = R.attention(Q, K, Val, lens, **kw)
    n = sum(lens)
    R.within(out[:n], o[:n], eo[:n], "O")
    R.within(lse[:n], z[:n], el[:n], "lse")
    return out, lse


# lengths, query heads, KV heads
BATCHES = {
    "one token": ([1], 1, 1),
    "two tokens": ([2], 3, 3),
    "block borders": ([127, 128, 129], 2, 2),
    "half blocks": ([63, 64, 65, 191, 192, 193], 2, 1),
    "tile borders": ([255, 256, 257, 511, 513], 1, 1),
    "five to a head": ([300, 77, 530], 10, 2),
    "seven to a head": ([200, 18, 37, 19], 7, 1),
    "twelve to a head": ([90, 10, 11, 21], 12, 1),
    "one shared head": ([513, 64, 8, 9], 16, 1),
    "forty to a head": ([130, 3, 7], 40, 1),
    "more heads than rows": ([140, 1], 130, 1),
    "a prime number of heads": ([150, 40], 37, 1),
    "empty sequences": ([0, 40, 0, 0, 300, 0], 4, 4),
    "many short": ([(b * 7) % 23 for b in range(200)], 4, 2),
    "long": ([2111], 4, 2),
    "long and short": ([900, 1, 64, 1500, 5], 8, 4),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", BATCHES)
def test_prompts(V, name, causal):
    lens, Hq, H = BATCHES[name]
    _check(V, lens, *_inputs(lens, Hq, H, seed=len(name)), causal=causal)


@pytest.mark.parametrize("softcap", [0.5, 30.0, 64.0, 65.0, 3000.0, 1e-30, 1e30])
@pytest.mark.parametrize("name", ["half blocks", "five to a head", "long"])
def test_capped(V, name, softcap):
    lens, Hq, H = BATCHES[name]
    for causal in (True, False):
        _check(V, lens, *_inputs(lens, Hq, H, seed=40), causal=causal, softcap=softcap)


def test_average_error_is_that_of_two_roundings(V):
    """P and O round to bf16, 2^-8 at most and 2^-8 / sqrt 3 on average each."""
    lens = [1500]
    Q, K, Val, start = _inputs(lens, 4, 2, seed=50)
    out, _ = V.prompt_attention(Q, K, Val, start, causal=False)
    o = R.attention(Q, K, Val, lens, causal=False)[0]
    assert float((out.double() - o).norm() / o.norm()) <= 2.0 ** -8


@pytest.mark.parametrize("magnitude", [2.0 ** -40, 2.0 ** 30])
def test_scales_of_any_magnitude(V, magnitude):
    lens = [300, 70]
    Q, K, Val, start = _inputs(lens, 4, 2, seed=51)
    _check(V, lens, (Q.float() * magnitude).bfloat16(), K, Val, start, softmax_scale=0.11 / magnitude)
    _check(V, lens, (Q.float() * magnitude).bfloat16(), K, Val, start, softmax_scale=0.11 / magnitude, softcap=20.0)
    _check(V, lens, Q, K, (Val.float() * magnitude).bfloat16(), start)


def test_scores_far_apart(V):
    """Maxima that rise block by block by more than the kernel's threshold, and fall."""
    for step in (3.0, -3.0):
        lens = [1100]
        Q, K, Val, start = _inputs(lens, 2, 1, seed=52)
        Q[..., 0] = 8.0
        K[..., 0] = (torch.arange(1100, device="cuda") // 100 * step).bfloat16()[:, None]
        for causal in (True, False):
            _check(V, lens, Q, K, Val, start, causal=causal, softmax_scale=1.0)


LAYOUTS = {
    "heads first": lambda T, H, g: torch.randn((H, T, 128), generator=g).bfloat16().cuda().transpose(0, 1),
    "wide rows": lambda T, H, g: torch.randn((T, H + 3, 128), generator=g).bfloat16().cuda()[:, 1:H + 1],
    "odd distances": lambda T, H, g: torch.randn(T * (H * 136 + 8) + 256, generator=g).bfloat16().cuda().as_strided(
        (T, H, 128), (H * 136 + 8, 136, 1)),
    "heads far apart": lambda T, H, g: torch.randn(H * (T * 136 + 24) + 256, generator=g).bfloat16().cuda().as_strided(
        (T, H, 128), (136, T * 136 + 24, 1)),
}


@pytest.mark.parametrize("layout", LAYOUTS)
def test_layouts(V, layout):
    g = torch.Generator().manual_seed(53)
    lens = [200, 131]
    Q, K, Val = (LAYOUTS[layout](sum(lens), h, g) for h in (6, 2, 2))
    assert not Q.is_contiguous()
    for causal in (True, False):
        _check(V, lens, Q, K, Val, R.starts(lens), causal=causal)


def test_shared_keys_as_an_expanded_view(V):
    lens = [150, 90]
    Q, K, _, start = _inputs(lens, 8, 1, seed=54)
    _check(V, lens, Q, K.expand(-1, 4, -1), K.expand(-1, 4, -1), start)


def test_offsets_beyond_32_bits(V):
    """Heads more than 2^32 elements apart."""
    T, far = 40, (1 << 32) + 64
    buf = torch.empty(far + T * 128, dtype=torch.bfloat16, device="cuda")
    x = buf.as_strided((T, 2, 128), (128, far, 1))
    x.copy_(R.rows(T, 2, 55))
    _check(V, [T], x, x, x, R.starts([T]))


@pytest.mark.parametrize("name", ["half blocks", "five to a head", "long and short"])
def test_joined_with_a_prior(V, name):
    lens, Hq, H = BATCHES[name]
    Q, K, Val, start = _inputs(lens, Hq, H, seed=56)
    T = sum(lens)
    o = R.rows(T, Hq, 57, outliers=False)
    z = torch.randn((T, Hq), generator=torch.Generator().manual_seed(58)).cuda() * 40.0
    z[::3] = -math.inf
    o[::3] = math.nan      # not read
    for causal, cap in ((True, 0.0), (False, 0.0), (True, 30.0), (True, 500.0)):
        _check(V, lens, Q, K, Val, start, causal=causal, softcap=cap, prior=(o, z))
    # in place
    out, lse = o.clone(), z.clone()
    again = V.prompt_attention(Q, K, Val, start, prior=(o, z))
    V.prompt_attention(Q, K, Val, start, prior=(out, lse), out=out, lse=lse)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_rows_behind_the_last_sequence_stay(V):
    lens = [60, 0, 130]
    Q, K, Val, start = _inputs(lens, 4, 2, seed=59, extra=9)
    K[190:], Val[190:], Q[190:] = math.nan, math.nan, math.nan
    out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(Q.shape[:2], 7.0, device="cuda")
    V.prompt_attention(Q, K, Val, start, out=out, lse=lse)
    o, z, eo, el = R.attention(Q, K, Val, lens)
    R.within(out[:190], o[:190], eo[:190], "O")
    R.within(lse[:190], z[:190], el[:190], "lse")
    assert bool((out[190:] == 7).all()) and bool((lse[190:] == 7).all())


def test_neighbours_of_nan_and_infinity(V):
    """What other sequences hold, before and behind, does not reach a sequence."""
    lens = [70, 200, 129, 40]
    for bad in (math.nan, math.inf, -math.inf):
        for causal in (True, False):
            for cap in (0.0, 30.0, 200.0):
                Q, K, Val, start = _inputs(lens, 10, 2, seed=60)
                o, z, eo, el = R.attention(Q, K, Val, lens, causal=causal, softcap=cap)
                for x in (Q, K, Val):
                    x[:70], x[270:399] = bad, bad
                out, lse = V.prompt_attention(Q, K, Val, start, causal=causal, softcap=cap)
                for sl in (slice(70, 270), slice(399, 439)):
                    R.within(out[sl], o[sl], eo[sl], "O")
                    R.within(lse[sl], z[sl], el[sl], "lse")


def test_a_key_of_nan_reaches_only_the_rows_that_see_it(V):
    lens = [300, 40]
    Q, K, Val, start = _inputs(lens, 4, 2, seed=61)
    o, z, eo, el = R.attention(Q, K, Val, lens)
    K[77, 0, 3] = math.nan
    Q[20, 1, 5] = math.nan
    out, lse = V.prompt_attention(Q, K, Val, start)
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool, device="cuda")
    bad[77:300, :2] = True
    bad[20, 1] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    R.within(out[~bad], o[~bad], eo[~bad], "O")
    R.within(lse[~bad], z[~bad], el[~bad], "lse")


@pytest.mark.parametrize("many", [False, True])
def test_starts_that_fall(V, many):
    """The sequences before the fall are right, the rows behind are nobody's, and the call says so."""
    lens = [3 + b % 9 for b in range(400)] if many else [100, 60, 70, 50]
    at = 300 if many else 2
    n = sum(lens[:at])
    for wrong in (-5, n - 4, sum(lens) + 1, 1 << 30):
        Q, K, Val, start = _inputs(lens, 4, 2, seed=62)
        o, z, eo, el = R.attention(Q, K, Val, lens)
        start[at + 1] = wrong
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(Q.shape[:2], 7.0, device="cuda")
        V.prompt_attention(Q, K, Val, start, out=out, lse=lse, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == V.VCA_ERR_INVALID_ARG
        R.within(out[:n], o[:n], eo[:n], "O")
        R.within(lse[:n], z[:n], el[:n], "lse")
        assert bool((out[n:] == 7).all()) and bool((lse[n:] == 7).all())


@pytest.mark.parametrize("causal", [True, False])
def test_more_sequences_than_are_sorted(V, causal):
    lens = [(b * 37) % 61 for b in range(700)]
    _check(V, lens, *_inputs(lens, 6, 2, seed=63), causal=causal)
    lens = [0] * 300 + [400] + [0] * 300
    _check(V, lens, *_inputs(lens, 2, 2, seed=64), causal=causal)


def test_as_many_sequences_as_there_can_be(V):
    """Single tokens: O is the value, lse the score (two of 128 exact products and their sum's rounding)."""
    B = 65535
    lens = torch.arange(B) % 3 != 1
    T = int(lens.sum())
    start = torch.nn.functional.pad(torch.cumsum(lens, 0), (1, 0)).to(torch.int32).cuda()
    Q, K, Val = R.rows(T, 3, 78), R.rows(T, 1, 79), R.rows(T, 1, 80)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.prompt_attention(Q, K, Val, start, dev_status=status)
    assert int(status) == 0 and torch.equal(out, Val.expand(-1, 3, -1))
    s = (Q.double() * K.double()).sum(-1) / math.sqrt(128)
    mag = (Q.double() * K.double()).abs().sum(-1) / math.sqrt(128)
    R.within(lse, s, 2.0 ** -16 * mag + 2.0 ** -20 * (1 + s.abs()), "lse")


def test_outputs_at_any_place(V):
    """O need not be 32-byte aligned, lse may be left out."""
    lens = [140, 33]
    Q, K, Val, start = _inputs(lens, 5, 1, seed=65)
    ref, _ = V.prompt_attention(Q, K, Val, start)
    buf = torch.zeros(Q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = buf[8:].view(Q.shape)
    assert out.data_ptr() % 32 == 16
    V.vca_prompt_attention(Q, K, Val, start, 1, 0.0, 0.0, None, None, out, None)
    assert torch.equal(out, ref) and not bool(buf[:8].any())


def test_no_rows(V):
    Q, K, Val, _ = _inputs([0], 4, 2)
    out, lse = V.prompt_attention(Q, K, Val, torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4)
    Q, K, Val, start = _inputs([5, 5], 4, 2)
    out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    V.prompt_attention(Q, K, Val, torch.zeros_like(start), out=out)
    assert bool((out == 7).all())


def test_equal_calls_give_equal_bits(V):
    lens = [1300, 40, 700, 2]
    Q, K, Val, start = _inputs(lens, 10, 2, seed=66)
    first = V.prompt_attention(Q, K, Val, start)
    for _ in range(20):
        again = V.prompt_attention(Q, K, Val, start)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_a_work_may_last_longer_than_a_wait(V):
    """The limit is that of waits for a block; 100,001 tokens are 782 of them in a row."""
    n = 100001
    Q, K, Val, start = _inputs([n], 1, 1, seed=69)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    V.vca_set_wait_limit_ns(400_000)
    try:
        out, lse = V.prompt_attention(Q, K, Val, start, causal=False, dev_status=status)
        torch.cuda.synchronize()
    finally:
        V.vca_set_wait_limit_ns(2_000_000_000)
    assert int(status) == 0
    at = torch.tensor([0, 1, 777, n // 2, n - 1], device="cuda")
    s = Q[at, 0].double() @ K[:, 0].double().T / math.sqrt(128)
    assert torch.allclose(lse[at, 0].double(), torch.logsumexp(s, -1), rtol=1e-5)
    o = torch.softmax(s, -1) @ Val[:, 0].double()
    assert float((out[at, 0].double() - o).norm() / o.norm()) <= 2.0 ** -7      # P's and O's rounding, 2^-8 each at most


def test_waits_that_run_out(V):
    """A limit shorter than a copy from memory: the call says so (or was quick enough), and the next is right."""
    lens = [3000, 70]
    Q, K, Val, start = _inputs(lens, 4, 2, seed=77)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(3):
        V.vca_set_wait_limit_ns(1000)
        try:
            V.prompt_attention(Q, K, Val, start, dev_status=status)
            torch.cuda.synchronize()
        finally:
            V.vca_set_wait_limit_ns(2_000_000_000)
        assert int(status) in (0, V.VCA_ERR_TIMEOUT)
        status.zero_()
        _check(V, lens, Q, K, Val, start)


def test_captured_and_on_other_streams(V):
    """One graph replayed over new inputs and lengths, beside calls on another stream."""
    lens, other = [300, 40, 500], [100, 640, 100]
    Q, K, Val, start = _inputs(lens, 8, 2, seed=67)
    out, lse = torch.empty_like(Q), torch.empty(Q.shape[:2], device="cuda")
    V.prompt_attention(Q, K, Val, start, out=out, lse=lse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.prompt_attention(Q, K, Val, start, out=out, lse=lse)
    q2, k2, v2, s2 = _inputs(other, 8, 2, seed=68)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x, y in ((Q, q2), (K, k2), (Val, v2), (start, s2)):
        x.copy_(y)
    mine = torch.empty_like(out), torch.empty_like(lse)
    for _ in range(3):
        graph.replay()
        V.vca_prompt_attention(q2, k2, v2, s2, 1, 0.0, 0.0, None, None, *mine, stream=side)
    torch.cuda.synchronize()
    o, z, eo, el = R.attention(q2, k2, v2, other)
    for x in ((out, lse), mine):
        R.within(x[0], o, eo, "O")
        R.within(x[1], z, el, "lse")


def test_a_prompt_on_its_way_into_the_cache(V):
    """Plan, prompt attention, append; then a chunk behind it (joined with the cache's attention),
    single tokens, an eviction into fresh pages and a plan that gets the old pages again."""
    import cache_reference as C
    H, Hq, B = 2, 6, 3
    cache = V.alloc_cache(pages=14, H=H, B=B, cols=6)
    weight = torch.zeros((14, H, 128), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    host = C.Case(*(getattr(cache, f).cpu() for f in ("k8", "v8", "sk", "sv", "table", "length")), None)
    held = [0] * B

    def step(news, seed):
        T = sum(news)
        before = V.Cache(cache.k8, cache.v8, cache.sk, cache.sv, cache.table, cache.length.clone())
        start, slot, position = V.cache_plan(cache, torch.tensor(news, dtype=torch.int32, device="cuda"), T + 2, dev_status=status)
        t, length, s, sl, pos, _ = R.plan(host.table.tolist(), held, news, 14, T + 2)
        assert cache.table.tolist() == t and cache.length.tolist() == length and start.tolist() == s
        assert slot.tolist() == sl + [-1, -1] and position.tolist() == pos + [-1, -1]
        host.table, host.length, host.start = torch.tensor(t, dtype=torch.int32), torch.tensor(length, dtype=torch.int32), start.cpu()
        held[:] = length
        Q, K, Val = R.rows(T, Hq, seed), R.rows(T, H, seed + 1), R.rows(T, H, seed + 2, outliers=False)
        return before, start, Q, K, Val

    # the prompts
    news = [200, 37, 129]
    before, start, Q, K, Val = step(news, 70)
    out, lse = V.prompt_attention(Q, K, Val, start, dev_status=status)
    V.cache_append(cache, K, Val, start, dev_status=status, weight=weight)
    o, z, eo, el = R.attention(Q, K, Val, news)
    R.within(out, o, eo, "O of the prompts")
    C.append(host, K.cpu(), Val.cpu())
    # a chunk behind them
    news = [60, 0, 100]
    before, start, Q, K, Val = step(news, 73)
    prior = V.cache_attention(before, Q, start, causal=False, dev_status=status)
    out, lse = V.prompt_attention(Q, K, Val, start, prior=prior, dev_status=status)
    V.cache_append(cache, K, Val, start, dev_status=status, weight=weight)
    o, z, eo, el = R.attention(Q, K, Val, news, prior=prior)
    R.within(out, o, eo, "O of the chunk")
    R.within(lse, z, el, "lse of the chunk")
    C.append(host, K.cpu(), Val.cpu())
    # single tokens
    news = [1, 1, 1]
    before, start, Q, K, Val = step(news, 76)
    V.cache_append(cache, K, Val, start, dev_status=status, weight=weight)
    C.append(host, K.cpu(), Val.cpu())
    out, lse = V.cache_attention(cache, Q, start, dev_status=status)
    o, z, eo, el = C.attention(host, Q.cpu())
    R.within(out.cpu(), o, eo, "O of the tokens")
    V.cache_weigh(cache, Q, start, lse, weight, dev_status=status)
    # the eviction
    dst = V.cache_fresh(cache, 130, out=torch.full((B, 4), -1, dtype=torch.int32, device="cuda"), dev_status=status)
    assert dst.tolist() == R.fresh(host.table.tolist(), held, 14, 130, [[-1] * 4] * B)
    new_len, kept = V.cache_evict(cache, weight, dst, 130, 16, dev_status=status)
    assert new_len.tolist() == [min(m, 130) for m in held]
    cut = V.Cache(cache.k8, cache.v8, cache.sk, cache.sv, dst, new_len)
    # the pages of before are free again
    t, length, s, sl, _, code = R.plan(dst.tolist(), [min(m, 130) for m in held], [200, 0, 0], 14, 200)
    assert code == 0 and t[0][2] in host.table[:, :3].flatten().tolist()
    start, slot, _ = V.cache_plan(cut, torch.tensor([200, 0, 0], dtype=torch.int32, device="cuda"), 200, dev_status=status)
    assert cut.table.tolist() == t and cut.length.tolist() == length and slot.tolist() == sl
    torch.cuda.synchronize()
    assert int(status) == 0
