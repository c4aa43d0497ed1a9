"""The 8-bit cache's kernels against the 64-bit reference: codes, scales, lengths
and kept slots bit for bit; attention, lse and weights within the bounds that
their arithmetic gives (cache_reference.py)."""
import math

import pytest
import torch

import cache_reference as R

pytestmark = pytest.mark.gpu


def _same_codes(got, ref):
    """Equal bytes, any NaN code for a NaN."""
    got, ref = got.cpu(), ref
    nan = (ref & 0x7F) == 0x7F
    assert torch.equal(nan, (got & 0x7F) == 0x7F)
    assert torch.equal(got[~nan], ref[~nan])


def _within(got, ref, bound, what):
    got = got.double().cpu()
    assert torch.equal(torch.isfinite(got), torch.isfinite(ref)), what
    fin = torch.isfinite(ref)
    assert torch.equal(got[~fin], ref[~fin]), what
    over = ((got - ref).abs() - bound)[fin]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{what}: off by {float(over.max()):.3e} more than allowed"


def _check_attention(V, c, Q, **kw):
    cache, start = c.on(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.cache_attention(cache, Q.cuda() if not Q.is_cuda else Q, start, dev_status=status, **kw)
    torch.cuda.synchronize()
    assert int(status) == 0
    kw.pop("softmax_scale", None)
    o, z, eo, el = R.attention(c, Q.cpu(), **kw)
    n = int(c.start[-1])
    _within(out[:n], o[:n], eo[:n], "O")
    _within(lse[:n], z[:n], el[:n], "lse")
    return out, lse


# lengths and new rows of each sequence, query heads, KV heads
BATCHES = {
    "one token": ([1], [1], 1, 1),
    "page borders": ([127, 128, 129, 1], [1, 1, 1, 1], 4, 2),
    "five to a head": ([300, 77, 1030], [1, 1, 1], 10, 2),
    "one shared head": ([513, 64], [1, 1], 16, 1),
    "seven to a head": ([700], [3], 7, 1),
    "ragged rows": ([400, 131, 260, 90], [1, 17, 0, 5], 6, 3),
    "an empty sequence": ([0, 40, 0], [2, 1, 0], 4, 4),
    "long": ([20011], [1], 2, 1),
    "long and short": ([9000, 1, 200, 5000], [1, 1, 1, 1], 8, 4),
    "a chunk": ([1000], [200], 4, 2),
    "a prompt": ([333, 129], [333, 129], 8, 2),
    "wide rows": ([520, 260], [50, 33], 40, 8),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", BATCHES)
def test_attention(V, name, causal):
    lens, news, Hq, H = BATCHES[name]
    c = R.make_case(lens, news, H, seed=len(name))
    _check_attention(V, c, R.rows(sum(news), Hq, seed=3), causal=causal)


@pytest.mark.parametrize("name", ["five to a head", "ragged rows", "a chunk", "wide rows"])
@pytest.mark.parametrize("softcap", [30.0, 0.5])
def test_attention_capped(V, name, softcap):
    lens, news, Hq, H = BATCHES[name]
    c = R.make_case(lens, news, H, seed=11)
    _check_attention(V, c, R.rows(sum(news), Hq, seed=4), causal=True, softcap=softcap)


@pytest.mark.parametrize("news", [[1, 1], [40, 300]])
def test_attention_of_strided_rows(V, news):
    c = R.make_case([500, 301], news, 4, seed=5)
    wide = R.rows(sum(news), 8, seed=6, strided=True, device="cuda")
    assert not wide.is_contiguous()
    _check_attention(V, c, wide, causal=True)
    # heads first in memory
    flipped = R.rows(sum(news), 8, seed=6).cuda().transpose(0, 1).contiguous().transpose(0, 1)
    _check_attention(V, c, flipped, causal=False)


@pytest.mark.parametrize("news", [[3, 5], [150, 140]])
def test_rows_that_see_nothing(V, news):
    """Causal rows in front of the cache's first token: O = 0, lse = -inf."""
    c = R.make_case([2, 130], news, 2, seed=7)
    out, lse = _check_attention(V, c, R.rows(sum(news), 4, seed=8), causal=True)
    hidden = news[0] - 2
    assert hidden > 0 and bool((out[:hidden] == 0).all()) and bool((lse[:hidden] == -math.inf).all())


@pytest.mark.parametrize("news", [[1], [130]])
def test_page_scales_far_apart(V, news):
    """Neighbouring pages whose scales differ by large powers of two, a page of zeros among them."""
    c = R.make_case([900], news, 1, seed=9)
    for j, e in enumerate([-6, -30, -7, -120, -3, -60, 10, -6]):
        p = int(c.table[0, j])
        c.sv[p] = 2.0 ** e
        if e == -120:
            c.v8[p] = 0
        c.sk[p] = 2.0 ** -7
    _check_attention(V, c, R.rows(news[0], 2, seed=10), causal=True)
    # all of the weight on the page of the smallest values: relative to them the result must hold
    c.sk[:] = 2.0 ** -20
    p = int(c.table[0, 1])
    c.sk[p] = 2.0 ** -1
    _check_attention(V, c, R.rows(news[0], 2, seed=12), causal=False)


@pytest.mark.parametrize("magnitude", [2.0 ** -60, 2.0 ** 40])
@pytest.mark.parametrize("news", [[1], [140]])
def test_queries_of_any_magnitude(V, news, magnitude):
    c = R.make_case([300], news, 2, seed=13)
    c.sk *= 1.0 / magnitude
    Q = (R.rows(news[0], 2, seed=14).double() * magnitude).to(torch.bfloat16)
    _check_attention(V, c, Q, causal=True)


def test_rows_behind_the_last_sequence_stay(V):
    for news in ([1, 1], [70, 90]):
        c = R.make_case([200, 140], news, 2, seed=15)
        T = sum(news) + 3
        Q = R.rows(T, 4, seed=16).cuda()
        out = torch.full((T, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, 4), 7.0, device="cuda")
        cache, start = c.on(V)
        V.cache_attention(cache, Q, start, out=out, lse=lse)
        assert bool((out[-3:] == 7).all()) and bool((lse[-3:] == 7).all()) and bool((lse[:-3] != 7).all())


def test_other_sequences_do_not_see_a_nan(V):
    for news in ([1, 1, 1], [60, 60, 60]):
        c = R.make_case([200, 140, 300], news, 2, seed=17)
        clean = c.clone()
        p = int(c.table[1, 0])
        c.k8[p, :, 5] = 0x7F
        c.v8[p, :, 6] = 0xFF
        Q = R.rows(sum(news), 4, seed=18)
        cache, start = c.on(V)
        out, lse = V.cache_attention(cache, Q.cuda(), start, causal=False)
        o, z, eo, el = R.attention(clean, Q, causal=False)
        n0, n1 = int(c.start[1]), int(c.start[2])
        for sl in (slice(0, n0), slice(n1, None)):
            _within(out[sl], o[sl], eo[sl], "O")
        assert bool(torch.isnan(out[n0:n1]).all()) and bool(torch.isnan(lse[n0:n1]).all())


def test_bad_tables_and_lengths_are_reported(V):
    """Device-side indices out of range are checked before use: the call reports
    them, and the other sequences are right."""
    for news in ([1, 1, 1], [60, 60, 60]):
        c = R.make_case([200, 140, 300], news, 2, seed=19, cols=3)
        Q = R.rows(sum(news), 4, seed=20)
        o, z, eo, el = R.attention(c, Q)
        n0, n1 = int(c.start[1]), int(c.start[2])
        for kind in ("page", "negative page", "length", "negative length", "start"):
            d = c.clone()
            if kind == "page":
                d.table[1, 0] = 1 << 30
            elif kind == "negative page":
                d.table[1, 1] = -5
            elif kind == "length":
                d.length[1] = 1 << 30
            elif kind == "negative length":
                d.length[1] = -1
            else:
                d.start[2] = 0      # sequence 1 falls, sequence 2 takes every row
            cache, start = d.on(V)
            status = torch.zeros(1, dtype=torch.int32, device="cuda")
            out, lse = V.cache_attention(cache, Q.cuda(), start, dev_status=status)
            torch.cuda.synchronize()
            assert int(status) == V.VCA_ERR_INVALID_ARG, kind
            if kind == "start":
                continue
            for sl in (slice(0, n0), slice(n1, None)):
                _within(out[sl], o[sl], eo[sl], f"O ({kind})")
                _within(lse[sl], z[sl], el[sl], f"lse ({kind})")
            weight = torch.zeros((*c.sk.shape, 128), device="cuda")
            status.zero_()
            V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), weight, dev_status=status)
            torch.cuda.synchronize()
            assert int(status) == V.VCA_ERR_INVALID_ARG, kind
            K = R.rows(sum(news), 2, seed=21).cuda()
            status.zero_()
            V.cache_append(cache, K, K, start, dev_status=status)
            torch.cuda.synchronize()
            assert int(status) == (V.VCA_ERR_INVALID_ARG if kind != "page" or news[1] > 12 else 0), kind


@pytest.mark.parametrize("name", ["page borders", "five to a head", "ragged rows", "an empty sequence", "long and short",
                                  "a chunk", "a prompt", "wide rows", "one shared head"])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_weigh(V, name, softcap):
    lens, news, Hq, H = BATCHES[name]
    for causal in (True, False):
        c = R.make_case(lens, news, H, seed=23)
        Q = R.rows(sum(news), Hq, seed=24)
        _, z, _, _ = R.attention(c, Q, causal=causal, softcap=softcap)
        g = torch.Generator().manual_seed(25)
        weight = torch.rand((*c.sk.shape, 128), generator=g)
        w, e = R.weigh(c, Q, z.float(), weight, causal=causal, softcap=softcap)
        got = weight.cuda()
        cache, start = c.on(V)
        V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), got, causal=causal, softcap=softcap)
        _within(got, w, e, "weight")


@pytest.mark.parametrize("lens,news", [([1], [1]), ([130], [3]), ([128, 256], [128, 5]), ([700, 129, 5], [611, 2, 5]),
                                       ([260, 0, 40], [0, 0, 40]), ([384], [384])])
@pytest.mark.parametrize("strided", [False, True])
def test_append(V, lens, news, strided):
    c = R.make_case(lens, news, 3, seed=31)
    K, W = R.rows(sum(news) + 2, 3, seed=32, strided=strided), R.rows(sum(news) + 2, 3, seed=33, strided=strided)
    # a large token makes the scale of an open page grow, a small chunk lets it stand
    K[0] *= 64
    cache, start = c.on(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    big_k = torch.empty((K.shape[0], 5, 128), dtype=torch.bfloat16, device="cuda")[:, 1:4].copy_(K) if strided else K.cuda()
    V.cache_append(cache, big_k, W.cuda(), start, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    R.append(c, K, W)
    for got, ref in ((cache.k8, c.k8), (cache.v8, c.v8)):
        _same_codes(got, ref)
    assert torch.equal(cache.sk.cpu(), c.sk) and torch.equal(cache.sv.cpu(), c.sv)


def test_append_of_extremes(V):
    """Zeros, the largest and the smallest bf16, values at the border of a scale, NaN and infinities."""
    c = R.make_case([150], [150], 2, seed=34)
    K = R.rows(150, 2, seed=35)
    K[:128, 0] = 0
    K[:128, 1] = 448.0
    K[130, 0, 3], K[130, 0, 4], K[131, 0, 5] = math.nan, math.inf, -math.inf
    W = K.clone()
    W[:, 0] = 3.3e38
    W[:, 1] = 1e-39
    W[5, 1, 7] = 450.0
    cache, start = c.on(V)
    V.cache_append(cache, K.cuda(), W.cuda(), start)
    R.append(c, K, W)
    _same_codes(cache.k8, c.k8)
    _same_codes(cache.v8, c.v8)
    assert torch.equal(cache.sk.cpu(), c.sk) and torch.equal(cache.sv.cpu(), c.sv)


@pytest.mark.parametrize("lens,budget,recent", [([1, 300, 129], 100, 20), ([1000, 640], 257, 0), ([500], 130, 130),
                                                ([40, 0, 200], 300, 7), ([5000, 1300], 1024, 100), ([129], 1, 0)])
def test_evict(V, lens, budget, recent):
    H = 3
    cols = -(-budget // 128) + 1
    c = R.make_case(lens, [0] * len(lens), H, seed=41, spare=len(lens) * cols, scales=(-6, -7, -9))
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(len(c.sk)) if p not in used]
    dst = torch.full((len(lens), cols), -1, dtype=torch.int32)
    for b, m in enumerate(lens):
        for j in range(-(-min(m, budget) // 128)):
            dst[b, j] = free.pop()
    g = torch.Generator().manual_seed(42)
    weight = torch.rand((*c.sk.shape, 128), generator=g).round(decimals=1) - 0.3      # many ties
    weight[torch.rand(weight.shape, generator=g) < 0.05] = math.nan
    weight[torch.rand(weight.shape, generator=g) < 0.02] = math.inf
    weight[torch.rand(weight.shape, generator=g) < 0.02] = -math.inf
    weight[torch.rand(weight.shape, generator=g) < 0.02] = -0.0
    kept = torch.full((len(lens), H, budget), -1, dtype=torch.int32)
    cache, _ = c.on(V)
    got_w, got_kept = weight.cuda(), kept.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_len, _ = V.cache_evict(cache, got_w, dst.cuda(), budget, recent, kept=got_kept, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    ref_len = R.evict(c, weight, dst, budget, recent, kept)
    assert torch.equal(new_len.cpu(), ref_len) and torch.equal(got_kept.cpu(), kept)
    _same_codes(cache.k8, c.k8)
    _same_codes(cache.v8, c.v8)
    assert torch.equal(cache.sk.cpu(), c.sk) and torch.equal(cache.sv.cpu(), c.sv)
    assert torch.equal(got_w.cpu().view(torch.int32), weight.view(torch.int32))


def test_equal_calls_give_equal_bits(V):
    for lens, news in (([20011, 300], [1, 1]), ([3000, 900], [200, 100])):
        c = R.make_case(lens, news, 2, seed=51)
        cache, start = c.on(V)
        Q = R.rows(sum(news), 8, seed=52).cuda()
        first = V.cache_attention(cache, Q, start)
        w1 = torch.zeros((*c.sk.shape, 128), device="cuda")
        V.cache_weigh(cache, Q, start, first[1], w1)
        for _ in range(3):
            again = V.cache_attention(cache, Q, start)
            assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
            w2 = torch.zeros_like(w1)
            V.cache_weigh(cache, Q, start, again[1], w2)
            assert torch.equal(w1, w2)


def test_a_sequence_of_calls(V):
    """A prompt, an eviction, then tokens: append, attend, weigh and evict one
    after another as a server runs them, on a stream of its own, against the
    reference doing the same."""
    H, Hq, B = 2, 6, 2
    lens = [300, 170]
    c = R.make_case([0, 0], [0, 0], H, cols=4, seed=61, spare=16)
    c.table[0, :4] = torch.tensor([3, 9, 1, 12])
    c.table[1, :4] = torch.tensor([7, 0, 14, 5])
    cache, _ = c.on(V)
    weight = torch.zeros((*c.sk.shape, 128))
    got_w = weight.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step(news, seed):
        nonlocal weight
        c.length += torch.tensor(news, dtype=torch.int32)
        c.start = torch.tensor([0, news[0], sum(news)], dtype=torch.int32)
        K, W = R.rows(sum(news), H, seed), R.rows(sum(news), H, seed + 1, outliers=False)
        Q = R.rows(sum(news), Hq, seed + 2)
        with torch.cuda.stream(side):
            cache.length.copy_(c.length)
            start = c.start.cuda()
            V.cache_append(cache, K.cuda(), W.cuda(), start)
            out, lse = V.cache_attention(cache, Q.cuda(), start, softcap=25.0)
            V.cache_weigh(cache, Q.cuda(), start, lse, got_w, softcap=25.0)
        side.synchronize()
        R.append(c, K, W)
        _same_codes(cache.k8, c.k8)
        _same_codes(cache.v8, c.v8)
        o, z, eo, el = R.attention(c, Q, softcap=25.0)
        _within(out, o, eo, "O")
        _within(lse, z, el, "lse")
        w, e = R.weigh(c, Q, lse.cpu(), weight, softcap=25.0)
        _within(got_w, w, e, "weight")
        weight = got_w.cpu()

    step(lens, 100)
    dst = torch.tensor([[2, 4, 6], [8, 10, 11]], dtype=torch.int32)
    kept = torch.full((B, H, 150), -1, dtype=torch.int32)
    with torch.cuda.stream(side):
        new_len, got_kept = V.cache_evict(cache, got_w, dst.cuda(), 150, 30)
    side.synchronize()
    ref_len = R.evict(c, weight, dst, 150, 30, kept)
    assert torch.equal(new_len.cpu(), ref_len) and torch.equal(got_kept.cpu(), kept)
    _same_codes(cache.k8, c.k8)
    c.table, c.length = dst, ref_len
    cache = V.Cache(cache.k8, cache.v8, cache.sk, cache.sv, dst.cuda(), new_len)
    for i in range(3):
        step([1, 2], 200 + 10 * i)
    step([0, 1], 300)


def test_capture_and_replay(V):
    """A captured step replays with new rows, lengths and tables in the same buffers."""
    lens, news, H, Hq = [200, 700], [1, 1], 2, 4
    c = R.make_case([m - 1 for m in lens], [0, 0], H, cols=8, seed=71, spare=4)
    c.length += 1
    c.start = torch.tensor([0, 1, 2], dtype=torch.int32)
    cache, start = c.on(V)
    K, W = R.rows(2, H, 72).cuda(), R.rows(2, H, 73).cuda()
    Q = R.rows(2, Hq, 74).cuda()
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    ws = torch.empty(max(16, V.vca_cache_workspace_bytes(V.VCA_OP_CACHE_ATTENTION, 2, Hq, H, 2, 8),
                         V.vca_cache_workspace_bytes(V.VCA_OP_CACHE_WEIGH, 2, Hq, H, 2, 8)), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty((2, Hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((2, Hq), device="cuda")

    def step():
        V.cache_append(cache, K, W, start)
        V.cache_attention(cache, Q, start, out=out, lse=lse, ws=ws)
        V.cache_weigh(cache, Q, start, lse, weight, ws=ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        if i:
            c.length += 1
            cache.length.copy_(c.length)
            K.copy_(R.rows(2, H, 80 + i))
            W.copy_(R.rows(2, H, 90 + i))
            Q.copy_(R.rows(2, Hq, 95 + i))
        weight.zero_()
        graph.replay()
        torch.cuda.synchronize()
        R.append(c, K.cpu(), W.cpu())
        _same_codes(cache.k8, c.k8)
        o, z, eo, el = R.attention(c, Q.cpu())
        _within(out, o, eo, "O")
        _within(lse, z, el, "lse")
        w, e = R.weigh(c, Q.cpu(), lse.cpu(), torch.zeros(weight.shape))
        _within(weight, w, e, "weight")
