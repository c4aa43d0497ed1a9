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


@pytest.mark.parametrize("news", [1, 30])
def test_starts_that_fall_end_the_list(V, news):
    """Every second sequence's start falls and the others claim every row: the
    rows of those before the first fall are right, the rest counts as none,
    whatever number of rows the list would come to."""
    B, H, Hq = 70, 2, 4
    T = B * news
    c = R.make_case([200] * 2, [T, 0], H, seed=81)
    c.table = c.table[:1].repeat(B, 1)
    c.length = c.length[:1].repeat(B)
    good = c.clone()
    good.start = torch.tensor([0] + [T] * B, dtype=torch.int32)
    c.start = torch.tensor([T * (b & 1) for b in range(B + 1)], dtype=torch.int32)
    Q = R.rows(T, Hq, seed=82)
    o, z, eo, el = R.attention(good, Q, causal=False)
    cache, start = c.on(V)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.cache_attention(cache, Q.cuda(), start, causal=False, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == V.VCA_ERR_INVALID_ARG
    _within(out, o, eo, "O")
    _within(lse, z, el, "lse")
    for causal in (False, True):
        _, z, _, _ = R.attention(good, Q, causal=causal)
        w, e = R.weigh(good, Q, z.float(), torch.zeros((*c.sk.shape, 128)), causal=causal)
        weight = torch.zeros((*c.sk.shape, 128), device="cuda")
        status.zero_()
        V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), weight, causal=causal, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == V.VCA_ERR_INVALID_ARG
        _within(weight, w, e, "weight")
    K = R.rows(T, H, seed=83)
    before = cache.k8.clone()
    status.zero_()
    V.cache_append(cache, K.cuda(), K.cuda(), start, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == V.VCA_ERR_INVALID_ARG
    if T > 200:      # more rows than tokens: sequence 0 is invalid too
        assert torch.equal(cache.k8, before)
    else:
        R.append(good, K, K)
        _same_codes(cache.k8, good.k8)


@pytest.mark.parametrize("news", [1, 20])
def test_many_sequences(V, news):
    """More than 32 sequences; one of the last has a bad length and only it suffers."""
    B, H, Hq = 75, 2, 4
    lens = [20 + (37 * b) % 300 for b in range(B)]
    c = R.make_case(lens, [news] * B, H, seed=84)
    Q = R.rows(B * news, Hq, seed=85)
    _check_attention(V, c, Q, causal=True)
    _, z, _, _ = R.attention(c, Q)
    for bad in (False, True):
        d, keep = c.clone(), c.clone()
        if bad:
            d.length[70] = 1 << 20
            keep.length[70] = 0
        w, e = R.weigh(keep, Q, z.float(), torch.zeros((*c.sk.shape, 128)))
        cache, start = d.on(V)
        weight = torch.zeros((*c.sk.shape, 128), device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), weight, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == (V.VCA_ERR_INVALID_ARG if bad else 0)
        _within(weight, w, e, "weight")


@pytest.mark.parametrize("name", ["five to a head", "a chunk", "wide rows"])
@pytest.mark.parametrize("softcap", [1e-3, 4.0, 1000.0, 1e6, 1e30])
def test_caps_of_any_size(V, name, softcap):
    lens, news, Hq, H = BATCHES[name]
    c = R.make_case(lens, news, H, seed=11)
    Q = R.rows(sum(news), Hq, seed=86)
    _, lse = _check_attention(V, c, Q, causal=True, softcap=softcap)
    w, e = R.weigh(c, Q, lse.cpu(), torch.zeros((*c.sk.shape, 128)), softcap=softcap)
    cache, start = c.on(V)
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    V.cache_weigh(cache, Q.cuda(), start, lse, weight, softcap=softcap)
    _within(weight, w, e, "weight")


def test_heads_in_rounds(V):
    """So many rows that the queries of all heads are not laid out at once."""
    H, n = 16, 16100
    c = R.make_case([64], [n], H, seed=87)
    _check_attention(V, c, R.rows(n, H, seed=88), causal=False)


def test_queries_that_are_not_finite(V):
    """A NaN or an infinity in a row stays in that row."""
    for news in ([1, 1], [70, 60]):
        c = R.make_case([200, 300], news, 2, seed=89)
        Q = R.rows(sum(news), 4, seed=90)
        o, z, eo, el = R.attention(c, Q)
        Q[0, 1, 5], Q[-1, 3, 100], Q[-1, 2, 0] = math.nan, math.inf, -math.inf
        cache, start = c.on(V)
        out, lse = V.cache_attention(cache, Q.cuda(), start)
        bad = torch.zeros(Q.shape[:2], dtype=torch.bool)
        bad[0, 1] = bad[-1, 3] = bad[-1, 2] = True
        assert bool(torch.isnan(out.cpu()[bad]).all())
        _within(out.cpu()[~bad], o[~bad], eo[~bad], "O")
        _within(lse.cpu()[~bad], z[~bad], el[~bad], "lse")


def test_empty_caches(V):
    """Rows of sequences without tokens: O = 0, lse = -inf, nothing weighed."""
    for news in ([1, 2], [40, 90]):
        c = R.make_case([0, 0], news, 2, seed=91)
        Q = R.rows(sum(news), 4, seed=92)
        out, lse = _check_attention(V, c, Q, causal=False)
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())
        cache, start = c.on(V)
        weight = torch.full((*c.sk.shape, 128), 0.5, device="cuda")
        V.cache_weigh(cache, Q.cuda(), start, lse, weight, causal=False)
        kept = torch.full((2, 2, 5), -1, dtype=torch.int32, device="cuda")
        new_len, _ = V.cache_evict(cache, weight, torch.zeros((2, 1), dtype=torch.int32, device="cuda"), 5, 2, kept=kept)
        assert bool((weight == 0.5).all()) and bool((new_len == 0).all()) and bool((kept == -1).all())


def test_shared_pages(V):
    """Two sequences with a common prompt read the same pages; their weights add up."""
    for news in ([1, 1], [50, 70]):
        c = R.make_case([400, 390], news, 2, seed=93)
        c.table[1, :2] = c.table[0, :2]
        Q = R.rows(sum(news), 4, seed=94)
        _, lse = _check_attention(V, c, Q, causal=True)
        w, e = R.weigh(c, Q, lse.cpu(), torch.zeros((*c.sk.shape, 128)))
        cache, start = c.on(V)
        weight = torch.zeros((*c.sk.shape, 128), device="cuda")
        V.cache_weigh(cache, Q.cuda(), start, lse, weight)
        _within(weight, w, e, "weight")


def test_pages_that_repeat_in_a_long_table(V):
    """A table may name a page many times: more tokens than the pool holds."""
    c = R.make_case([300], [1], 1, seed=95)
    c.table = c.table[:, :2].repeat(1, 700)
    c.length[0] = 1400 * 128 - 5
    _check_attention(V, c, R.rows(1, 2, seed=96))
    c.start[1] = 12
    _check_attention(V, c, R.rows(12, 2, seed=97))


@pytest.mark.parametrize("len_,budget,recent", [(20000, 900, 100), (170000, 300, 40), (170000, 200, 0)])
def test_evict_of_long_sequences(V, len_, budget, recent):
    """Several CTAs to a head, and runs that a CTA's shared memory does not hold."""
    cols = -(-budget // 128)
    c = R.make_case([len_, 700], [0, 0], 1, seed=98, spare=2 * cols)
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(len(c.sk)) if p not in used]
    dst = torch.tensor(free[:2 * cols], dtype=torch.int32).view(2, cols)
    g = torch.Generator().manual_seed(99)
    weight = torch.rand((*c.sk.shape, 128), generator=g)
    if recent == 0:
        weight = (weight * 4).floor()      # mostly ties
    kept = torch.full((2, 1, budget), -1, dtype=torch.int32)
    cache, _ = c.on(V)
    got_w, got_kept = weight.cuda(), kept.cuda()
    new_len, _ = V.cache_evict(cache, got_w, dst.cuda(), budget, recent, kept=got_kept)
    torch.cuda.synchronize()
    ref_len = R.evict(c, weight, dst, budget, recent, kept)
    assert torch.equal(new_len.cpu(), ref_len) and torch.equal(got_kept.cpu(), kept)
    _same_codes(cache.k8, c.k8)
    _same_codes(cache.v8, c.v8)
    assert torch.equal(cache.sk.cpu(), c.sk) and torch.equal(got_w.cpu(), weight)


def test_a_pool_beyond_32_bits(V):
    """Pages whose codes lie more than 4 GB into the pool."""
    c = R.make_case([330, 140], [10, 3], 1, seed=100, spare=4)
    small, far = len(c.sk), 270000
    cache, start = c.on(V)

    def wide(x):
        y = torch.zeros((far + small, *x.shape[1:]), dtype=x.dtype, device="cuda")
        y[far:] = x
        return y

    table = torch.where(cache.table >= 0, cache.table + far, cache.table)
    big = V.Cache(wide(cache.k8), wide(cache.v8), wide(cache.sk), wide(cache.sv), table, cache.length)
    K, W, Q = R.rows(13, 1, 101), R.rows(13, 1, 102), R.rows(13, 2, 103)
    V.cache_append(big, K.cuda(), W.cuda(), start)
    R.append(c, K, W)
    _same_codes(big.k8[far:], c.k8)
    _same_codes(big.v8[far:], c.v8)
    for rows in ([0, 10, 13], [0, 2, 3]):
        c.start = torch.tensor(rows, dtype=torch.int32)
        o, z, eo, el = R.attention(c, Q[:rows[2]])
        out, lse = V.cache_attention(big, Q[:rows[2]].cuda(), c.start.cuda())
        _within(out, o, eo, "O")
        weight = torch.zeros((*big.sk.shape, 128), device="cuda")
        V.cache_weigh(big, Q[:rows[2]].cuda(), c.start.cuda(), lse, weight)
        w, e = R.weigh(c, Q[:rows[2]], lse.cpu(), torch.zeros((*c.sk.shape, 128)))
        _within(weight[far:], w, e, "weight")
    used = set(c.table[c.table >= 0].tolist())
    dst = torch.tensor([p for p in range(small) if p not in used][:4], dtype=torch.int32).view(2, 2)
    kept = torch.full((2, 1, 130), -1, dtype=torch.int32)
    _, got_kept = V.cache_evict(big, weight, dst.cuda() + far, 130, 20)
    w = weight[far:].cpu()
    R.evict(c, w, dst, 130, 20, kept)
    assert torch.equal(got_kept.cpu(), kept)
    _same_codes(big.k8[far:], c.k8)
    assert torch.equal(big.sv[far:].cpu(), c.sv)


@pytest.mark.parametrize("news", [[1, 1, 1], [90, 40, 70]])
def test_two_streams_at_once(V, news):
    """Calls that overlap, each with a workspace of its own, do not disturb one another."""
    cases = [R.make_case([9000, 300, 1200], news, 2, seed=s) for s in (104, 105)]
    Q = [R.rows(sum(news), 8, seed=s).cuda() for s in (106, 107)]
    on = [c.on(V) for c in cases]
    alone = [V.cache_attention(cache, q, start) for (cache, start), q in zip(on, Q)]
    weights = [torch.zeros((*c.sk.shape, 128), device="cuda") for c in cases]
    for (cache, start), q, (_, lse), w in zip(on, Q, alone, weights):
        V.cache_weigh(cache, q, start, lse, w)
    streams = [torch.cuda.Stream() for _ in cases]
    got, gw = [[] for _ in cases], [[] for _ in cases]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                cache, start = on[i]
                got[i].append(V.cache_attention(cache, Q[i], start))
                gw[i].append(torch.zeros_like(weights[i]))
                V.cache_weigh(cache, Q[i], start, got[i][-1][1], gw[i][-1])
    torch.cuda.synchronize()
    for i in range(len(cases)):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
        for w in gw[i]:
            assert torch.equal(w, weights[i])


def test_an_eviction_replayed(V):
    """A captured eviction replays with other lengths and weights."""
    H, budget, recent = 2, 200, 30
    c = R.make_case([700, 150], [0, 0], H, seed=108, spare=4)
    used = set(c.table[c.table >= 0].tolist())
    dst = torch.tensor([p for p in range(len(c.sk)) if p not in used][:4], dtype=torch.int32).view(2, 2)
    cache, _ = c.on(V)
    weight, got_dst = torch.zeros((*c.sk.shape, 128), device="cuda"), dst.cuda()
    new_len = torch.empty(2, dtype=torch.int32, device="cuda")
    kept = torch.empty((2, H, budget), dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.vca_cache_evict(cache, weight, got_dst, budget, recent, new_len, kept)
    for i, lens in enumerate(([700, 150], [333, 1])):
        w = torch.rand(weight.shape, generator=torch.Generator().manual_seed(109 + i))
        c.length = torch.tensor(lens, dtype=torch.int32)
        cache.length.copy_(c.length)
        weight.copy_(w)
        kept.fill_(-1)
        graph.replay()
        torch.cuda.synchronize()
        ref = torch.full((2, H, budget), -1, dtype=torch.int32)
        assert torch.equal(new_len.cpu(), R.evict(c, w, dst, budget, recent, ref))
        assert torch.equal(kept.cpu(), ref)
        _same_codes(cache.k8, c.k8)
        assert torch.equal(weight.cpu(), w)


@pytest.mark.parametrize("causal", [True, False])
def test_pages_of_nan(V, causal):
    """Whole pages of NaN keys: the call ends, and only rows that see them are NaN."""
    for news in ([1, 1], [70, 200]):
        c = R.make_case([500, 300], news, 2, seed=111)
        Q = R.rows(sum(news), 4, seed=112)
        o, z, eo, el = R.attention(c, Q, causal=causal)
        c.k8[c.table[0, 1].long()] = 0x7F
        n0 = news[0]
        for cap in (0.0, 20.0):
            cache, start = c.on(V)
            out, lse = V.cache_attention(cache, Q.cuda(), start, causal=causal, softcap=cap)
            assert bool(torch.isnan(out[:n0]).all()) and bool(torch.isnan(lse[:n0]).all())
            if cap == 0.0:
                _within(out[n0:], o[n0:], eo[n0:], "O")
                _within(lse[n0:], z[n0:], el[n0:], "lse")
            weight = torch.zeros((*c.sk.shape, 128), device="cuda")
            V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), weight, causal=causal, softcap=cap)
            page = c.table[0, 1].long()
            assert bool(torch.isnan(weight[page]).all())
            weight[page] = 0
            assert bool(torch.isfinite(weight).all())


@pytest.mark.parametrize("pages", [1, 3, 8, 19])
def test_weights_of_ragged_rows(V, pages):
    """Few rows on average, several hundred of some sequences: many tiles of 16 rows to a page."""
    for news in ([12] * 4 + [1] * 12, [60] + [1] * 15, [30, 2, 30] + [1] * 13):
        lens = [pages * 128 - 11 * (b % 7) for b in range(16)]
        c = R.make_case(lens, news, 2, seed=113)
        Q = R.rows(sum(news), 16, seed=114)
        for causal in (True, False):
            _, z, _, _ = R.attention(c, Q, causal=causal)
            w, e = R.weigh(c, Q, z.float(), torch.zeros((*c.sk.shape, 128)), causal=causal)
            cache, start = c.on(V)
            for _ in range(5):
                status = torch.zeros(1, dtype=torch.int32, device="cuda")
                weight = torch.zeros((*c.sk.shape, 128), device="cuda")
                V.cache_weigh(cache, Q.cuda(), start, z.float().cuda(), weight, causal=causal, dev_status=status)
                torch.cuda.synchronize()
                assert int(status) == 0
                _within(weight, w, e, "weight")


# between a tile of eight rows and one of 128: lengths, new rows, query heads, KV heads
MIDDLE = {
    "nine rows": ([700], [9], 1, 1),
    "a full tile": ([1500, 129], [8, 8], 8, 2),
    "five tokens": ([9000, 40, 1300], [5, 5, 5], 20, 4),
    "one much longer": ([800, 300, 90, 700, 128, 256], [40, 1, 1, 2, 1, 1], 6, 2),
    "long": ([30011], [7], 8, 2),
    "many short": ([130 + 7 * b for b in range(80)], [3] * 80, 16, 4),
    "in front of the cache": ([2, 300], [6, 6], 8, 2),
}


@pytest.mark.parametrize("softcap", [0.0, 30.0, 0.5])
@pytest.mark.parametrize("name", MIDDLE)
def test_attention_of_middle_rows(V, name, softcap):
    lens, news, Hq, H = MIDDLE[name]
    c = R.make_case(lens, news, H, seed=115)
    for causal in (True, False):
        first = _check_attention(V, c, R.rows(sum(news), Hq, seed=116), causal=causal, softcap=softcap)
        again = _check_attention(V, c, R.rows(sum(news), Hq, seed=116), causal=causal, softcap=softcap)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_middle_rows_of_nan_and_far_scales(V):
    c = R.make_case([900, 500], [7, 4], 1, seed=117)
    for j, e in enumerate([-6, -30, -7, -120, -3, -60, 10, -6]):
        p = int(c.table[0, j])
        c.sv[p] = 2.0 ** e
        if e == -120:
            c.v8[p] = 0
        c.sk[p] = 2.0 ** -7
    Q = R.rows(11, 3, seed=118)
    _check_attention(V, c, Q, causal=True)
    o, z, eo, el = R.attention(c, Q)
    Q[2, 1, 5], Q[9, 0, 7] = math.nan, math.inf
    cache, start = c.on(V)
    out, lse = V.cache_attention(cache, Q.cuda(), start)
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool)
    bad[2, 1] = bad[9, 0] = True
    assert bool(torch.isnan(out.cpu()[bad]).all())
    _within(out.cpu()[~bad], o[~bad], eo[~bad], "O")
    _within(lse.cpu()[~bad], z[~bad], el[~bad], "lse")


def test_a_stream_that_is_named(V):
    """The entries with a stream argument run there, whatever the current stream is."""
    c = R.make_case([300, 90], [5, 6], 2, seed=119, spare=5)
    K, Q = R.rows(11, 2, 120), R.rows(11, 4, 121)
    cache, start = c.on(V)
    side = torch.cuda.Stream()
    Kd, Qd = K.cuda(), Q.cuda()
    out, lse = torch.empty((11, 4, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((11, 4), device="cuda")
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    ws = torch.empty(max(V.vca_cache_workspace_bytes(op, 11, 4, 2, *c.table.shape)
                         for op in (V.VCA_OP_CACHE_ATTENTION, V.VCA_OP_CACHE_WEIGH)), dtype=torch.uint8, device="cuda")
    used = set(c.table[c.table >= 0].tolist())
    dst = torch.tensor([p for p in range(len(c.sk)) if p not in used][:4], dtype=torch.int32).view(2, 2)
    dd = dst.cuda()
    new_len, kept = torch.empty(2, dtype=torch.int32, device="cuda"), torch.full((2, 2, 200), -1, dtype=torch.int32, device="cuda")
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 1e-2      # the calls must wait for this on `side`
        V.vca_cache_append(cache, Kd, Kd, start, stream=side)
    V.vca_cache_attention(cache, Qd, start, 1, 0.0, 0.0, out, lse, ws, stream=side)
    V.vca_cache_weigh(cache, Qd, start, 1, 0.0, 0.0, lse, weight, ws, stream=side)
    V.vca_cache_evict(cache, weight, dd, 200, 20, new_len, kept, stream=side)
    side.synchronize()
    R.append(c, K, K)
    o, z, eo, el = R.attention(c, Q)
    _within(out, o, eo, "O")
    _within(lse, z, el, "lse")
    got = weight.cpu()
    w, e = R.weigh(c, Q, lse.cpu(), torch.zeros(got.shape))
    for b in range(2):
        for p in c.table[b, :-(-int(c.length[b]) // 128)].tolist():
            _within(got[p], w[p], e[p], "weight")
    ref = torch.full((2, 2, 200), -1, dtype=torch.int32)
    assert torch.equal(new_len.cpu(), R.evict(c, got.clone(), dst, 200, 20, ref)) and torch.equal(kept.cpu(), ref)
    _same_codes(cache.k8, c.k8)


def test_calls_without_rows(V):
    c = R.make_case([300], [0], 2, seed=122)
    cache, start = c.on(V)
    K, Q = R.rows(0, 2, 1).cuda(), R.rows(0, 4, 1).cuda()
    before = cache.k8.clone()
    V.cache_append(cache, K, K, start)
    out, lse = V.cache_attention(cache, Q, start)
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    V.cache_weigh(cache, Q, start, lse, weight)
    assert out.shape == (0, 4, 128) and lse.shape == (0, 4) and not bool(weight.any()) and torch.equal(cache.k8, before)


def test_middle_rows_beside_bad_sequences(V):
    """A bad page or length of one sequence leaves the others right, and rows behind the last stay."""
    news = [6, 6, 6]
    c = R.make_case([200, 140, 300], news, 2, seed=123, cols=3)
    Q = R.rows(sum(news) + 2, 4, seed=124)
    o, z, eo, el = R.attention(c, Q)
    for kind in ("page", "length"):
        d = c.clone()
        if kind == "page":
            d.table[1, 0] = 1 << 30
        else:
            d.length[1] = -7
        cache, start = d.on(V)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((20, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((20, 4), 7.0, device="cuda")
        V.cache_attention(cache, Q.cuda(), start, out=out, lse=lse, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == V.VCA_ERR_INVALID_ARG, kind
        assert bool((out[18:] == 7).all()) and bool((lse[18:] == 7).all())
        for sl in (slice(0, 6), slice(12, 18)):
            _within(out[sl], o[sl], eo[sl], f"O ({kind})")
            _within(lse[sl], z[sl], el[sl], f"lse ({kind})")
