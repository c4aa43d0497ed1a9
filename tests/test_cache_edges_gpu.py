"""The 8-bit cache at the edges of what its documentation allows -- page scales that
fall again and again, caps and scales of any size, pages used twice, budgets
beyond the cache -- against the 64-bit reference (cache_reference.py)."""
import math

import pytest
import torch

import cache_reference as R
from test_cache_gpu import _check_attention, _same_codes, _within

pytestmark = pytest.mark.gpu

# new rows of a sequence, sequences, KV heads: a token, tiles of 32 rows and of 128,
# cut into parts of pages (few tiles) and whole (too many tiles to be cut)
FORMS = {"a token": (1, 1, 2), "32 rows, cut": (20, 1, 2), "32 rows, whole": (20, 8, 24), "128 rows, cut": (130, 1, 2),
         "128 rows, whole": (130, 8, 20)}
Z = None      # a page of zeros, which append gives the scale 2^-120
FALLS = {
    "two zeros at the end": [-6] * 10 + [Z, Z],
    "three zeros in the middle": [-6] * 5 + [Z] * 3 + [-6] * 4,
    "ten zeros": [-6] * 4 + [Z] * 10 + [-6, -7],
    "zeros first": [Z, Z, -6, -6, Z, Z, -7, -6],
    "down and up": [-6, -6, Z, Z, -6, -5, Z, Z, 3, -6, Z, Z],
    "steps": [-6] * 6 + [-40, -75, -110, -120] + [-7, -6],
    "small ones at the end": [-6] * 4 + [-30, -60, -90, -118],
}


def _case_of_scales(scales, news, B, H, seed):
    """B sequences over the same pages; V of one sign, so that O grows with every token."""
    c = R.make_case([128 * len(scales) - 3], [0], H, seed=seed)
    g = torch.Generator().manual_seed(seed + 1)
    for j, e in enumerate(scales):
        p = int(c.table[0, j])
        v = torch.randn((H, 128, 128), generator=g).abs() * 32 + 256
        c.v8[p] = 0 if e is Z else v.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8)
        c.sv[p] = 2.0 ** (-120 if e is Z else e)
    c.v8[int(c.table[0, -1]), :, 125:] = 0x7F      # behind the last token
    c.table, c.length = c.table.repeat(B, 1), c.length.repeat(B)
    c.start = torch.arange(B + 1, dtype=torch.int32) * news
    return c


@pytest.mark.parametrize("softcap", [0.0, 20.0])
@pytest.mark.parametrize("name", FALLS)
@pytest.mark.parametrize("form", FORMS)
def test_scales_that_fall_again(V, form, name, softcap):
    """O is summed in units that follow the pages' scales down: it stays finite
    however often they fall, with weights spread over every token."""
    news, B, H = FORMS[form]
    c = _case_of_scales(FALLS[name], news, B, H, seed=201)
    Q = (R.rows(news * B, H, seed=202).float() * 0.05).to(torch.bfloat16)
    _check_attention(V, c, Q, causal=B == 1, softcap=softcap)


@pytest.mark.parametrize("form", FORMS)
def test_outputs_of_the_smallest_scale(V, form):
    """All values equal, at the scale 2^-120, and softmax sums of 2^25 in units of
    the reference maximum, which the first page's scores set 2^7.65 below the others':
    the outputs are the value, to bf16 (2^-8), the probabilities' fp16 (2^-11) and
    1,400 pages' eight additions of products (2^-23 each)."""
    news, B, H = FORMS[form]
    c = R.make_case([256], [0], H, seed=203)
    first, other = c.table[0].tolist()
    c.k8[first] = 0
    c.k8[other] = torch.tensor(0.46875).to(torch.float8_e4m3fn).view(torch.uint8)
    c.sk[:] = 1.0
    c.v8[:] = torch.tensor(288.0).to(torch.float8_e4m3fn).view(torch.uint8)
    c.sv[:] = 2.0 ** -120
    c.table = torch.tensor([[first] + [other] * 1399] * B, dtype=torch.int32)
    c.length = torch.full((B,), 1400 * 128 - 5, dtype=torch.int32)
    c.start = torch.arange(B + 1, dtype=torch.int32) * news
    cache, start = c.on(V)
    out, _ = V.cache_attention(cache, torch.ones((news * B, H, 128), dtype=torch.bfloat16, device="cuda"), start, causal=False)
    off = (out.double() / (288.0 * 2.0 ** -120) - 1.0).abs().max()
    assert float(off) <= 2.0 ** -8 + 2.0 ** -11 + 1400 * 8 * 2.0 ** -23


def _check_weigh(V, c, Q, lse, **kw):
    cache, start = c.on(V)
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    V.cache_weigh(cache, Q.cuda(), start, lse, weight, **kw)
    w, e = R.weigh(c, Q, lse.cpu(), torch.zeros(weight.shape), **kw)
    _within(weight, w, e, "weight")


# a token, middle rows, many rows: lengths, new rows, query heads, KV heads
ROWS = {"tokens": ([700, 129], [1, 1], 6, 2), "middle": ([1500, 260], [5, 4], 10, 2), "many": ([900, 333], [150, 40], 4, 2)}


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("softcap", [1e-30, 2.0 ** -40, 2.0 ** 39, 2.0 ** 40, 1e20, 1e36, 8e37])
def test_caps_at_the_ends_of_their_range(V, name, softcap):
    """A cap of any accepted size: tiny ones leave no score, huge ones every score."""
    lens, news, Hq, H = ROWS[name]
    c = R.make_case(lens, news, H, seed=211)
    Q = R.rows(sum(news), Hq, seed=212)
    _, lse = _check_attention(V, c, Q, causal=True, softcap=softcap)
    _check_weigh(V, c, Q, lse, softcap=softcap)


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("softcap", [1e-30, 30.0, 1e6, 2.0 ** 39, 1e30])
@pytest.mark.parametrize("magnitude", [2.0 ** -50, 2.0 ** 50])
def test_caps_of_queries_of_any_magnitude(V, name, softcap, magnitude):
    """Page scales far from 1 against queries far from 1, with a cap."""
    lens, news, Hq, H = ROWS[name]
    c = R.make_case(lens, news, H, seed=213)
    c.sk *= 1.0 / magnitude
    Q = (R.rows(sum(news), Hq, seed=214).double() * magnitude).to(torch.bfloat16)
    _, lse = _check_attention(V, c, Q, causal=True, softcap=softcap)
    _check_weigh(V, c, Q, lse, softcap=softcap)


def test_pages_used_twice(V):
    """Append, attend, weigh and evict in a pool whose pages, weights included, held
    other tokens before: a new token's weight starts at 0, also in the slots behind
    an eviction's last token, and other slots' weights stay."""
    H, Hq, B, budget, recent = 2, 6, 2, 200, 20
    c = R.make_case([0, 0], [0, 0], H, cols=4, seed=221, spare=12)
    g = torch.Generator().manual_seed(222)
    c.k8, c.v8 = R.random_codes(g, c.k8.shape), R.random_codes(g, c.v8.shape)
    weight = torch.rand((*c.sk.shape, 128), generator=g) * 100.0
    got = weight.cuda()
    cache, _ = c.on(V)

    def new_slots(news):
        for b, n in enumerate(news):
            for t in range(int(c.length[b]) - n, int(c.length[b])):
                weight[int(c.table[b, t // 128]), :, t % 128] = 0.0

    def step(news, seed):
        nonlocal weight
        c.length += torch.tensor(news, dtype=torch.int32)
        c.start = torch.tensor([0, news[0], sum(news)], dtype=torch.int32)
        K, W, Q = R.rows(sum(news), H, seed), R.rows(sum(news), H, seed + 1, outliers=False), R.rows(sum(news), Hq, seed + 2)
        cache.length.copy_(c.length)
        start = c.start.cuda()
        V.cache_append(cache, K.cuda(), W.cuda(), start, weight=got)
        R.append(c, K, W)
        new_slots(news)
        assert torch.equal(got.cpu(), weight)
        out, lse = V.cache_attention(cache, Q.cuda(), start)
        V.cache_weigh(cache, Q.cuda(), start, lse, got)
        w, e = R.weigh(c, Q, lse.cpu(), weight)
        _within(got, w, e, "weight")
        weight = got.cpu()

    def cut(pages):
        dst = torch.tensor(pages, dtype=torch.int32).view(B, 2)
        kept = torch.full((B, H, budget), -1, dtype=torch.int32)
        new_len, got_kept = V.cache_evict(cache, got, dst.cuda(), budget, recent)
        ref = R.evict(c, weight, dst, budget, recent, kept)
        assert torch.equal(new_len.cpu(), ref) and torch.equal(got_kept.cpu(), kept) and torch.equal(got.cpu(), weight)
        c.table = torch.cat([dst, torch.full((B, 2), -1, dtype=torch.int32)], 1)
        c.length = ref.clone()
        cache.table.copy_(c.table)

    c.table = torch.tensor([[0, 1, 2, -1], [3, 4, 5, -1]], dtype=torch.int32)
    cache.table.copy_(c.table)
    step([300, 140], 230)
    cut([6, 7, 8, 9])
    step([1, 1], 240)
    step([40, 100], 250)      # into the pages that the eviction filled in part, and one more of the first sequence's
    c.table[:, 2] = torch.tensor([0, 3])      # pages of tokens that are gone
    cache.table.copy_(c.table)
    step([60, 30], 260)
    cut([1, 2, 4, 5])
    step([3, 2], 270)


@pytest.mark.parametrize("budget", [1000, 2 ** 31 - 1])
def test_budgets_beyond_the_cache(V, budget):
    """A budget above every length, up to the largest int32: all tokens stay, in fresh pages."""
    c = R.make_case([300, 129], [0, 0], 1, seed=231, spare=6)
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(len(c.sk)) if p not in used]
    dst = torch.tensor([free[:3], free[3:6]], dtype=torch.int32)
    cols = -(-budget // 128)
    big = torch.full((2, cols), -1, dtype=torch.int32, device="cuda")
    big[:, :3] = dst.cuda()
    weight = torch.rand((*c.sk.shape, 128), generator=torch.Generator().manual_seed(232))
    cache, _ = c.on(V)
    got_w, got_kept = weight.cuda(), torch.full((2, 1, budget), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new_len, _ = V.cache_evict(cache, got_w, big, budget, 7, kept=got_kept, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0 and new_len.tolist() == [300, 129]
    kept = torch.full((2, 1, 400), -1, dtype=torch.int32)
    R.evict(c, weight, dst, 400, 7, kept)
    assert torch.equal(got_kept[..., :400].cpu(), kept) and not bool((got_kept[..., 400:] != -1).any())
    _same_codes(cache.k8, c.k8)
    _same_codes(cache.v8, c.v8)
    assert torch.equal(cache.sk.cpu(), c.sk) and torch.equal(got_w.cpu(), weight)


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("softcap", [0.0, 4.0])
@pytest.mark.parametrize("scale", [0.25, 0.011, 0.0, -3.0])
def test_scales_of_scores(V, name, softcap, scale):
    """softmax_scale as it is given; 1 / sqrt(128) where it is not above 0."""
    lens, news, Hq, H = ROWS[name]
    c = R.make_case(lens, news, H, seed=241)
    Q = R.rows(sum(news), Hq, seed=242, outliers=False)
    cache, start = c.on(V)
    out, lse = V.cache_attention(cache, Q.cuda(), start, softmax_scale=scale, softcap=softcap)
    used = scale if scale > 0 else 1.0 / math.sqrt(128.0)
    o, z, eo, el = R.attention(c, Q, softcap=softcap, scale=used)
    _within(out, o, eo, "O")
    _within(lse, z, el, "lse")
    weight = torch.zeros((*c.sk.shape, 128), device="cuda")
    V.cache_weigh(cache, Q.cuda(), start, lse, weight, softmax_scale=scale, softcap=softcap)
    w, e = R.weigh(c, Q, lse.cpu(), torch.zeros(weight.shape), softcap=softcap, scale=used)
    _within(weight, w, e, "weight")
