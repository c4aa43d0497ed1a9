"""Refusals of prompt attention and of the cache's planning on a machine without a GPU:
the C entries' status codes before any CUDA call, and the binding's checks of tensors."""
import pytest
import torch

import prompt_reference as R


@pytest.fixture(scope="module")
def V():
    from bit_attention_video_smooth_gb300 import build
    build.build()
    from bit_attention_video_smooth_gb300 import vca
    return vca


FAKE = 0x10000     # aligned, never dereferenced
OK, INVALID = 0, 1


def _attend(V, Q=FAKE, qt=512, qh=128, K=FAKE, kt=256, kh=128, Val=FAKE, vt=256, vh=128, start=FAKE, B=2, T=3, Hq=4, H=2, d=128,
            causal=1, scale=0.0, cap=0.0, prior=None, prior_lse=None, O=FAKE, lse=None, status=None):
    return V._lib.vca_prompt_attention(Q, qt, qh, K, kt, kh, Val, vt, vh, start, B, T, Hq, H, d, causal, scale, cap, prior, prior_lse,
                                       O, lse, status, None)


def _plan(V, table=FAKE, length=2 * FAKE, pages=10, B=2, cols=4, held=3 * FAKE, news=4 * FAKE, start=5 * FAKE, slot=None,
          position=None, T=3, status=None):
    return V._lib.vca_cache_plan(table, length, pages, B, cols, held, news, start, slot, position, T, status, None)


def _fresh(V, table=FAKE, length=2 * FAKE, pages=10, B=2, cols=4, budget=200, dst=3 * FAKE, dst_cols=2, status=None):
    return V._lib.vca_cache_fresh(table, length, pages, B, cols, budget, dst, dst_cols, status, None)


@pytest.mark.parametrize("bad", [
    dict(Q=None), dict(Q=FAKE + 8), dict(qt=250), dict(qh=4), dict(qt=0), dict(qh=0), dict(qt=-512), dict(qh=-128), dict(K=None),
    dict(K=FAKE + 2), dict(kt=100), dict(kh=1), dict(kt=0), dict(kt=-256), dict(kh=-128), dict(kt=1 << 39), dict(kh=1 << 39),
    dict(Val=None), dict(Val=FAKE + 4), dict(vt=0), dict(vh=-8), dict(vt=1 << 40), dict(start=None), dict(start=FAKE + 2), dict(B=0),
    dict(B=40000), dict(T=-1), dict(Hq=3), dict(Hq=0), dict(H=0), dict(T=1 << 30), dict(d=64), dict(causal=2), dict(causal=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e38), dict(cap=-1.0), dict(cap=float("nan")), dict(cap=3e38),
    dict(scale=1e30, cap=1e-10), dict(prior=FAKE), dict(prior_lse=FAKE), dict(prior=FAKE + 8, prior_lse=FAKE),
    dict(prior=FAKE, prior_lse=FAKE + 1), dict(O=None), dict(O=FAKE + 8), dict(lse=FAKE + 2), dict(status=FAKE + 1)])
def test_prompt_arguments(V, bad):
    assert _attend(V, **bad) == INVALID


def test_no_rows_launch_nothing(V):
    assert _attend(V, T=0, Q=None, K=None, Val=None, O=None) == OK


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(table=FAKE + 2), dict(length=None), dict(length=2 * FAKE + 1), dict(pages=0), dict(pages=1 << 24), dict(B=0),
    dict(B=65536), dict(cols=0), dict(cols=1 << 24), dict(held=None), dict(news=None), dict(start=None), dict(start=FAKE + 3),
    dict(slot=FAKE + 2), dict(position=FAKE + 1), dict(T=-1), dict(status=FAKE + 2), dict(news=2 * FAKE), dict(start=2 * FAKE),
    dict(start=3 * FAKE), dict(start=4 * FAKE)])
def test_plan_arguments(V, bad):
    assert _plan(V, **bad) == INVALID


@pytest.mark.parametrize("bad", [
    dict(table=None), dict(length=None), dict(pages=0), dict(pages=1 << 24), dict(B=0), dict(B=65536), dict(cols=0), dict(budget=0),
    dict(budget=-3), dict(dst=None), dict(dst=FAKE + 2), dict(dst_cols=0), dict(dst_cols=1), dict(dst=FAKE), dict(dst=2 * FAKE),
    dict(status=FAKE + 2)])
def test_fresh_arguments(V, bad):
    assert _fresh(V, **bad) == INVALID


def test_the_status_of_a_full_pool_has_a_name(V):
    assert V.vca_status_string(V.VCA_ERR_FULL) == "too few free pages"


def _ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_right_tensors_fail_only_on_the_device(V):
    Q, K, start = R.rows(5, 6, 1, "cpu"), R.rows(5, 2, 2, "cpu"), _ints(3)
    cache = V.alloc_cache(6, 2, 2, 3, device="cpu")
    for call in (lambda: V.prompt_attention(Q, K, K, start), lambda: V.prompt_attention(Q, K, K, start, prior=(Q, torch.zeros(5, 6))),
                 lambda: V.cache_plan(cache, _ints(2), 4), lambda: V.cache_fresh(cache, 200)):
        with pytest.raises(ValueError, match="is not a CUDA tensor"):
            call()


def test_wrong_tensors_are_named(V):
    Q, K, start = R.rows(5, 6, 1, "cpu"), R.rows(5, 2, 2, "cpu"), _ints(3)
    cache = V.alloc_cache(6, 2, 2, 3, device="cpu")

    def refuses(match, call):
        with pytest.raises(ValueError, match=match):
            call()

    refuses("Q must be", lambda: V.prompt_attention(Q.half(), K, K, start))
    refuses("Q must be", lambda: V.prompt_attention(Q[0], K, K, start, out=Q, lse=torch.zeros(5, 6)))
    refuses("K must be", lambda: V.prompt_attention(Q, K.float(), K, start))
    refuses("K has 4 rows", lambda: V.prompt_attention(Q, K[:4], K, start))
    refuses("V must be", lambda: V.prompt_attention(Q, K, R.rows(5, 3, 1, "cpu"), start))
    refuses("channels of V", lambda: V.prompt_attention(Q, K, K.transpose(1, 2).contiguous().transpose(1, 2), start))
    refuses("start must be", lambda: V.prompt_attention(Q, K, K, start.long()))
    refuses("O must be", lambda: V.prompt_attention(Q, K, K, start, out=K))
    refuses("lse must be", lambda: V.prompt_attention(Q, K, K, start, lse=torch.zeros(5, 2)))
    refuses("prior must be", lambda: V.prompt_attention(Q, K, K, start, prior=(Q.float(), torch.zeros(5, 6))))
    refuses("prior_lse must be", lambda: V.prompt_attention(Q, K, K, start, prior=(Q, torch.zeros(5, 5))))
    refuses("together", lambda: V.vca_prompt_attention(Q, K, K, start, 1, 0.0, 0.0, Q, None, Q, None))
    refuses("news must be", lambda: V.cache_plan(cache, _ints(3), 4))
    refuses("news must be", lambda: V.cache_plan(cache, _ints(2).long(), 4))
    refuses("held must be", lambda: V.cache_plan(cache, _ints(2), 4, held=_ints(1)))
    refuses("start must be", lambda: V.cache_plan(cache, _ints(2), 4, start=_ints(2)))
    refuses("slot must be", lambda: V.cache_plan(cache, _ints(2), 4, slot=_ints(5)))
    refuses("position must be", lambda: V.cache_plan(cache, _ints(2), 4, position=torch.zeros(4)))
    refuses("T = -1", lambda: V.cache_plan(cache, _ints(2), -1))
    refuses("T = ", lambda: V.cache_plan(cache, _ints(2), 1 << 31))
    refuses("dst_table must be", lambda: V.cache_fresh(cache, 200, out=_ints(3, 2)))
    refuses("dst_table must be", lambda: V.cache_fresh(cache, 200, out=_ints(4)))
    refuses("budget", lambda: V.cache_fresh(cache, 0))
    refuses("budget", lambda: V.cache_fresh(cache, 1 << 31))
    bad = V.Cache(cache.k8, cache.v8, cache.sk, cache.sv, cache.table.t().contiguous().t(), cache.length)
    refuses("table must be contiguous", lambda: V.cache_plan(bad, _ints(2), 4))
    bad = V.Cache(cache.k8, cache.v8, cache.sk, cache.sv, cache.table[0], cache.length)
    refuses("table", lambda: V.cache_plan(bad, _ints(2), 4))
    refuses("table", lambda: V.cache_fresh(bad, 200))


def test_reference_attention_is_a_softmax():
    lens = [70, 1, 30]
    Q, K, Val = R.rows(101, 4, 1, "cpu"), R.rows(101, 2, 2, "cpu"), R.rows(101, 2, 3, "cpu")
    o, lse, eo, _ = R.attention(Q, K, Val, lens)
    q, k, v = (x[:70].double().transpose(0, 1) for x in (Q, K.repeat_interleave(2, 1), Val.repeat_interleave(2, 1)))
    ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, is_causal=True)
    assert torch.allclose(o[:70].transpose(0, 1), ref, rtol=1e-10, atol=1e-10) and bool((eo >= 0).all())
    # joined with a prior over half of the keys: the whole
    first = R.attention(Q[:40], K[:40], Val[:40], [40], causal=False)
    k2, v2 = torch.cat([K[:40], K[40:80]]), torch.cat([Val[:40], Val[40:80]])
    s = Q[:40, 0].double() @ k2[:, 0].double().T / 128 ** 0.5
    both = R.attention(Q[:40], K[40:80], Val[40:80], [40], causal=False, prior=(first[0], first[1]))
    assert torch.allclose(both[1][:, 0], torch.logsumexp(s, -1), rtol=1e-10) and \
        torch.allclose(both[0][:, 0], torch.softmax(s, -1) @ v2[:, 0].double(), rtol=1e-9, atol=1e-9)


def test_reference_plan():
    table, length, start, slot, position, code = R.plan([[3, -1], [1, -1]], [128, 5], [2, 1], 5, 3)
    assert (table, length, start, code) == ([[3, 0], [1, -1]], [130, 6], [0, 2, 3], 0)
    assert slot == [0, 1, 128 + 5] and position == [128, 129, 5]
    assert R.plan([[3, -1]], [128], [1], 4, 1)[5] == 0 and R.plan([[0, -1]], [128], [1], 1, 1)[5] == 6
    assert R.plan([[0, -1]], [128], [200], 9, 200)[5] == 1
