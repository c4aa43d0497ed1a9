"""The 8-bit cache's refusals on a machine without a GPU: the C entries' status
codes before any CUDA call, and the binding's checks of tensors."""
import ctypes

import pytest
import torch

import cache_reference as R


@pytest.fixture(scope="module")
def V():
    from bit_attention_video_smooth_gb300 import build
    build.build()
    from bit_attention_video_smooth_gb300 import vca
    return vca


FAKE = 0x10000     # aligned, never dereferenced
OK, INVALID, WORKSPACE = 0, 1, 5


def _struct(V, **kw):
    f = dict(k8=FAKE, v8=FAKE, sk=FAKE, sv=FAKE, table=FAKE, len=FAKE, pages=10, H=2, d=128, B=3, cols=4)
    f.update(kw)
    return V._CacheStruct(**f)


def _append(V, s, K=FAKE, kt=256, kh=128, start=FAKE, T=3, status=None):
    return V._lib.vca_cache_append(s, K, kt, kh, FAKE, 256, 128, start, T, status, None)


def _attend(V, s, Q=FAKE, qt=512, qh=128, start=FAKE, T=3, Hq=4, causal=1, scale=0.0, cap=0.0, O=FAKE, lse=None, ws=FAKE,
            ws_bytes=1 << 40, status=None):
    return V._lib.vca_cache_attention(s, Q, qt, qh, start, T, Hq, causal, scale, cap, O, lse, ws, ws_bytes, status, None)


def _weigh(V, s, Q=FAKE, T=3, Hq=4, causal=1, cap=0.0, lse=FAKE, weight=FAKE):
    return V._lib.vca_cache_weigh(s, Q, 512, 128, FAKE, T, Hq, causal, 0.0, cap, lse, weight, FAKE, 1 << 40, None, None)


def _evict(V, s, weight=FAKE, dst=2 * FAKE, dst_cols=2, budget=200, recent=10, new_len=3 * FAKE, kept=FAKE):
    return V._lib.vca_cache_evict(s, weight, dst, dst_cols, budget, recent, new_len, kept, None, None)


@pytest.mark.parametrize("bad", [dict(k8=None), dict(v8=None), dict(sk=None), dict(sv=None), dict(table=None),
                                 dict(len=None), dict(k8=FAKE + 8), dict(v8=FAKE + 4), dict(sk=FAKE + 2), dict(len=FAKE + 1),
                                 dict(d=64), dict(pages=0), dict(H=0), dict(B=0), dict(cols=0), dict(B=40000, H=2),
                                 dict(pages=1 << 24, H=1), dict(cols=1 << 24)])
def test_a_bad_cache_is_refused_by_every_entry(V, bad):
    s = _struct(V, **bad)
    for call in (_append, _attend, _weigh, _evict):
        assert call(V, s) == INVALID


def test_bad_arguments(V):
    s = _struct(V)
    assert V._lib.vca_cache_append(None, FAKE, 256, 128, FAKE, 256, 128, FAKE, 3, None, None) == INVALID
    for kw in (dict(K=None), dict(K=FAKE + 8), dict(kt=250), dict(kh=4), dict(start=None), dict(T=-1), dict(status=FAKE + 2)):
        assert _append(V, s, **kw) == INVALID, kw
    for kw in (dict(Q=None), dict(Q=FAKE + 2), dict(qt=100), dict(qh=1), dict(start=None), dict(T=-1), dict(Hq=3), dict(Hq=0),
               dict(causal=2), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
               dict(O=None), dict(O=FAKE + 4), dict(lse=FAKE + 2), dict(T=1 << 30, Hq=4), dict(status=FAKE + 1)):
        assert _attend(V, s, **kw) == INVALID, kw
    need = V.vca_cache_workspace_bytes(V.VCA_OP_CACHE_ATTENTION, 3, 4, 2, 3, 4)
    assert need > 0
    for kw in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=FAKE + 8)):
        assert _attend(V, s, **kw) == WORKSPACE, kw
    for kw in (dict(Q=None), dict(Hq=5), dict(causal=-1), dict(cap=-0.5), dict(lse=None), dict(lse=FAKE + 2), dict(weight=None),
               dict(weight=FAKE + 4), dict(T=-2)):
        assert _weigh(V, s, **kw) == INVALID, kw
    for kw in (dict(weight=None), dict(dst=None), dict(dst_cols=1), dict(dst_cols=0), dict(budget=0), dict(recent=-1),
               dict(recent=201), dict(new_len=None), dict(kept=None), dict(kept=FAKE + 2)):
        assert _evict(V, s, **kw) == INVALID, kw


def test_no_rows_launch_nothing(V):
    s = _struct(V)
    assert _append(V, s, T=0, K=None) == OK
    assert _attend(V, s, T=0, Q=None, O=None, ws=None) == OK
    assert _weigh(V, s, T=0, Q=None, lse=None, weight=None) == OK


def test_workspace_sizes(V):
    ws = V.vca_cache_workspace_bytes
    assert ws(V.VCA_OP_CACHE_ATTENTION, 1, 1, 1, 1, 1) > 0
    # bounded however long the sequences are: it holds shares of tiles, not scores
    assert ws(V.VCA_OP_CACHE_ATTENTION, 64, 40, 8, 64, 1 << 20) < 1 << 30
    for bad in ((0, 4, 2, 1, 1), (1, 3, 2, 1, 1), (1, 4, 2, 0, 1), (1, 4, 2, 1, 0), (1, 0, 1, 1, 1)):
        assert ws(V.VCA_OP_CACHE_ATTENTION, *bad) == 0
    assert ws(V.VCA_OP_GROUP, 1, 4, 2, 1, 1) == 0


def _host_cache(V, pages=6, H=2, B=2, cols=3):
    return V.alloc_cache(pages, H, B, cols, device="cpu")


def test_right_tensors_fail_only_on_the_device(V):
    c = _host_cache(V)
    start = torch.zeros(3, dtype=torch.int32)
    K, Q = R.rows(4, 2, 1), R.rows(4, 6, 2, strided=True)
    lse, w = torch.zeros(4, 6), torch.zeros(6, 2, 128)
    dst = torch.zeros((2, 2), dtype=torch.int32)
    for call in (lambda: V.cache_append(c, K, K, start), lambda: V.cache_attention(c, Q, start),
                 lambda: V.cache_weigh(c, Q, start, lse, w), lambda: V.cache_evict(c, w, dst, 200, 10)):
        with pytest.raises(ValueError, match="is not a CUDA tensor"):
            call()


def test_wrong_tensors_are_named(V):
    c = _host_cache(V)
    start = torch.zeros(3, dtype=torch.int32)
    K, Q = R.rows(4, 2, 1), R.rows(4, 6, 2)

    def refuses(match, call):
        with pytest.raises(ValueError, match=match):
            call()

    refuses("K must be", lambda: V.cache_append(c, K.float(), K, start))
    refuses("V must be", lambda: V.cache_append(c, K, R.rows(4, 3, 1), start))
    refuses("V has 3 rows", lambda: V.cache_append(c, K, K[:3], start))
    refuses("channels of K", lambda: V.cache_append(c, K.transpose(1, 2).contiguous().transpose(1, 2), K, start))
    refuses("start must be", lambda: V.cache_append(c, K, K, start[:2]))
    refuses("start must be", lambda: V.cache_append(c, K, K, start.long()))
    refuses("Q must be", lambda: V.cache_attention(c, Q.half(), start))
    refuses("O must be", lambda: V.cache_attention(c, Q, start, out=torch.zeros(4, 6, 64, dtype=torch.bfloat16)))
    refuses("lse must be", lambda: V.cache_attention(c, Q, start, lse=torch.zeros(4, 5)))
    refuses("lse must be", lambda: V.cache_weigh(c, Q, start, torch.zeros(3, 6), torch.zeros(6, 2, 128)))
    refuses("weight must be", lambda: V.cache_weigh(c, Q, start, torch.zeros(4, 6), torch.zeros(6, 2, 64)))
    refuses("weight must be", lambda: V.cache_evict(c, torch.zeros(5, 2, 128), torch.zeros((2, 2), dtype=torch.int32), 200, 1))
    refuses("dst_table must be", lambda: V.cache_evict(c, torch.zeros(6, 2, 128), torch.zeros((3, 2), dtype=torch.int32), 200, 1))
    refuses("kept must be", lambda: V.cache_evict(c, torch.zeros(6, 2, 128), torch.zeros((2, 2), dtype=torch.int32), 200, 1,
                                                  kept=torch.zeros((2, 2, 100), dtype=torch.int32)))
    bad = V.Cache(c.k8, c.v8[:5], c.sk, c.sv, c.table, c.length)
    refuses("v8 must be", lambda: V.cache_append(bad, K, K, start))
    bad = V.Cache(c.k8, c.v8, c.sk.double(), c.sv, c.table, c.length)
    refuses("sk must be", lambda: V.cache_append(bad, K, K, start))
    bad = V.Cache(c.k8, c.v8, c.sk, c.sv, c.table.t().contiguous().t(), c.length)
    refuses("table must be contiguous", lambda: V.cache_append(bad, K, K, start))


def test_scales_of_the_reference():
    """The page scale the reference uses: smallest power of two that holds the largest value within 448."""
    assert R.scale_for(448.0) == 1.0 and R.scale_for(449.0) == 2.0 and R.scale_for(0.0) == 2.0 ** -120
    assert R.scale_for(224.0) == 0.5 and R.scale_for(1.75) == 2.0 ** -8


def test_reference_attention_is_a_softmax():
    c = R.make_case([70, 200], [70, 3], 2, seed=1)
    Q = R.rows(73, 4, 2)
    o, lse, eo, _ = R.attention(c, Q)
    k = torch.stack([R.seq_values(c, 0, h // 2, c.k8, c.sk) for h in range(4)])
    v = torch.stack([R.seq_values(c, 0, h // 2, c.v8, c.sv) for h in range(4)])
    ref = torch.nn.functional.scaled_dot_product_attention(Q[:70].double().transpose(0, 1), k, v, is_causal=True)
    assert torch.allclose(o[:70].transpose(0, 1), ref, rtol=1e-10, atol=1e-10) and bool((eo >= 0).all())


def test_caps_beyond_fp32_are_refused(V):
    """softcap and softmax_scale / softcap have to be fp32 numbers after a factor of 4."""
    s = _struct(V)
    for cap in (1e-40, 3e38):
        assert _attend(V, s, cap=cap) == INVALID and _weigh(V, s, cap=cap) == INVALID
    assert _attend(V, s, scale=1e30, cap=1e-10) == INVALID
    # in range: on to the next check
    assert _attend(V, s, cap=1e-30, ws=None) == WORKSPACE and _attend(V, s, cap=1e30, ws=None) == WORKSPACE


def test_a_pool_of_another_rank_is_named(V):
    c = _host_cache(V)
    flat = V.Cache(c.k8.view(6, -1), c.v8, c.sk, c.sv, c.table, c.length)
    start = torch.zeros(3, dtype=torch.int32)
    K, Q = R.rows(4, 2, 1), R.rows(4, 6, 2)
    w, dst = torch.zeros(6, 2, 128), torch.zeros((2, 2), dtype=torch.int32)
    kept = torch.zeros((2, 2, 200), dtype=torch.int32)
    for call in (lambda: V.vca_cache_append(flat, K, K, start),
                 lambda: V.vca_cache_attention(flat, Q, start, 1, 0.0, 0.0, Q, None, None),
                 lambda: V.vca_cache_weigh(flat, Q, start, 1, 0.0, 0.0, torch.zeros(4, 6), w, None),
                 lambda: V.vca_cache_evict(flat, w, dst, 200, 10, torch.zeros(2, dtype=torch.int32), kept)):
        with pytest.raises(ValueError, match="k8 must be"):
            call()


def test_an_eviction_in_place_is_refused(V):
    s = _struct(V)
    assert _evict(V, s, new_len=FAKE) == INVALID and _evict(V, s, dst=FAKE) == INVALID
