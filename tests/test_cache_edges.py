"""The 8-bit cache's checks and constants at the edges of what its documentation
allows, on a machine without a GPU."""
import pytest
import torch

import cache_reference as R
from test_cache_checks import FAKE, INVALID, OK, WORKSPACE, V, _attend, _struct  # noqa: F401  (V: fixture)


def test_scales_of_scores_beyond_fp32_are_refused(V):
    """softmax_scale too has to be an fp32 number after a factor of 4, with and without a cap."""
    s = _struct(V)
    assert _attend(V, s, scale=1e38) == INVALID and _attend(V, s, scale=1e38, cap=1e30) == INVALID
    assert _attend(V, s, scale=8e37, ws=None) == WORKSPACE and _attend(V, s, scale=1.0, cap=8e37, ws=None) == WORKSPACE


def test_weights_of_new_tokens_are_checked(V):
    s = _struct(V)

    def call(weight):
        return V._lib.vca_cache_append_ex(s, FAKE, 256, 128, FAKE, 256, 128, FAKE, 0, weight, None, None)

    assert call(None) == OK and call(FAKE) == OK and call(FAKE + 4) == INVALID
    c, K = V.alloc_cache(6, 2, 2, 3, device="cpu"), R.rows(4, 2, 1)
    start = torch.zeros(3, dtype=torch.int32)
    for bad in (torch.zeros(6, 2, 64), torch.zeros(5, 2, 128), torch.zeros(6, 2, 128).double()):
        with pytest.raises(ValueError, match="weight must be"):
            V.cache_append(c, K, K, start, weight=bad)
    with pytest.raises(ValueError, match="is not a CUDA tensor"):
        V.cache_append(c, K, K, start, weight=torch.zeros(6, 2, 128))


def test_ranks_are_named(V):
    """Tensors of another rank are named before anything is allocated from their shapes."""
    c, start = V.alloc_cache(6, 2, 2, 3, device="cpu"), torch.zeros(3, dtype=torch.int32)
    Q, lse, w = R.rows(4, 6, 2), torch.zeros(4, 6), torch.zeros(6, 2, 128)
    dst = torch.zeros((2, 2), dtype=torch.int32)

    def refuses(match, call):
        with pytest.raises(ValueError, match=match):
            call()

    for bad in (Q[0, 0], Q[0], Q[None], Q[0, 0, 0]):
        refuses("Q must be", lambda: V.cache_attention(c, bad, start))
        refuses("Q must be", lambda: V.cache_weigh(c, bad, start, lse, w))
        refuses("Q must be", lambda: V.cache_attention(c, bad, start, ws=w))
        refuses("Q must be", lambda: V.cache_weigh(c, bad, start, lse, w, ws=w))
        refuses("K must be", lambda: V.cache_append(c, bad, bad, start))
    refuses("weight must be", lambda: V.cache_weigh(c, Q, start, lse, w[0]))
    refuses("dst_table must be", lambda: V.cache_evict(c, w, dst[0], 200, 10))
    for name, what in (("k8", "k8 must be"), ("table", "table \\[B, cols\\]"), ("length", "length must be"), ("sk", "sk must be")):
        for shape in ((), (5,), (5, 1, 1, 1, 1)):
            if len(shape) == getattr(c, name).dim():
                continue
            d = V.Cache(*(torch.zeros(shape, dtype=getattr(c, f).dtype) if f == name else getattr(c, f)
                          for f in ("k8", "v8", "sk", "sv", "table", "length")))
            refuses(what, lambda: V.cache_attention(d, Q, start))
            refuses(what, lambda: V.cache_weigh(d, Q, start, lse, w))
            refuses(what, lambda: V.cache_append(d, R.rows(4, 2, 1), R.rows(4, 2, 1), start))
            refuses(what, lambda: V.cache_evict(d, w, dst, 200, 10))


def test_numbers_beyond_32_bits_are_refused(V):
    """The C interface's ints are 32 bits wide: a larger number must not be cut."""
    c, start = V.alloc_cache(6, 2, 2, 3, device="cpu"), torch.zeros(3, dtype=torch.int32)
    w, dst = torch.zeros(6, 2, 128), torch.zeros((2, 2), dtype=torch.int32)
    many = R.rows(1, 2, 1).expand(2 ** 32 + 1, 2, 128)
    lse = torch.zeros(1).expand(2 ** 32 + 1, 2)
    for call in (lambda: V.cache_append(c, many, many, start), lambda: V.vca_cache_append(c, many, many, start),
                 lambda: V.vca_cache_attention(c, many, start, 1, 0.0, 0.0, many, None, None),
                 lambda: V.cache_weigh(c, many, start, lse, w, ws=torch.zeros(16, dtype=torch.uint8)),
                 lambda: V.cache_weigh(c, many, start, lse, w)):
        with pytest.raises(ValueError, match="more than 2147483647 rows"):
            call()
    wide = R.rows(4, 1, 1).expand(4, 2 ** 32 + 2, 128)
    for call in (lambda: V.cache_attention(c, wide, start), lambda: V.cache_weigh(c, wide, start, lse[:4], w)):
        with pytest.raises(ValueError, match="rows or heads"):
            call()
    for sizes in ((2 ** 32 + 1, 4, 2, 1, 1), (1, 2 ** 32 + 2, 2, 1, 1), (1, 4, 2, 1, 2 ** 32 + 1)):
        assert V.vca_cache_workspace_bytes(V.VCA_OP_CACHE_ATTENTION, *sizes) == 0
    for budget, recent in ((200, 2 ** 32), (200, -2 ** 32 + 1), (2 ** 32 + 200, 10), (-2 ** 32 + 200, 10)):
        with pytest.raises(ValueError, match="32 bits"):
            V.cache_evict(c, w, dst, budget, recent)
        with pytest.raises(ValueError, match="32 bits"):
            V.vca_cache_evict(c, w, dst, budget, recent, c.length.clone(), torch.zeros((2, 2, 200), dtype=torch.int32))
