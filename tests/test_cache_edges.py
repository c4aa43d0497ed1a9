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
