"""The 8-bit cache's checks and constants at the edges of what its documentation
allows, on a machine without a GPU."""
from test_cache_checks import INVALID, WORKSPACE, V, _attend, _struct  # noqa: F401  (V: fixture)


def test_scales_of_scores_beyond_fp32_are_refused(V):
    """softmax_scale too has to be an fp32 number after a factor of 4, with and without a cap."""
    s = _struct(V)
    assert _attend(V, s, scale=1e38) == INVALID and _attend(V, s, scale=1e38, cap=1e30) == INVALID
    assert _attend(V, s, scale=8e37, ws=None) == WORKSPACE and _attend(V, s, scale=1.0, cap=8e37, ws=None) == WORKSPACE
