"""Prompt attention's bounded waits: those that are as long as whole works, and those that run out."""
import math

import pytest
import torch

import prompt_reference as R

pytestmark = pytest.mark.gpu


def _call(V, lens, limit_ns, causal, seed, softcap=0.0):
    T = sum(lens)
    Q, K, Val = R.rows(T, 1, seed), R.rows(T, 1, seed + 1), R.rows(T, 1, seed + 2, outliers=False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = R.starts(lens)
    torch.cuda.synchronize()
    V.vca_set_wait_limit_ns(limit_ns)
    try:
        out, lse = V.prompt_attention(Q, K, Val, start, causal=causal, softcap=softcap, dev_status=status)
        torch.cuda.synchronize()
    finally:
        V.vca_set_wait_limit_ns(2_000_000_000)
    return Q, K, Val, out, lse, int(status)


def _some_rows(lens, causal, Q, K, Val, out, lse):
    lo = 0
    for n in lens:
        at = torch.tensor(sorted({0, 1, n // 2, max(0, n - 130), n - 1}), device="cuda")
        q, k, v = Q[lo + at, 0].double(), K[lo:lo + n, 0].double(), Val[lo:lo + n, 0].double()
        s, mag = q @ k.T / math.sqrt(128), q.abs() @ k.abs().T / math.sqrt(128)
        if causal:
            hide = torch.arange(n, device="cuda") > at[:, None]
            s, mag = s.masked_fill(hide, -math.inf), mag.masked_fill(hide, 0.0)
        # the bounds of prompt_reference.attention
        es, z, p = 2.0 ** -16 * mag.amax(-1) + 2.0 ** -20, torch.logsumexp(s, -1), torch.softmax(s, -1)
        R.within(lse[lo + at, 0], z, es + 2.0 ** -22 * z.abs() + 2.0 ** -20 + 2.0 ** -23 * n, "lse")
        o = p @ v
        R.within(out[lo + at, 0], o, (2.0 ** -8 + 2 * es + 2.0 ** -23 * n)[:, None] * (p @ v.abs()) + 2.0 ** -8 * o.abs(), "O")
        lo += n


@pytest.mark.parametrize("lens,causal", [([100097], True), ([100097, 100097], False)])
def test_a_tile_without_rows_waits_for_whole_works(V, lens, causal):
    """391 pairs of tiles and one tile alone, of 782 blocks.  The CTA that has it takes a pair next, whose second tile waits for
    all of the lone tile's blocks: longer than the limit of a block."""
    *tensors, status = _call(V, lens, 400_000, causal, 81)
    assert status == 0
    _some_rows(lens, causal, *tensors)


def test_waits_that_cannot_but_run_out(V):
    """Works of 782 blocks and the smallest limit there is, 1 us a block.  The softmax of a small cap has three operations of
    the special function unit a score, 32 a cycle at most: 1.48 us a block of both tiles (256 x 128 scores) at 2,070 MHz.
    So the epilogue's wait for a work, 0.784 ms of 1.16, runs out, and the call says so; the next one is right."""
    lens = [100001, 70]
    for _ in range(2):
        assert _call(V, lens, 1000, False, 84, softcap=64.0)[-1] == V.VCA_ERR_TIMEOUT
        *tensors, status = _call(V, lens, 2_000_000_000, False, 84)
        assert status == 0
        _some_rows(lens, False, *tensors)
