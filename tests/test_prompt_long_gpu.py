"""Prompt attention of calls with a long average prompt, which have code of their own: several sequences, several
works a CTA, and all rows against the definition in 64 bits."""
import math

import pytest
import torch

import prompt_reference as R
from test_prompt_gpu import _check, _inputs

pytestmark = pytest.mark.gpu

BATCHES = {
    "two long": ([5000, 2300], 40, 8),
    "a short and a long": ([129, 9000], 20, 4),
    "a head each": ([4300, 1, 4000, 513], 12, 12),
    "two to a head": ([3329, 2561], 16, 8),
}


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", BATCHES)
def test_prompts(V, name, causal):
    lens, Hq, H = BATCHES[name]
    assert sum(lens) > 2048 * len(lens)
    _check(V, lens, *_inputs(lens, Hq, H, seed=100 + len(name)), causal=causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("name", ["two long", "a head each"])
def test_joined_with_a_prior(V, name, causal):
    lens, Hq, H = BATCHES[name]
    Q, K, Val, start = _inputs(lens, Hq, H, seed=110)
    T = sum(lens)
    o = R.rows(T, Hq, 111, outliers=False)
    z = torch.randn((T, Hq), generator=torch.Generator().manual_seed(112)).cuda() * 40.0
    z[::3] = -math.inf
    o[::3] = math.nan      # not read
    first = _check(V, lens, Q, K, Val, start, causal=causal, prior=(o, z))
    out, lse = o.clone(), z.clone()      # in place
    V.prompt_attention(Q, K, Val, start, causal=causal, prior=(out, lse), out=out, lse=lse)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_neighbours_of_nan_and_infinity(V, bad):
    lens = [2500, 4100, 3001, 2200]
    for causal in (True, False):
        Q, K, Val, start = _inputs(lens, 10, 2, seed=113)
        o, z, eo, el = R.attention(Q, K, Val, lens, causal=causal)
        for x in (Q, K, Val):
            x[:2500], x[6600:9601] = bad, bad
        out, lse = V.prompt_attention(Q, K, Val, start, causal=causal)
        for sl in (slice(2500, 6600), slice(9601, 11801)):
            R.within(out[sl], o[sl], eo[sl], "O")
            R.within(lse[sl], z[sl], el[sl], "lse")


def test_a_key_of_nan_reaches_only_the_rows_that_see_it(V):
    lens = [4500, 2300]
    Q, K, Val, start = _inputs(lens, 10, 2, seed=114)
    o, z, eo, el = R.attention(Q, K, Val, lens)
    K[1977, 0, 3] = math.nan
    Q[20, 6, 5] = math.nan
    out, lse = V.prompt_attention(Q, K, Val, start)
    bad = torch.zeros(Q.shape[:2], dtype=torch.bool, device="cuda")
    bad[1977:4500, :5] = True
    bad[20, 6] = True
    assert bool(torch.isnan(out[bad]).all()) and bool(torch.isnan(lse[bad]).all())
    R.within(out[~bad], o[~bad], eo[~bad], "O")
    R.within(lse[~bad], z[~bad], el[~bad], "lse")


def test_starts_that_fall_and_rows_behind(V):
    lens = [4700, 3300, 2500]
    n = 8000
    Q, K, Val, start = _inputs(lens, 10, 2, seed=115, extra=9)
    o, z, eo, el = R.attention(Q, K, Val, lens)
    for wrong in (None, -5, n - 4, sum(lens) + 10, 1 << 30):
        if wrong is not None:
            start[3] = wrong
        rows = sum(lens) if wrong is None else n
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full(Q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full(Q.shape[:2], 7.0, device="cuda")
        V.prompt_attention(Q, K, Val, start, out=out, lse=lse, dev_status=status)
        torch.cuda.synchronize()
        assert int(status) == (0 if wrong is None else V.VCA_ERR_INVALID_ARG)
        R.within(out[:rows], o[:rows], eo[:rows], "O")
        R.within(lse[:rows], z[:rows], el[:rows], "lse")
        assert bool((out[rows:] == 7).all()) and bool((lse[rows:] == 7).all())


def test_equal_bits_at_any_place(V):
    """Equal calls, O off 32 bytes, strided inputs and a replayed graph: the same bits."""
    lens = [5000, 129, 3300]
    Q, K, Val, start = _inputs(lens, 10, 2, seed=116)
    first = V.prompt_attention(Q, K, Val, start)
    buf = torch.zeros(Q.numel() + 8, dtype=torch.bfloat16, device="cuda")
    out = buf[8:].view(Q.shape)
    assert out.data_ptr() % 32 == 16
    fused = torch.cat([Q, K, Val], 1)
    views = fused[:, :10], fused[:, 10:12], fused[:, 12:]
    lse = torch.empty_like(first[1])
    V.prompt_attention(*views, start, out=out, lse=lse)
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1]) and not bool(buf[:8].any())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.prompt_attention(*views, start, out=out, lse=lse)
    for _ in range(20):
        again = V.prompt_attention(Q, K, Val, start)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        out.zero_()
        lse.zero_()
        graph.replay()
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
