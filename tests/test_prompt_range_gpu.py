"""Prompt attention at the ends of its values' range and of its layouts."""
import pytest
import torch

import prompt_reference as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("softcap", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("causal", [True, False])
def test_values_near_the_largest(V, causal, softcap):
    """Scores that rise by 7.2 in log2 units, less than what moves the reference maximum, with values of 2^126: the
    sums of magnitudes over a sequence stay below 2^128, and so do O and all sums on its way."""
    lens = [300, 140]
    T = sum(lens)
    Q = torch.zeros((T, 2, 128), dtype=torch.bfloat16, device="cuda")
    K = torch.zeros((T, 1, 128), dtype=torch.bfloat16, device="cuda")
    Val = R.rows(T, 1, 91, outliers=False)
    Q[..., 0] = 1.0
    K[128:300, :, 0] = 5.0
    K[300 + 128:, :, 0] = 5.0
    Val[130], Val[131], Val[300 + 129] = 2.0 ** 126, -(2.0 ** 126), 1.5 * 2.0 ** 126
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = V.prompt_attention(Q, K, Val, R.starts(lens), causal=causal, softmax_scale=1.0, softcap=softcap, dev_status=status)
    assert int(status) == 0
    o, z, eo, el = R.attention(Q, K, Val, lens, causal=causal, scale=1.0, softcap=softcap)
    assert bool(torch.isfinite(o.float()).all()) and float(o.abs().max()) > 2.0 ** 118
    R.within(out, o, eo, "O")
    R.within(lse, z, el, "lse")


@pytest.mark.parametrize("of", ["Q", "K", "V"])
def test_one_row_or_head_has_any_distance(V, of):
    """A dimension of one entry is never stepped over: its distance may be anything."""
    g = torch.Generator().manual_seed(92)
    for T, H, distances in ((1, 2, (3, 128, 1)), (1, 2, (0, 128, 1)), (5, 1, (128, 5, 1)), (5, 1, (128, 0, 1)), (1, 1, (1, 1, 1))):
        x = {n: torch.randn((T, H, 128), generator=g).bfloat16().cuda() for n in "QKV"}
        buf = torch.randn(2048, generator=g).bfloat16().cuda()
        view = buf.as_strided((T, H, 128), distances)
        x[of] = view.copy_(x[of])
        plain = {n: torch.empty((T, H, 128), dtype=torch.bfloat16, device="cuda").copy_(t) for n, t in x.items()}
        start = R.starts([T])
        got, want = V.prompt_attention(x["Q"], x["K"], x["V"], start), V.prompt_attention(plain["Q"], plain["K"], plain["V"], start)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
