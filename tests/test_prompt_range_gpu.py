"""Prompt attention at the ends of its values' range and of its layouts."""
import pytest
import torch

import prompt_reference as R

pytestmark = pytest.mark.gpu


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
