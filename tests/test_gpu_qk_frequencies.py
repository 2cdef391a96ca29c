"""Frequencies of the q/k norm's rotation that are not finite, on the GPU: their pairs are not
a number, as in the formula, and the others what they are without them."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,R", [(64, 64), (64, 12), (128, 32)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_frequency_not_finite(bad, D, R, inter):
    gen = torch.Generator().manual_seed(D + R)
    r = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    q, k, dq, dk, w = r(2, 40, 3, D), r(2, 40, 1, D), r(2, 40, 3, D), r(2, 40, 1, D), r(D)
    freq = (10000.0 ** (-torch.arange(0, R, 2) / R)).cuda()
    i = 1
    wrong = freq.clone()
    wrong[i] = bad
    pair = [2 * i, 2 * i + 1] if inter else [i, i + R // 2]
    rest = [n for n in range(D) if n not in pair]
    run = lambda f: G.gdn_qk_norm(q, k, w, None, None, f, interleaved=inter)  # noqa: E731
    for got, want in zip(run(wrong), run(freq)):
        assert torch.isnan(got[..., pair]).all()
        assert torch.equal(got[..., rest], want[..., rest])
    back = lambda f: G.gdn_qk_norm_bwd(q, k, dq, dk, w, None, None, f, interleaved=inter)  # noqa: E731
    got, want = back(wrong), back(freq)
    assert torch.isnan(got["dq"]).all() and torch.isnan(got["dk"]).all()   # (through the norm)
    assert torch.isnan(got["dq_weight"][pair]).all()
    assert torch.equal(got["dq_weight"][rest], want["dq_weight"][rest])
