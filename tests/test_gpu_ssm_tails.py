"""The scan's backward pass where the last tile of 8 tokens is not full, on the GPU: a last
state that is not finite belongs to no gradient of A."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("T", [1, 8, 13, 61, 1500])
def test_infinite_last_input(T, S, dtype):
    """x_T enters h_T, y_T and the gradients of delta_T, b_T, D_skip and gate_T; dA_log, dx, dc
    before T, db before T and dh0 are the same as with a finite x_T, bit for bit."""
    D = 24
    gen = torch.Generator().manual_seed(T + S)
    r = lambda *s: torch.randn(*s, generator=gen).to(dtype).cuda()  # noqa: E731
    f = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, dt, d_y, gate, b, c = r(2, T, D), r(2, T, D), r(2, T, D), r(2, T, D), r(2, T, 1, S), r(2, T, 1, S)
    A_log, h0, bias, skip = 0.3 * f(D, S), f(2, D, S), f(D) - 2, f(D)
    for d_last in (None, f(2, D, S)):
        run = lambda x: G.gdn_ssm_bwd(x, dt, A_log, b, c, d_y, h0, None, d_last, D_skip=skip,  # noqa: E731
                                      gate=gate, dt_bias=bias, dt_softplus=True, check=True)
        want = run(x)
        for bad in (float("inf"), float("nan")):
            y = x.clone()
            y[1, T - 1, 5] = bad
            got = run(y)
            for n in ("dA_log", "dx", "dh0"):
                assert torch.equal(got[n], want[n]), (n, bad)
            for n in ("db", "dc", "ddt", "dgate"):
                assert torch.equal(got[n][0], want[n][0]) and \
                    torch.equal(got[n][1, :T - 1], want[n][1, :T - 1]), (n, bad)
            assert not torch.isfinite(got["dD_skip"][5]) and not torch.isfinite(got["ddt"][1, T - 1, 5])
