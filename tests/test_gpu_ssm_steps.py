"""The scan's step delta = softplus(v) and its derivative by themselves, on the GPU: after one
token from zero, x = b = 1, the state is delta, and with a gradient of 1 for one of its states
ddt_bias is softplus'(v).

Bounds, relative: with e = exp(-|v|), the hardware's exp2 is off by 2^-22, the fma that puts
its argument right (fp32 storage) by 2^-24 twice; 2 + e (or 1 + e) and its reciprocal by 2^-24
and 2^-23, their product by 2^-24; the polynomial and the last sum by 2^-24 each and 4e-9:
3 x 2^-22 together.  With bf16 storage the argument's rounding stays, |v| 2^-24 of e, and that
of log2(e), |v| 1.34e-8.  (delta and its derivative are no farther off than e.)"""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_step_and_its_derivative(S, dtype):
    D = 4096
    v = torch.cat([torch.linspace(-80, -5, D // 2, dtype=torch.float64),
                   torch.linspace(-5, 80, D // 2, dtype=torch.float64)]).float().cuda()
    zero = torch.zeros(1, 1, D, dtype=dtype, device="cuda")
    one, b = zero + 1, torch.ones(1, 1, 1, S, dtype=dtype, device="cuda")
    A_log = torch.zeros(D, S, device="cuda")
    w = v.double()
    delta = w.clamp(min=0) + torch.log1p(torch.exp(-w.abs()))
    slope = torch.where(w < 0, torch.exp(-w.abs()), 1.0) / (1 + torch.exp(-w.abs()))
    bound = 3 * 2.0 ** -22 + (0 if dtype == torch.float32 else w.abs() * (2.0 ** -24 + 1.34e-8))
    how = dict(dt_bias=v, dt_softplus=True, check=True)
    _, h = G.gdn_ssm_fwd(one, zero, A_log, b, b, **how)
    for n in range(S):
        assert ((h[0, :, n].double() - delta).abs() <= bound * delta).all()
    _, out = G.gdn_ssm_step(one[0], zero[0], A_log, b[0], b[0], None, state_out=torch.empty_like(h), **how)
    assert ((out[0, :, 0].double() - delta).abs() <= bound * delta).all()
    d_last = torch.zeros(1, D, S, device="cuda")
    d_last[..., S - 1] = 1
    g = G.gdn_ssm_bwd(one, zero, A_log, b, b, zero, None, None, d_last, **how)
    assert ((g["ddt_bias"].double() - slope).abs() <= bound * slope).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_limits(dtype):
    """Steps and derivatives of infinities and of logits whose exponential is zero."""
    D = 8
    v = torch.tensor([float("inf"), -float("inf"), 200.0, -200.0, 0.0, 100.0, -110.0, float("nan")]).cuda()
    zero = torch.zeros(1, 1, D, dtype=dtype, device="cuda")
    b = torch.ones(1, 1, 1, 8, dtype=dtype, device="cuda")
    A_log = torch.zeros(D, 8, device="cuda")
    how = dict(dt_bias=v, dt_softplus=True)
    _, h = G.gdn_ssm_fwd(zero + 1, zero, A_log, b, b, **how)
    d = h[0, :, 0].tolist()
    assert d[0] == float("inf") and d[1] == d[3] == d[6] == 0 and d[2] == 200 and d[5] == 100
    assert abs(d[4] - 0.6931471805599453) < 2.0 ** -21 and d[7] != d[7]
    d_last = torch.ones(1, D, 8, device="cuda") / 8
    g = G.gdn_ssm_bwd(zero + 1, zero, A_log, b, b, zero, None, None, d_last, **how)["ddt_bias"].tolist()
    assert g[1] == g[3] == g[6] == 0 and g[2] == g[5] == 1 and abs(g[4] - 0.5) < 2.0 ** -22 and g[7] != g[7]
