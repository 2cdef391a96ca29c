"""GPU parity of the group norm with an activation (gdn_group_norm and its
backward) against the 64-bit definition.

Bounds, relative L2 (derived).  fp32: the statistics are sums joined pairwise
(about 2^-24 times the square root of a thread's own terms, a few hundred) and
a value takes some ten roundings of 2^-24 after them, gradients about twice
that: 5e-6.  The channels' sums dweight and dbias cancel: 2e-5.  bf16 outputs
add one rounding to 8 bits, 1.6e-3 in root mean square: 2.5e-3 with room for
small samples."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin
from parity import rel

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
TOL = {"fp32": 5e-6, "bf16": 2.5e-3}


def f64(t):
    return t.double().cpu().numpy()


def make(N, S, C, dtype, gate, seed=0, shift=0.5, affine=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x = (r(N, S, C) * (0.5 + r(C).abs()) + shift * r(C)).to(DT[dtype])
    d = dict(x=x, w=1 + 0.2 * r(C) if affine else None, b=0.2 * r(C) if affine else None,
             gate=r(N, S, C).to(DT[dtype]) if gate else None, dy=r(N, S, C).to(DT[dtype]))
    return {n: t if t is None else t.cuda() for n, t in d.items()}


def check(d, groups, dtype, silu, stat=2e-6):
    y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], groups, gate=d["gate"], silu=silu)
    y_ref, m_ref, r_ref = lin.group_norm(d["x"], d["w"], d["b"], groups, d["gate"], silu)
    assert y.dtype == d["x"].dtype and rel(f64(y), y_ref) <= TOL[dtype]
    assert rel(f64(rstd), r_ref) <= stat
    # a mean may be near zero: its error is measured in standard deviations
    assert np.abs((f64(mean) - m_ref) * r_ref).max() <= 2e-6 * max(1.0, np.abs(m_ref * r_ref).max())
    g = G.gdn_group_norm_bwd(d["x"], d["w"], d["b"], groups, mean, rstd, d["dy"], gate=d["gate"],
                             silu=silu)
    ref = lin.group_norm_bwd(d["x"], d["w"], d["b"], groups, d["dy"], d["gate"], silu)
    assert rel(f64(g["dx"]), ref["dx"]) <= TOL[dtype]
    if d["gate"] is None:
        assert g["dgate"] is None
    else:
        assert rel(f64(g["dgate"]), ref["dgate"]) <= TOL[dtype]
    assert rel(f64(g["dweight"]), ref["dweight"]) <= 2e-5
    assert rel(f64(g["dbias"]), ref["dbias"]) <= 2e-5
    return y, g


MODES = [(False, False), (True, False), (False, True), (True, True)]


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("silu,gate", MODES)
@pytest.mark.parametrize("N,S,C,groups", [
    (300, 1, 1024, 16), (37, 1, 128, 1), (5, 1, 96, 3), (70, 1, 30, 3), (3, 7, 40, 4),
    (2, 300, 320, 32), (1, 1000, 64, 8), (2, 65, 6, 6), (4, 50, 512, 1), (1, 2500, 1280, 40)])
def test_shapes(dtype, silu, gate, N, S, C, groups):
    check(make(N, S, C, dtype, gate, seed=N + C), groups, dtype, silu)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,S,C,groups", [(40, 1, 2048, 1), (3, 1, 8192, 8), (2, 3, 8190, 2),
                                          (1, 2, 8192, 8192), (1, 9000, 16, 1), (2500, 1, 64, 2),
                                          (3, 4096, 8, 2), (7, 16, 3, 1)])
def test_wide_narrow_long(dtype, N, S, C, groups):
    d = make(N, S, C, dtype, True, seed=C)
    if S * C // groups == 1 or C == groups and S < 4:
        # groups of one or two values: every deviation is rounding or as large
        # as the spread; only finite results are asked for
        y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], groups, gate=d["gate"])
        assert torch.isfinite(y).all() and torch.isfinite(rstd).all()
        return
    check(d, groups, dtype, True)


@pytest.mark.parametrize("N,S", [(64, 1), (2, 400)])
def test_a_mean_far_from_zero(N, S):
    """x = 1000 + noise in fp32: what 24 bits leave of the deviations (2^-14 of
    them) is all in x itself, which the definition reads too; the mean of some
    thousand values is rounded once to 24 bits, which shifts every deviation by
    up to 2^-15, squared in the variance."""
    g = torch.Generator().manual_seed(4)
    d = make(N, S, 256, "fp32", False)
    d["x"] = (1000 + torch.randn(N, S, 256, generator=g)).cuda()
    y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], 4)
    y_ref, m_ref, r_ref = lin.group_norm(d["x"], d["w"], d["b"], 4)
    assert np.abs(f64(mean) - m_ref).max() <= 2 ** -14
    assert rel(f64(rstd), r_ref) <= 1e-5
    assert rel(f64(y), y_ref) <= 1e-4


def test_constant_input_has_no_spread():
    d = make(3, 4, 64, "fp32", False, affine=False)
    d["x"].fill_(3.0)
    y, mean, rstd = G.gdn_group_norm(d["x"], None, None, 4)
    assert (y == 0).all() and (mean == 3).all()
    assert np.allclose(f64(rstd), 1 / np.sqrt(1e-5), rtol=1e-6)


def test_without_weight_and_bias_and_large_values():
    check(make(9, 5, 96, "fp32", True, affine=False), 3, "fp32", True)
    d = make(2, 3, 64, "fp32", True)
    d["gate"].fill_(-200.0)        # exp(200) overflows: silu is -0
    y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], 4, gate=d["gate"], silu=True)
    assert (y == 0).all()
    g = G.gdn_group_norm_bwd(d["x"], d["w"], d["b"], 4, mean, rstd, d["dy"], gate=d["gate"],
                             silu=True)
    assert all(torch.isfinite(t).all() for t in g.values())


def test_a_bad_sample_stays_alone():
    for N, S, C, groups in ((50, 1, 128, 2), (3, 200, 64, 4)):
        d = make(N, S, C, "bf16", True)
        y0, g0 = check(d, groups, "bf16", True)
        d["x"][1, S // 2, 3] = float("nan")
        y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], groups, gate=d["gate"], silu=True)
        keep = [n for n in range(N) if n != 1]
        assert torch.equal(y[keep], y0[keep])
        assert torch.equal(y[1, :, C // groups:], y0[1, :, C // groups:])
        assert torch.isnan(y[1, :, : C // groups]).all()


def test_gradient_is_the_difference_of_the_loss():
    """Differences in 64 bits of the definition along random directions."""
    d = make(2, 6, 32, "fp32", True, seed=9)
    _, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], 4, gate=d["gate"], silu=True)
    g = G.gdn_group_norm_bwd(d["x"], d["w"], d["b"], 4, mean, rstd, d["dy"], gate=d["gate"],
                             silu=True)
    for name, grad in (("x", "dx"), ("w", "dweight"), ("b", "dbias"), ("gate", "dgate")):
        way = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(2)).cuda().double()

        def loss(e):
            x = {n: t.double() for n, t in d.items()}
            x[name] = x[name] + e * way
            y = lin.group_norm(x["x"], x["w"], x["b"], 4, x["gate"], True)[0]
            return (y * f64(d["dy"])).sum()
        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        dot = float((g[grad].double() * way).sum())
        assert abs(diff - dot) <= 1e-5 * float(g[grad].double().norm() * way.norm())


def test_repeated_calls_and_another_stream():
    d = make(4, 700, 320, "bf16", True)
    y, mean, rstd = G.gdn_group_norm(d["x"], d["w"], d["b"], 32, gate=d["gate"], silu=True)
    g = G.gdn_group_norm_bwd(d["x"], d["w"], d["b"], 32, mean, rstd, d["dy"], gate=d["gate"],
                             silu=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(2):
        y2, m2, r2 = G.gdn_group_norm(d["x"], d["w"], d["b"], 32, gate=d["gate"], silu=True,
                                      stream=side)
        g2 = G.gdn_group_norm_bwd(d["x"], d["w"], d["b"], 32, m2, r2, d["dy"], gate=d["gate"],
                                  silu=True, stream=side)
        side.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_nothing_to_do():
    w = torch.ones(8, device="cuda")
    for shape in ((0, 3, 8), (3, 0, 8)):
        x = torch.empty(shape, device="cuda")
        y, mean, rstd = G.gdn_group_norm(x, w, w, 2)
        assert y.shape == x.shape and mean.shape == (shape[0], 2)
        g = G.gdn_group_norm_bwd(x, w, w, 2, mean, rstd, x)
        assert (g["dweight"] == 0).all() and (g["dbias"] == 0).all()
