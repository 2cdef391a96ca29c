"""The fp64 oracle of the selective scan, the short convolution and the q/k norm against
independent statements: closed forms, library routines, differences."""
import math

import numpy as np
import pytest
import torch

import oracle.ssm as O

torch.set_default_dtype(torch.float32)


def rnd(*s, seed=0, lo=None):
    g = torch.Generator().manual_seed(seed + 31 * len(s) + sum(s))
    t = torch.randn(*s, generator=g, dtype=torch.float64)
    return t if lo is None else t.abs() + lo


def scan_inputs(B=2, T=7, D=8, S=3, G=2):
    return dict(x=rnd(B, T, D), dt=rnd(B, T, D, seed=1), A_log=0.3 * rnd(D, S), b=rnd(B, T, G, S),
                c=rnd(B, T, G, S, seed=2), h0=rnd(B, D, S), D_skip=rnd(D), gate=rnd(B, T, D, seed=3),
                dt_bias=rnd(D, seed=4))


def test_scan_is_the_unrolled_sum():
    i = scan_inputs()
    y, last = O.scan(**i, dt_softplus=True)
    delta = np.log1p(np.exp((i["dt"] + i["dt_bias"]).numpy()))
    A, x, b, c = (i[n].numpy() for n in ("A_log", "x", "b", "c"))
    A = -np.exp(A)
    total = np.cumsum(delta, 1)
    for n in range(2):
        for d in range(8):
            g = d // 4
            for t in range(7):
                want = sum(
                    sum(math.exp(A[d, s] * (total[n, t, d] - total[n, u, d])) * delta[n, u, d] *
                        x[n, u, d] * b[n, u, g, s] for u in range(t + 1)) * c[n, t, g, s] +
                    math.exp(A[d, s] * total[n, t, d]) * float(i["h0"][n, d, s]) * c[n, t, g, s]
                    for s in range(3)) + float(i["D_skip"][d]) * x[n, t, d]
                z = float(i["gate"][n, t, d])
                assert abs(want * z / (1 + math.exp(-z)) - float(y[n, t, d])) < 1e-12


def test_scan_with_one_rate_a_head_is_the_diagonal_recurrence():
    import oracle.diag
    B, T, H, S, Dh = 1, 9, 2, 4, 3
    v, b, c = rnd(B, T, H, Dh), rnd(B, T, H, S), rnd(B, T, H, S, seed=5)
    g, A_log = rnd(B, T, H, lo=0.1), 0.2 * rnd(H, S)
    o, s = oracle.diag.forward(v.numpy(), b.numpy(), c.numpy(), g.numpy(), A_log.numpy(), None)
    wide = lambda t: t.repeat_interleave(Dh, -1)  # noqa: E731
    delta = wide(g)
    y, last = O.scan(v.reshape(B, T, H * Dh) / delta, delta, A_log.repeat_interleave(Dh, 0), b, c)
    assert np.abs(y.numpy().reshape(o.shape) - o).max() < 1e-12
    assert np.abs(last.view(B, H, Dh, S).transpose(2, 3).numpy() - s).max() < 1e-12


def test_packed_sequences_are_separate_ones():
    i = scan_inputs(B=1, T=9)
    cu = [0, 4, 4, 9]
    h0 = rnd(3, 8, 3, seed=9)
    y, last = O.scan(**{**i, "h0": h0}, cu=cu)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        part = {k: (v[:, a:b] if v.dim() > 2 and k != "h0" else v) for k, v in i.items()}
        yn, ln = O.scan(**{**part, "h0": h0[n:n + 1]})
        assert torch.equal(yn[0], y[0, a:b]) and torch.equal(ln[0], last[n])
    w, bias, prev = rnd(8, 4), rnd(8), rnd(3, 3, 8)
    y, tail = O.conv(i["x"], w, bias, prev, cu)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        yn, tn = O.conv(i["x"][:, a:b], w, bias, prev[n:n + 1])
        assert torch.equal(yn[0], y[0, a:b]) and torch.equal(tn[0], tail[n])
    assert torch.equal(tail[1], prev[1])


@pytest.mark.parametrize("K", [1, 2, 4])
def test_conv_is_the_library_convolution(K):
    x, w, bias = rnd(2, 11, 6), rnd(6, K), rnd(6)
    want = torch.nn.functional.conv1d(x.transpose(1, 2), w[:, None], bias, padding=K - 1, groups=6)
    want = torch.nn.functional.silu(want[..., :11]).transpose(1, 2)
    assert torch.allclose(O.conv(x, w, bias)[0], want, atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_turns_complex_numbers(interleaved):
    x, f = rnd(2, 5, 3, 8), torch.tensor([1.0, 0.25, 1e-3], dtype=torch.float64)
    pos = torch.tensor([[0, 1, 2, 1000, 70000], [5, 4, 3, 2, 1]])
    u = O.qk(x, positions=pos, inv_freq=f, interleaved=interleaved)
    n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    for i in range(3):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + 3)
        for p in range(5):
            z = complex(0, 1) * float(pos[1, p]) * float(f[i])
            e = np.exp(z) * (n[1, p, :, a].numpy() + 1j * n[1, p, :, b].numpy())
            assert np.abs(e - (u[1, p, :, a].numpy() + 1j * u[1, p, :, b].numpy())).max() < 1e-12
    assert torch.equal(u[..., 6:], n[..., 6:])
    assert torch.allclose((u * u).sum(-1), (n * n).sum(-1))


def check_differences(fn, inputs, d_outs, **how):
    """Autograd against central differences along random directions."""
    g = O.grads(fn, inputs, d_outs, **how)

    def value(ins):
        outs = fn(**ins, **how)
        outs = outs if isinstance(outs, tuple) else (outs,)
        return float(sum((o * d).sum() for o, d in zip(outs, d_outs) if d is not None))

    for n, t in inputs.items():
        v = rnd(*t.shape, seed=77)
        e = 1e-5
        diff = (value({**inputs, n: t + e * v}) - value({**inputs, n: t - e * v})) / (2 * e)
        assert abs(diff - float((g[n] * v).sum())) < 1e-6 * max(1.0, abs(diff)), n


def test_gradients_are_differences():
    i = scan_inputs()
    check_differences(O.scan, i, (rnd(2, 7, 8, seed=50), rnd(2, 8, 3, seed=51)), dt_softplus=True)
    c = dict(x=rnd(2, 7, 6), w=rnd(6, 3), bias=rnd(6), x_prev=rnd(2, 2, 6))
    check_differences(O.conv, c, (rnd(2, 7, 6, seed=52), rnd(2, 2, 6, seed=53)))
    q = dict(x=rnd(2, 4, 3, 8), weight=rnd(8))
    for l2 in (False, True):
        check_differences(O.qk, q, (rnd(2, 4, 3, 8, seed=54),), l2norm=l2, scale=0.7,
                          inv_freq=torch.tensor([1.0, 0.1]), positions=torch.arange(8).view(2, 4))
