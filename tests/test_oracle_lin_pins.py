"""CPU pins of the 64-bit definitions in oracle/lin.py: closed forms,
differences of the loss, autograd."""
import numpy as np
import pytest
import torch

from oracle import lin

RNG = np.random.default_rng(3)


def _inputs(B=2, T=7, H=2, dk=3, dv=4):
    q, k = RNG.standard_normal((2, B, T, H, dk))
    return q, k, RNG.standard_normal((B, T, H, dv)), np.array([-0.3, -0.05])[:H], \
        RNG.standard_normal((B, H, dk, dv))


def test_forward_is_the_masked_product():
    """o_t = sum_{s<=t} lam^(t-s) (q_t.k_s) v_s + lam^(t+1) S_0^T q_t, summed directly."""
    q, k, v, ld, s0 = _inputs()
    o, sT = lin.forward(q, k, v, ld, s0)
    T = q.shape[1]
    t = np.arange(T)
    w = np.exp(ld[:, None, None] * np.maximum(t[:, None] - t[None], 0)) * (t[:, None] >= t[None])
    ref = np.einsum("bthi,bshi,hts,bshj->bthj", q, k, w, v) + \
        np.einsum("th,bhij,bthi->bthj", np.exp(np.outer(t + 1, ld)), s0, q)
    assert np.abs(o - ref).max() < 1e-12
    end = np.einsum("sh,bshi,bshj->bhij", np.exp(np.outer(T - 1 - t, ld)), k, v) + \
        np.exp(T * ld)[:, None, None] * s0
    assert np.abs(sT - end).max() < 1e-12


def test_packed_sequences_are_separate_ones():
    q, k, v, ld, _ = _inputs(B=1, T=9)
    cu = [0, 4, 4, 9]
    s0 = RNG.standard_normal((3, 2, 3, 4))
    o, sT = lin.forward(q, k, v, ld, s0, cu)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        o1, s1 = lin.forward(q[:, a:b], k[:, a:b], v[:, a:b], ld, s0[n:n + 1])
        assert np.array_equal(o[:, a:b], o1) and np.array_equal(sT[n], s1[0])


def test_gradients_are_differences_of_the_loss():
    q, k, v, ld, s0 = _inputs(B=1, T=5)
    d_o, d_s = RNG.standard_normal(v.shape), RNG.standard_normal(s0.shape)
    g = lin.backward(q, k, v, ld, d_o, s0, d_s)

    def loss():
        o, s = lin.forward(q, k, v, ld, s0)
        return (o * d_o).sum() + (s * d_s).sum()

    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dh0", s0)):
        for at in RNG.choice(x.size, 12, replace=False):
            i, old, h = np.unravel_index(at, x.shape), x.flat[at], 1e-6
            x[i] = old + h
            up = loss()
            x[i] = old - h
            down = loss()
            x[i] = old
            assert abs((up - down) / (2 * h) - g[name][i]) < 1e-6 * max(1, abs(g[name][i]))


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_group_norm_and_gradients_match_autograd(silu, gated):
    N, S, C, G = 2, 3, 12, 3
    x, dy, z = (torch.from_numpy(RNG.standard_normal((N, S, C))) for _ in range(3))
    w, b = (torch.from_numpy(RNG.standard_normal(C)) for _ in range(2))
    for t in (x, z, w, b):
        t.requires_grad_()
    y = torch.nn.functional.group_norm(x.permute(0, 2, 1), G, w, b, 1e-5).permute(0, 2, 1)
    y = torch.nn.functional.silu(y) if silu else y
    y = y * torch.nn.functional.silu(z) if gated else y
    y.backward(dy)
    a = [t.detach().numpy() for t in (x, w, b)]
    gate = z.detach().numpy() if gated else None
    got, _, _ = lin.group_norm(a[0], a[1], a[2], G, gate, silu)
    assert np.abs(got - y.detach().numpy()).max() < 1e-12
    g = lin.group_norm_bwd(a[0], a[1], a[2], G, dy.numpy(), gate, silu)
    for name, t in (("dx", x), ("dweight", w), ("dbias", b)) + ((("dgate", z),) if gated else ()):
        assert np.abs(g[name] - t.grad.numpy()).max() < 1e-11


def test_pages_keep_every_row_s_contents():
    """Fork, snapshot, free and compact never change what a row's pages hold."""
    P, R, M = 24, 10, 4
    pool = RNG.standard_normal((P, 2))
    pages = lin.Pages(np.full((R, M), -1), np.zeros(R), np.zeros(P), pool)
    pages.fork([-1, -1, -1], [0, 1, 2])
    assert (pages.pool[:3] == 0).all()
    pages.pool[:3] = RNG.standard_normal((3, 2))
    pages.fork([0, 1], [0, 1])            # snapshots
    pages.fork([0, 0, 1, 2], [5, 6, 7, 8])

    def contents():
        return {r: pages.pool[pages.table[r, :pages.counts[r]]].tolist() for r in range(R)
                if pages.counts[r]}

    before = contents()
    assert before[5] == before[6] == before[0] and before[7] == before[1]
    pages.free([0, 2, 6])
    want = {r: c for r, c in contents().items()}
    live = pages.compact()
    assert contents() == want == {r: before[r] for r in want}
    assert live == (pages.refs > 0).sum() and (pages.refs[live:] == 0).all()
    held = np.bincount([p for r in range(R) for p in pages.table[r, :pages.counts[r]]], minlength=P)
    assert np.array_equal(held, pages.refs)
