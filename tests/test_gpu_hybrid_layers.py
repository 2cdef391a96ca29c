"""The scan, the convolution, the q/k norm and linear attention together: the layers of
examples/hybrid_layers.py trained and served, and their gradients against autograd of the
formulas in 64 bits."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import hybrid_layers as X  # noqa: E402

import oracle.ssm as O  # noqa: E402

pytestmark = pytest.mark.gpu


def formula(m, u):
    """The layers' training pass in fp64 torch on the CPU."""
    w = {n: getattr(m, n).detach().cpu().double().requires_grad_()
         for n in ("w_in", "w_x", "w_dt", "w_out", "conv_w", "conv_b", "A_log", "D_skip", "dt_bias",
                   "w_qkv", "w_o", "q_norm", "k_norm")}
    S, R = m.states, m.rank
    x, z = (u @ w["w_in"]).chunk(2, -1)
    x, _ = O.conv(x, w["conv_w"], w["conv_b"])
    p = x @ w["w_x"]
    y, _ = O.scan(x, p[..., :R] @ w["w_dt"], w["A_log"], p[..., R:R + S].unsqueeze(-2),
                  p[..., R + S:].unsqueeze(-2), None, None, w["D_skip"], z, w["dt_bias"], True)
    u = u + y @ w["w_out"]
    B, T, _ = u.shape
    q, k, v = (u @ w["w_qkv"]).view(B, T, 3, m.heads, m.head).unbind(2)
    f = m.inv_freq.cpu()
    q = O.qk(q, w["q_norm"], None, f, m.head ** -0.5)
    k = O.qk(k, w["k_norm"], None, f)
    t = torch.arange(T)
    back = (t[:, None] - t[None]).clamp(min=0)
    decay = torch.exp(m.log_decay.cpu().double()[:, None, None] * back) * (t[:, None] >= t[None])
    o = torch.einsum("bthd,bshd->bhts", q, k) * decay
    o = torch.einsum("bhts,bshd->bthd", o, v).reshape(B, T, -1)
    return u + o @ w["w_o"], w


def test_training_pass_and_gradients():
    """In fp32: the library's matrix products round at 2^-24 (TF32 off), a chain of some ten
    operators over 60 tokens and sums of up to 256 terms: 2^-13 of a tensor's norm is
    2000 such roundings in a row."""
    torch.backends.cuda.matmul.allow_tf32 = False
    m = X.Layers(width=64, inner=64, dtype=torch.float32, heads=1)
    gen = torch.Generator().manual_seed(3)
    u, d = (torch.randn(2, 60, 64, generator=gen) for _ in range(2))
    y = m.train_forward(u.cuda())
    y.backward(d.cuda())
    ref, w = formula(m, u.double())
    ref.backward(d.double())
    assert float((y.detach().cpu().double() - ref.detach()).norm() / ref.detach().norm()) < 2.0 ** -13
    for n, t in w.items():
        got = getattr(m, n).grad.cpu().double()
        assert float((got - t.grad).norm() / t.grad.norm()) < 2.0 ** -13, n


def test_example_trains():
    losses = X.train(steps=3)
    assert len(losses) == 3 and all(l == l and l < float("inf") for l in losses)


def test_example_serves_what_one_pass_gives():
    """bf16 throughout: every one of some ten roundings on a token's way (2^-8 each, partly
    cancelling) may differ between the two, and earlier tokens' too: 2^-4 in all."""
    results, layers = X.serve()
    assert len(results) == 6
    for u, y in results:
        want = X.whole(layers, u)[-len(y):].float()
        assert float((y.float() - want).norm() / want.norm()) < 2.0 ** -4


def test_serving_step_in_a_graph():
    """The three single-token calls captured into two graphs that share a workspace, and
    replayed: the states move on as in eager calls."""
    m = X.Layers()
    gen = torch.Generator().manual_seed(1)
    N, P = 5, 9
    pages = torch.tensor([3, 0, 8, -1, 5], dtype=torch.int32).cuda()
    pools = [torch.randn(P, 3, m.inner, generator=gen).bfloat16().cuda(),
             torch.randn(P, m.inner, m.states, generator=gen).cuda()]
    again = [p.clone() for p in pools]
    x = torch.randn(N, m.inner, generator=gen).bfloat16().cuda()
    q = torch.randn(N, 1, m.heads, m.head, generator=gen).bfloat16().cuda()
    pos = torch.full((N, 1), 100000, dtype=torch.int32).cuda()
    ws = torch.zeros(256, dtype=torch.uint8).cuda()
    g = X.gdn

    @torch.no_grad()
    def step(convs, scans):
        y, _ = g.gdn_conv_step(x, m.conv_w, convs, m.conv_b, pages, workspace=ws)
        dt, b, c = (t.contiguous() for t in m.steps(y))
        y, _ = g.gdn_ssm_step(y, dt, m.A_log, b, c, scans, pages, D_skip=m.D_skip, dt_bias=m.dt_bias,
                              dt_softplus=True, workspace=ws)
        return (y, *g.gdn_qk_norm(q, q, m.q_norm, m.k_norm, pos, m.inv_freq))

    for _ in range(2):
        want = step(*pools)
    torch.cuda.synchronize()
    step(*[p.clone() for p in again])   # (what the libraries set up at their first call)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            got = step(*again)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert all(torch.equal(a, b) for a, b in zip(pools, again))
