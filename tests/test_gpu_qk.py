"""Norm of q and k with the rotation (gdn_qk_norm, gdn_qk_norm_bwd) on the GPU against the
fp64 oracle.  Tolerances, relative L2 of a tensor: a sum of D <= 256 squares (its terms all
of one sign: log2 steps over lanes, 8 in a row: 2^-20), a reciprocal root (2^-22), an angle
(2^-22 of a turn) and a few operations: 2^-19.  Sums over rows run over 64 rows, then over a
thread's, a CTA's and the CTAs' sums, some 300 in a row: 2^-24 300 sqrt(rows) of their
random terms.  bf16 adds 2^-8."""
import pytest
import torch

import oracle.ssm as O
from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


def inputs(B, T, Hq, Hk, D, R, dtype, seed=0, weights=True, far=False):
    g = torch.Generator().manual_seed(1000 * T + D + R + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    wide = r(B, T, (Hq + 2 * Hk) * D).to(dtype).cuda()
    i = dict(q=wide[..., :Hq * D].view(B, T, Hq, D),
             k=wide[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D),
             q_weight=(1 + 0.2 * r(D)).cuda() if weights else None,
             k_weight=(1 + 0.2 * r(D)).cuda() if weights else None,
             d_q=r(B, T, Hq, D).to(dtype).cuda(), d_k=r(B, T, Hk, D).to(dtype).cuda(),
             positions=None, inv_freq=None)
    if R:
        i["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2) / R)).cuda()
        i["positions"] = torch.randint(0, 2 ** 24 if far else 5000, (B, T), generator=g,
                                       dtype=torch.int32).cuda()
    return i


def close(got, ref, tol, what=""):
    tol = tol + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    err, size = float((got.detach().cpu().double() - ref).norm()), float(ref.norm())
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.2e} > {tol:.2e}"


def check(i, l2=False, inter=False, scale=0.3, eps=1e-6):
    how = dict(q_scale=scale, l2norm=l2, interleaved=inter, eps=eps)
    pos, freq = i["positions"], i["inv_freq"]
    out = G.gdn_qk_norm(i["q"], i["k"], i["q_weight"], i["k_weight"], pos, freq, **how)
    g = G.gdn_qk_norm_bwd(i["q"], i["k"], i["d_q"], i["d_k"], i["q_weight"], i["k_weight"], pos,
                          freq, **how)
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    for n, got, s in (("q", out[0], scale), ("k", out[1], 1.0)):
        kw = dict(positions=cpu(pos), inv_freq=cpu(freq), scale=s, l2norm=l2, interleaved=inter,
                  eps=eps)
        close(got, O.qk(O._d(i[n]), O._d(i[n + "_weight"]), **kw), 2.0 ** -19, n)
        ref = O.grads(O.qk, dict(x=i[n], weight=i[n + "_weight"]), (i["d_" + n],), **kw)
        close(g["d" + n], ref["x"], 2.0 ** -18, "d" + n)
        if i[n + "_weight"] is not None:
            rows = i[n].shape[0] * i[n].shape[1] * i[n].shape[2]
            close(g[f"d{n}_weight"], ref["weight"], 2.0 ** -19 + 300 * rows ** 0.5 * 2.0 ** -24)
    return out, g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,T,Hq,Hk,D,R", [
    (1, 1, 1, 1, 8, 8), (2, 3, 2, 1, 32, 32), (1, 17, 4, 2, 64, 64), (2, 9, 3, 3, 80, 40),
    (1, 33, 5, 1, 96, 48), (3, 5, 2, 2, 128, 32), (1, 9, 2, 1, 256, 256), (2, 21, 16, 4, 64, 6),
    (1, 40, 8, 8, 24, 0), (1, 7, 1, 1, 256, 2)])
def test_sizes(B, T, Hq, Hk, D, R, inter, dtype):
    check(inputs(B, T, Hq, Hk, D, R, dtype), inter=inter)


def test_many_tokens():
    check(inputs(2, 1601, 3, 1, 64, 32, torch.float32))
    check(inputs(1, 2500, 2, 2, 128, 128, torch.bfloat16))


@pytest.mark.parametrize("inter", [False, True])
def test_l2_without_weights(inter):
    check(inputs(2, 30, 4, 4, 64, 64, torch.float32, weights=False), l2=True, inter=inter)


def test_far_positions():
    """Positions of millions: an angle is as exact as a near one."""
    i = inputs(1, 64, 2, 2, 64, 64, torch.float32, far=True)
    check(i)
    i["positions"] = -i["positions"]
    check(i)
    i["inv_freq"] = i["inv_freq"] * 50   # more than a turn a token
    check(i)


def test_positions_count_up_by_default():
    i = inputs(3, 50, 2, 1, 64, 32, torch.bfloat16)
    how = (i["q"], i["k"], i["q_weight"], i["k_weight"])
    pos = torch.arange(50, dtype=torch.int32).expand(3, 50).contiguous().cuda()
    a, b = G.gdn_qk_norm(*how, None, i["inv_freq"]), G.gdn_qk_norm(*how, pos, i["inv_freq"])
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_zero_rows_and_values_that_are_not_finite():
    i = inputs(1, 8, 2, 2, 64, 64, torch.float32)
    i["q"] = i["q"].clone()
    i["q"][0, 3] = 0
    check(i)
    (q, k), g = check(i)
    i["q"][0, 5, 1, 7] = float("nan")
    q2, k2 = G.gdn_qk_norm(i["q"], i["k"], i["q_weight"], i["k_weight"], i["positions"],
                           i["inv_freq"], q_scale=0.3)
    q, q2 = q.view(16, 64), q2.view(16, 64)
    rest = [r for r in range(16) if r != 11]
    assert torch.equal(k, k2) and torch.equal(q[rest], q2[rest]) and torch.isnan(q2[11]).all()


def test_gradients_are_differences():
    i = inputs(1, 12, 2, 2, 32, 16, torch.float32)
    i["q"], i["k"] = i["q"].contiguous(), i["k"].contiguous()
    names = ("q", "k", "q_weight", "k_weight", "positions", "inv_freq")

    def value(j):
        q, k = G.gdn_qk_norm(*(j[n] for n in names))
        return float((q.double() * i["d_q"].double()).sum() + (k.double() * i["d_k"].double()).sum())

    g = G.gdn_qk_norm_bwd(i["q"], i["k"], i["d_q"], i["d_k"], *(i[n] for n in names[2:]))
    gen = torch.Generator().manual_seed(2)
    for n in names[:4]:
        v = torch.randn(i[n].shape, generator=gen).cuda()
        e = 2.0 ** -7
        diff = (value({**i, n: i[n] + e * v}) - value({**i, n: i[n] - e * v})) / (2 * e)
        exact = float((g["d" + n].double() * v.double()).sum())
        # the third derivative's share, e^2, and the outputs' rounding (28 x 28 of norm) over e
        assert abs(diff - exact) <= 30 * e * e * (abs(exact) + 1) + 1600 * 2.0 ** -21 / e, n


def test_reproducible_on_streams_and_in_graphs():
    i = inputs(2, 900, 4, 2, 64, 64, torch.bfloat16)
    names = ("q_weight", "k_weight", "positions", "inv_freq")
    run = lambda **kw: (*G.gdn_qk_norm(i["q"], i["k"], *(i[n] for n in names), **kw),  # noqa: E731
                        *G.gdn_qk_norm_bwd(i["q"], i["k"], i["d_q"], i["d_k"],
                                           *(i[n] for n in names), **kw).values())
    a = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = run()
    graph.replay()
    torch.cuda.synchronize()
    for other in (b, c):
        assert all(torch.equal(u, v) for u, v in zip(a, other))


def test_no_tokens():
    i = inputs(2, 0, 2, 1, 64, 64, torch.float32)
    q, k = G.gdn_qk_norm(i["q"], i["k"], i["q_weight"], i["k_weight"], i["positions"], i["inv_freq"])
    assert q.numel() == 0 and k.numel() == 0
    g = G.gdn_qk_norm_bwd(i["q"], i["k"], i["d_q"], i["d_k"], i["q_weight"], i["k_weight"],
                          i["positions"], i["inv_freq"])
    assert (g["dq_weight"] == 0).all() and (g["dk_weight"] == 0).all()
