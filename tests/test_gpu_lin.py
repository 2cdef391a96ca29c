"""GPU parity of linear attention with a decay for each head (gdn_lin_fwd,
gdn_lin_bwd, gdn_lin_decode) against the 64-bit definition.

Bounds, relative L2 (derived from the arithmetic, not from a run).  fp32
results are sums of at most a few hundred fp32 products, each with a relative
rounding of 2^-24, carried from chunk to chunk by a factor <= 1: 5e-6.  bf16
results see three independent roundings to 8 bits, of root mean square 1.6e-3
each: the weights inside a chunk, the state as it is read, and the output:
sqrt(3) * 1.6e-3 = 2.8e-3, with room for small samples 4e-3.  States stay in
fp32 and bf16 products are exact in it: 5e-6 for either storage type."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin
from parity import rel

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
TOL = {"fp32": 5e-6, "bf16": 4e-3}
STATE_TOL = 5e-6


def f64(t):
    return t.double().cpu().numpy()


def make(B, T, H, dk, dv, dtype, seed=0, N=None, init=True, decay=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(q=(r(B, T, H, dk) / dk ** 0.5).to(DT[dtype]), k=r(B, T, H, dk).to(DT[dtype]),
             v=r(B, T, H, dv).to(DT[dtype]), d_o=r(B, T, H, dv).to(DT[dtype]))
    d["log_decay"] = decay if decay is not None else \
        -torch.exp2(-8.0 * torch.arange(1, H + 1) / H).float()
    N = B if N is None else N
    d["s0"] = r(N, H, dk, dv) if init else None
    d["d_sT"] = r(N, H, dk, dv) / dk ** 0.5 if init else None
    return {n: t if t is None else t.cuda() for n, t in d.items()}


def check_fwd(d, dtype, cu=None, **kw):
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], cud, check=True, **kw)
    o_ref, s_ref = lin.forward(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], cu)
    assert rel(f64(o), o_ref) <= TOL[dtype]
    assert rel(f64(s), s_ref) <= STATE_TOL
    return o, s


def check_bwd(d, dtype, cu=None, **kw):
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], cud, d["d_sT"],
                      check=True, **kw)
    ref = lin.backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], d["d_sT"], cu)
    for name in ("dq", "dk", "dv"):
        assert g[name].dtype == DT[dtype]
        assert rel(f64(g[name]), ref[name]) <= TOL[dtype], name
    assert rel(f64(g["dh0"]), ref["dh0"]) <= STATE_TOL
    return g


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(dtype, dk, dv, T):
    d = make(2, T, 2, dk, dv, dtype, seed=T)
    check_fwd(d, dtype)
    check_bwd(d, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 96), (64, 128), (128, 64), (128, 256), (96, 64),
                                   (256, 128), (160, 32)])
def test_head_sizes(dtype, dk, dv):
    d = make(1, 200, 3, dk, dv, dtype, seed=dk + dv)
    check_fwd(d, dtype)
    check_bwd(d, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("init", [False, True])
def test_packed_sequences(dtype, init):
    """Ragged lengths, one token, empty sequences, whole chunks."""
    lens = [130, 1, 0, 64, 257, 128, 0, 5]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(1, cu[-1], 2, 64, 64, dtype, seed=5, N=len(lens), init=init)
    _, s = check_fwd(d, dtype, cu)
    g = check_bwd(d, dtype, cu)
    for n in (2, 6):  # an empty sequence: states pass through
        assert torch.equal(s[n], d["s0"][n] if init else torch.zeros_like(s[n]))
        assert torch.equal(g["dh0"][n], d["d_sT"][n] if init else torch.zeros_like(s[n]))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_values_outside_a_sequence_never_reach_it(dtype):
    """An infinity or NaN in a neighbour's tokens stays with the neighbour."""
    cu = [0, 100, 180, 300]
    d = make(1, 300, 2, 64, 64, dtype, seed=6, N=3)
    clean = {n: None if t is None else t.clone() for n, t in d.items()}
    for name, bad in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")),
                      ("d_o", float("-inf"))):
        d[name][:, 100:180] = bad
    d["s0"][1], d["d_sT"][1] = float("inf"), float("nan")
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    outs = []
    for x in (clean, d):
        o, s = G.gdn_lin_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], cud, check=True)
        g = G.gdn_lin_bwd(x["q"], x["k"], x["v"], x["log_decay"], x["d_o"], x["s0"], cud, x["d_sT"],
                          check=True)
        outs.append((o, s, g))
    (o0, s0, g0), (o1, s1, g1) = outs
    for a, b in [(o0, o1)] + [(g0[n], g1[n]) for n in ("dq", "dk", "dv")]:
        assert torch.equal(a[:, :100], b[:, :100]) and torch.equal(a[:, 180:], b[:, 180:])
    for a, b in ((s0, s1), (g0["dh0"], g1["dh0"])):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rate", [0.0, -1e-4, -3.0, -60.0, -1e6, float("-inf")])
def test_decays(dtype, rate):
    """No decay at all, a nearly lost one, and states that vanish at once."""
    d = make(1, 150, 2, 64, 64, dtype, seed=7, decay=torch.tensor([rate, -0.1]))
    if rate == float("-inf"):
        # lam = 0: the state is the last write; the definition's 0 * S is exact
        o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
        k, v = f64(d["k"])[0, -1, 0], f64(d["v"])[0, -1, 0]
        assert rel(f64(s)[0, 0], np.outer(k, v)) <= STATE_TOL
        assert torch.isfinite(o).all()
        return
    check_fwd(d, dtype)
    check_bwd(d, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_slices_of_one_projection(dtype):
    """q, k and v as they lie in one projection give the result of their copies, bit for bit."""
    B, T, H, D = 2, 150, 3, 64
    d = make(B, T, H, D, D, dtype, seed=8)
    qkv = torch.stack([d["q"], d["k"], d["v"]], dim=2)
    q, k, v = qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]
    assert not q.is_contiguous()
    a = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    b = G.gdn_lin_fwd(q, k, v, d["log_decay"], d["s0"], check=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"])
    gb = G.gdn_lin_bwd(q, k, v, d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"])
    assert all(torch.equal(ga[n], gb[n]) for n in ga)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_chained_calls_equal_one(dtype):
    d = make(2, 333, 2, 64, 64, dtype, seed=9)
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    state, outs = d["s0"].clone(), []
    for a, b in ((0, 100), (100, 101), (101, 333)):
        q, k, v = (d[n][:, a:b].contiguous() for n in "qkv")
        outs.append(G.gdn_lin_fwd(q, k, v, d["log_decay"], state, final_state=state)[0])
    assert rel(f64(torch.cat(outs, 1)), f64(o)) <= 2 * TOL[dtype]
    assert rel(f64(state), f64(s)) <= 2 * STATE_TOL


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 5000, 2, 64, 64), (1, 4100, 1, 128, 128),
                                   (2, 2500, 3, 128, 64), (3, 2048, 2, 32, 32)])
def test_few_long_sequences(dtype, shape):
    """Few units and a long axis (the calls that are split along it)."""
    d = make(*shape, dtype, seed=10)
    check_fwd(d, dtype)
    check_bwd(d, dtype)


def test_few_long_packed_sequences():
    cu = [0, 3000, 3001, 7300]
    d = make(1, 7300, 2, 128, 128, "bf16", seed=11, N=3)
    check_fwd(d, "bf16", cu)
    check_bwd(d, "bf16", cu)


@pytest.mark.parametrize("shape", [(8, 512, 16, 64, 64), (4, 384, 16, 128, 128)])
def test_many_units(shape):
    """More units than SMs, against the definition on a sample of them."""
    d = make(*shape, "bf16", seed=12)
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"],
                      check=True)
    for n, h in ((0, 0), (shape[0] - 1, shape[2] - 1), (1, 7)):
        part = {x: None if t is None else
                (t[h:h + 1] if x == "log_decay" else
                 t[n:n + 1, h:h + 1] if x in ("s0", "d_sT") else t[n:n + 1, :, h:h + 1])
                for x, t in d.items()}
        o_ref, s_ref = lin.forward(part["q"], part["k"], part["v"], part["log_decay"], part["s0"])
        ref = lin.backward(part["q"], part["k"], part["v"], part["log_decay"], part["d_o"],
                           part["s0"], part["d_sT"])
        assert rel(f64(o[n:n + 1, :, h:h + 1]), o_ref) <= TOL["bf16"]
        assert rel(f64(s[n:n + 1, h:h + 1]), s_ref) <= STATE_TOL
        for x in ("dq", "dk", "dv"):
            assert rel(f64(g[x][n:n + 1, :, h:h + 1]), ref[x]) <= TOL["bf16"], x
        assert rel(f64(g["dh0"][n:n + 1, h:h + 1]), ref["dh0"]) <= STATE_TOL


def test_gradients_are_differences_of_the_loss():
    """fp32 differences of the forward pass along random directions: the loss
    is linear in each input alone, so a central difference has no curvature and
    only the rounding of the losses is left (1e-3 of their size at this step)."""
    d = make(1, 90, 2, 32, 64, "fp32", seed=13)
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"],
                      check=True)

    def loss(x):
        o, s = G.gdn_lin_fwd(x["q"], x["k"], x["v"], x["log_decay"], x["s0"], check=True)
        return (o.double() * d["d_o"].double()).sum() + (s.double() * d["d_sT"].double()).sum()

    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("s0", "dh0")):
        way = torch.randn(d[name].shape, generator=torch.Generator().manual_seed(1)).cuda()
        up, down = ({**d, name: d[name] + e * way} for e in (1.0, -1.0))
        diff = (loss(up) - loss(down)) / 2
        dot = (g[grad].double() * way.double()).sum()
        scale = g[grad].double().norm() * way.double().norm()
        assert abs(diff - dot) <= 1e-4 * scale, name


def test_bad_offsets_are_reported():
    d = make(1, 40, 1, 64, 64, "bf16", N=3)
    for cu in ([0, 10, 9, 40], [1, 10, 20, 40], [0, 10, 20, 39]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        with pytest.raises(G.GdnError) as e:
            G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], cud, check=True)
        assert e.value.status == 6
        with pytest.raises(G.GdnError) as e:
            G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], cud, d["d_sT"],
                          check=True)
        assert e.value.status == 6


def test_no_tokens_pass_the_states_through():
    d = make(2, 0, 2, 64, 64, "bf16")
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    assert o.numel() == 0 and torch.equal(s, d["s0"])
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"])
    assert torch.equal(g["dh0"], d["d_sT"])


def test_another_stream_and_repeated_calls():
    """The same bits on a side stream, call after call (no atomics in sums)."""
    d = make(2, 700, 3, 64, 64, "bf16", seed=14)
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"])
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        o2, s2 = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], stream=side)
        g2 = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None,
                           d["d_sT"], stream=side)
        side.synchronize()
        assert torch.equal(o, o2) and torch.equal(s, s2)
        assert all(torch.equal(g[n], g2[n]) for n in g)


# ---- decode -----------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 32, 32), (5, 3, 64, 64), (3, 2, 128, 128),
                                       (4, 2, 64, 256), (2, 1, 256, 96), (33, 5, 96, 32)])
def test_decode_on_pages(dtype, N, H, dk, dv):
    """Pages in any order, a padded row, a pool of several layers (strided pages)."""
    d = make(N, 1, H, dk, dv, dtype, seed=N)
    q, k, v = (d[n][:, 0].contiguous() for n in "qkv")
    P = 2 * N + 1
    pool = torch.randn(P, 2, H, dk, dv, device="cuda")
    before = pool.clone()
    pages = torch.randperm(P)[:N].to(torch.int32)
    pages[N // 2] = -1 if N > 1 else pages[0]
    o, s = G.gdn_lin_decode(q, k, v, d["log_decay"], pool[:, 1], pages.cuda(), check=True)
    lam = np.exp(f64(d["log_decay"]))[:, None, None]
    ref = before.double().cpu().numpy()
    o_ref = np.zeros((N, H, dv))
    for n, p in enumerate(pages.tolist()):
        if p >= 0:
            ref[p, 1] = lam * ref[p, 1] + f64(k)[n][:, :, None] * f64(v)[n][:, None, :]
            o_ref[n] = np.einsum("hi,hij->hj", f64(q)[n], ref[p, 1])
    assert rel(f64(pool), ref) <= STATE_TOL
    assert torch.equal(pool[:, 0], before[:, 0])
    assert rel(f64(o), o_ref) <= TOL[dtype]
    if N > 1:
        assert (o[N // 2] == 0).all()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_decode_continues_a_prompt(dtype):
    """Prompt in one call, then token by token: the recurrence over all of them."""
    d = make(3, 80, 2, 64, 64, dtype, seed=15)
    T0 = 70
    o, s = G.gdn_lin_fwd(*(d[n][:, :T0].contiguous() for n in "qkv"), d["log_decay"], d["s0"])
    outs = [o]
    for t in range(T0, 80):
        o, s2 = G.gdn_lin_decode(*(d[n][:, t].contiguous() for n in "qkv"), d["log_decay"], s)
        assert s2 is s
        outs.append(o[:, None])
    o_ref, s_ref = lin.forward(d["q"], d["k"], d["v"], d["log_decay"], d["s0"])
    assert rel(f64(torch.cat(outs, 1)), o_ref) <= TOL[dtype]
    assert rel(f64(s), s_ref) <= STATE_TOL


def test_decode_without_a_state_and_out_of_place():
    d = make(3, 1, 2, 64, 64, "fp32", seed=16)
    q, k, v = (d[n][:, 0].contiguous() for n in "qkv")
    out = torch.full((3, 2, 64, 64), float("nan"), device="cuda")
    o, s = G.gdn_lin_decode(q, k, v, d["log_decay"], None, state_out=out)
    assert s is out
    assert rel(f64(s), f64(k)[..., :, None] * f64(v)[..., None, :]) <= STATE_TOL
    keep = d["s0"].clone()
    o, s = G.gdn_lin_decode(q, k, v, d["log_decay"], d["s0"], state_out=out)
    o2, s2 = G.gdn_lin_decode(q, k, v, d["log_decay"], keep)
    assert torch.equal(o, o2) and torch.equal(s, s2) and not torch.equal(keep, d["s0"])


def test_decode_reports_a_bad_page():
    d = make(2, 1, 1, 32, 32, "fp32")
    q, k, v = (d[n][:, 0].contiguous() for n in "qkv")
    pool = torch.randn(4, 1, 32, 32, device="cuda")
    before = pool.clone()
    for bad in (4, -2, 1 << 30):
        with pytest.raises(G.GdnError) as e:
            G.gdn_lin_decode(q, k, v, d["log_decay"], pool,
                             torch.tensor([bad, -1], dtype=torch.int32, device="cuda"), check=True)
        assert e.value.status == 7
    assert torch.equal(pool, before)
