"""What a token that is not finite reaches in linear attention: by the recurrence its own
and later outputs (earlier ones for the gradients that run backward in time), in the
columns that it has a bad value in, and nothing before it.  Bounds as in test_gpu_lin."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin
from parity import rel
from test_gpu_lin import STATE_TOL, TOL, f64, make

pytestmark = pytest.mark.gpu

FORMS = [("bf16", 64, 64), ("bf16", 128, 128), ("bf16", 128, 64), ("bf16", 64, 128), ("bf16", 32, 64),
         ("bf16", 96, 32), ("fp32", 64, 64), ("fp32", 128, 96), ("fp32", 32, 32)]
NAN, INF = float("nan"), float("inf")


def run(d, cu=None, **kw):
    cud = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    a = d["q"], d["k"], d["v"], d["log_decay"]
    o, s = G.gdn_lin_fwd(*a, d["s0"], cud, check=True, **kw)
    g = G.gdn_lin_bwd(*a, d["d_o"], d["s0"], cud, d["d_sT"], check=True, **kw)
    return {"o": o, "s": s, **g}


def reference(d, cu=None):
    o, s = lin.forward(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], cu)
    return {"o": o, "s": s, **lin.backward(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"],
                                           d["d_sT"], cu)}


def clean(got, want, tol, what):
    got = f64(got)
    assert np.isfinite(got).all(), what
    assert rel(got, want) <= tol, what


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
@pytest.mark.parametrize("T,j", [(200, 3), (200, 77), (200, 127), (200, 128), (200, 190), (128, 64),
                                 (64, 63), (9, 4)])
def test_one_bad_value(dtype, dk, dv, T, j):
    """A value of v, k, q or d_o at token j, head 1, in one column."""
    d = make(1, T, 2, dk, dv, dtype, seed=T + j)
    ref, tol = reference(d), TOL[dtype]
    # name: its column's gradients and outputs that it enters as a value, forward or
    # backward in time; those that it enters as a written row; as a read row
    roles = {"v": (("o", 1, None), ("dq", 1, True), ("dk", 0, True)),
             "k": (("dq", 1, None), ("o", 1, True), ("dv", 0, True)),
             "q": (("dk", -1, None), ("dv", -1, True), ("o", 0, True)),
             "d_o": (("dv", -1, None), ("dk", -1, True), ("dq", 0, True))}
    untouched = {"v": ("dv", "dh0"), "k": ("dk", "dh0"), "q": ("dq", "s"), "d_o": ("o", "s")}
    for name, bad in (("v", NAN), ("v", -INF), ("k", INF), ("q", NAN), ("d_o", INF)):
        x = {n: None if t is None else t.clone() for n, t in d.items()}
        col = x[name].shape[3] - 5
        x[name][0, j, 1, col] = bad
        out = run(x)
        for n in untouched[name]:
            clean(out[n], ref[n], STATE_TOL if n in ("s", "dh0") else tol, (name, n))
        for n, way, whole in roles[name]:
            got, want = out[n], ref[n]
            clean(got[:, :, 0], want[:, :, 0], tol, (name, n, "the other head"))
            before = slice(0, j) if way == 1 else slice(j + 1, T)
            if way == 0:   # its own row alone
                keep = [t for t in range(T) if t != j]
                clean(got[:, keep], want[:, keep], tol, (name, n))
                assert not torch.isfinite(got[0, j, 1]).any()
                continue
            if got[:, before].numel():
                clean(got[:, before], want[:, before], tol, (name, n, "before"))
            if got[:, before, 1].numel():   # (its column by itself: few values, one rounding each)
                clean(got[:, before, 1, col] if not whole else got[:, before, 1],
                      want[:, before, 1, col] if not whole else want[:, before, 1], 2 * tol, (name, n))
            after = slice(j, T) if way == 1 else slice(0, j + 1)
            if whole:
                assert not torch.isfinite(got[:, after, 1]).any(), (name, n)
            else:
                others = [c for c in range(got.shape[3]) if c != col]
                clean(got[:, after, 1][..., others], want[:, after, 1][..., others], tol, (name, n))
                assert not torch.isfinite(got[:, after, 1, col]).any(), (name, n)
        # the states: a column of v or d_o, a row of k or q
        state, at = ("s", name) if name in "vk" else ("dh0", {"d_o": "v", "q": "k"}[name])
        got, want = out[state], ref[state]
        others = [c for c in range(x[name].shape[3]) if c != col]
        axis = 3 if at == "v" else 2
        clean(got[:, 0], want[:, 0], STATE_TOL, (name, state))
        clean(got[:, 1:].index_select(axis, torch.tensor(others, device="cuda")),
              np.take(want[:, 1:], others, axis), STATE_TOL, (name, state))
        assert not torch.isfinite(got[:, 1].select(axis - 1, col)).any()


@pytest.mark.parametrize("dtype,dk,dv", FORMS)
def test_a_padded_tail_of_garbage(dtype, dk, dv):
    """Sequences of 300 tokens of which 1, 100, 200 and 299 are there and the rest is
    whatever lies in memory: the outputs of those that are there are the sequence's own."""
    lens, T = (1, 100, 200, 299), 300
    d = make(len(lens), T, 2, dk, dv, dtype, seed=5)
    ref = reference(d)
    bad = torch.tensor([NAN, INF, -INF, 3e38], device="cuda")
    for n, L in enumerate(lens):
        for name in "qkv":
            t = d[name][n, L:]
            t.copy_(bad[torch.arange(t.numel(), device="cuda") % 4].view(t.shape))
    o, _ = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    for n, L in enumerate(lens):
        clean(o[n, :L], ref["o"][n, :L], TOL[dtype], L)


@pytest.mark.parametrize("dtype,dk,dv,T", [("bf16", 64, 64, 5000), ("bf16", 128, 128, 4100),
                                           ("fp32", 64, 64, 2100), ("fp32", 32, 32, 2048)])
def test_long_sequences(dtype, dk, dv, T):
    """Cut along time: two bad tokens in different segments and columns, and the columns
    between them."""
    d = make(1, T, 1, dk, dv, dtype, seed=6)
    ref, tol = reference(d), TOL[dtype]
    j1, j2, c1, c2 = T // 3 + 1, T - 70, 7, dv - 1
    d["v"][0, j1, 0, c1], d["v"][0, j2, 0, c2] = INF, NAN
    d["d_o"][0, j1, 0, c2], d["d_o"][0, j2, 0, c1] = NAN, INF
    out = run(d)
    for n, (a, ca), (b, cb), way in (("o", (j1, c1), (j2, c2), 1), ("dv", (j2, c1), (j1, c2), -1)):
        got, want = out[n][0, :, 0], ref[n][0, :, 0]
        others = [c for c in range(dv) if c not in (c1, c2)]
        clean(got[:, others], want[:, others], tol, n)
        for j, c in ((a, ca), (b, cb)):
            before, after = (slice(0, j), slice(j, T)) if way == 1 else (slice(j + 1, T), slice(0, j + 1))
            clean(got[before, c], want[before, c], 2 * tol, (n, c))
            assert not torch.isfinite(got[after, c]).any(), (n, c)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_packed_sequences(dtype, dk, dv):
    """One bad token in the middle of a sequence's last tile: its neighbours are whole."""
    cu = [0, 130, 131, 300, 470]
    d = make(1, cu[-1], 3, dk, dv, dtype, seed=8, N=4)
    ref, tol = reference(d, cu), TOL[dtype]
    j, col = 200, 11
    d["v"][0, j, 2, col] = NAN
    d["d_o"][0, j, 2, col] = INF
    out = run(d, cu)
    for n, bad in (("o", slice(j, 300)), ("dv", slice(131, j + 1))):
        got = out[n].clone()
        assert not torch.isfinite(got[0, bad, 2, col]).any()
        got[0, bad, 2, col] = torch.tensor(ref[n][0, bad, 2, col], device="cuda").to(got.dtype)
        clean(got, ref[n], tol, n)


def test_a_state_that_is_not_finite():
    """A bad first state stays in its column, over many chunks; a bad query in its row."""
    for dtype, D in (("bf16", 64), ("bf16", 128), ("fp32", 64)):
        d = make(2, 700, 1, D, D, dtype, seed=9)
        ref = reference(d)
        d["s0"][1, 0, 3, 9] = NAN
        d["q"][0, 400] = INF
        o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
        keep = [t for t in range(700) if t != 400]
        clean(o[0, keep], ref["o"][0, keep], TOL[dtype], dtype)
        others = [c for c in range(D) if c != 9]
        clean(o[1][..., others], ref["o"][1][..., others], TOL[dtype], dtype)
        assert not torch.isfinite(o[1, :, 0, 9]).any() and not torch.isfinite(o[0, 400]).any()
        clean(s[0], ref["s"][0], STATE_TOL, dtype)
