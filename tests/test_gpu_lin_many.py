"""Linear attention on the tensor cores over more (sequence, head, value tile)s
than the GPU runs at a time, and over many chunks.  Bounds as in test_gpu_lin (the
arithmetic is the same); decays from none to immediate, since the number of bf16
terms of a chunk's state increment follows them."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G
from oracle import lin
from parity import rel
from test_gpu_lin import STATE_TOL, TOL, check_bwd, check_fwd, f64, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(10, 300, 16, 64, 64), (5, 650, 16, 128, 128),
                                   (11, 129, 5, 64, 192), (7, 1, 23, 64, 64),
                                   (3, 384, 30, 128, 128)])
def test_dense(shape):
    """Whole and ragged tiles, one token; one to three value tiles."""
    d = make(*shape, "bf16", seed=sum(shape))
    check_fwd(d, "bf16")
    check_bwd(d, "bf16")


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (64, 128)])
@pytest.mark.parametrize("init", [False, True])
def test_packed(dk, dv, init):
    """Empty sequences first, last and in between, single tokens, whole chunks and
    one sequence longer than the others together."""
    lens = [0, 130, 1, 1400, 0, 257, 128, 0, 5, 64, 300, 0]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(1, cu[-1], 16, dk, dv, "bf16", seed=dk + dv, N=len(lens), init=init)
    _, s = check_fwd(d, "bf16", cu)
    g = check_bwd(d, "bf16", cu)
    for n in (0, 4, 7, 11):
        assert torch.equal(s[n], d["s0"][n] if init else torch.zeros_like(s[n]))
        assert torch.equal(g["dh0"][n], d["d_sT"][n] if init else torch.zeros_like(s[n]))


def test_many_packed_sequences():
    lens = [(37 * n) % 200 for n in range(150)]
    cu = np.concatenate([[0], np.cumsum(lens)]).tolist()
    d = make(1, cu[-1], 3, 64, 64, "bf16", seed=3, N=len(lens))
    check_fwd(d, "bf16", cu)
    check_bwd(d, "bf16", cu)


@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("shape", [(1, 1100, 3), (2, 900, 80)])
@pytest.mark.parametrize("rate", [0.0, -1e-3, -6e-3, -0.02, -0.5, float("-inf")])
def test_decays_over_many_chunks(dk, shape, rate):
    """Few units and many: where the third term begins (never, at the last
    chunks, from the first) and where the output waits for its store."""
    B, T, H = shape
    decay = torch.full((H,), rate)
    d = make(B, T, H, dk, dk, "bf16", seed=4, decay=decay)
    o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    g = G.gdn_lin_bwd(d["q"], d["k"], d["v"], d["log_decay"], d["d_o"], d["s0"], None, d["d_sT"],
                      check=True)
    for h in (0, H - 1):
        one = lambda t, axis: t.narrow(axis, h, 1)  # noqa: E731
        q, k, v, d_o = (one(d[n], 2) for n in ("q", "k", "v", "d_o"))
        s0, d_sT, ld = one(d["s0"], 1), one(d["d_sT"], 1), d["log_decay"][h:h + 1]
        o_ref, s_ref = lin.forward(q, k, v, ld, s0)
        ref = lin.backward(q, k, v, ld, d_o, s0, d_sT)
        assert rel(f64(one(o, 2)), o_ref) <= TOL["bf16"]
        assert rel(f64(one(s, 1)), s_ref) <= STATE_TOL
        for n in ("dq", "dk", "dv"):
            assert rel(f64(one(g[n], 2)), ref[n]) <= TOL["bf16"], n
        assert rel(f64(one(g["dh0"], 1)), ref["dh0"]) <= STATE_TOL


def test_the_smallest_workspace():
    """256 bytes: the same values up to rounding; and call after call the same bits."""
    d = make(10, 500, 16, 64, 64, "bf16", seed=6)
    args = (d["q"], d["k"], d["v"], d["log_decay"], d["s0"])
    o, s = G.gdn_lin_fwd(*args, check=True)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    o1, s1 = G.gdn_lin_fwd(*args, workspace=small, check=True)
    assert rel(f64(o1), f64(o)) <= TOL["bf16"] and rel(f64(s1), f64(s)) <= STATE_TOL
    for _ in range(5):
        o2, s2 = G.gdn_lin_fwd(*args, check=True)
        assert torch.equal(o, o2) and torch.equal(s, s2)


def test_bad_offsets_are_reported():
    d = make(1, 400, 60, 64, 64, "bf16", N=3)
    for cu in ([0, 100, 90, 400], [1, 100, 200, 400], [0, 100, 200, 399]):
        cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
        with pytest.raises(G.GdnError) as e:
            G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], cud, check=True)
        assert e.value.status == 6


@pytest.mark.parametrize("dtype,shape", [("bf16", (1, 6000, 4, 64, 64)), ("bf16", (2, 4100, 3, 128, 128)),
                                         ("fp32", (1, 3000, 4, 64, 64)), ("fp32", (2, 2000, 1, 32, 96)),
                                         ("bf16", (1, 3000, 2, 32, 64))])
def test_long_sequences_update_their_state_in_place(dtype, shape):
    """Cut along time, with the last state written over the first."""
    d = make(*shape, dtype, seed=7)
    want_o, want_s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], d["s0"], check=True)
    for _ in range(3):
        state = d["s0"].clone()
        o, s = G.gdn_lin_fwd(d["q"], d["k"], d["v"], d["log_decay"], state, final_state=state,
                             check=True)
        assert s is state and torch.equal(o, want_o) and torch.equal(s, want_s)
    cu = torch.tensor([0, 0, shape[0] * shape[1]], dtype=torch.int32, device="cuda")
    flat = [d[n].reshape(1, -1, *d[n].shape[2:]) for n in "qkv"]
    state = torch.randn(2, *d["s0"].shape[1:], device="cuda")
    want_o, want_s = G.gdn_lin_fwd(*flat, d["log_decay"], state, cu, check=True)
    o, s = G.gdn_lin_fwd(*flat, d["log_decay"], state, cu, final_state=state, check=True)
    assert torch.equal(o, want_o) and torch.equal(s, want_s)
