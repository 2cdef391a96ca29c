"""The oracle's scan of sequences side by side (written-out adjoint) against the one token by
token (autograd)."""
import pytest
import torch

import oracle.ssm as O

NAMES = dict(x="dx", dt="ddt", A_log="dA_log", b="db", c="dc", h0="dh0", D_skip="dD_skip",
             gate="dgate", dt_bias="ddt_bias")


def inputs(N, T, D, S, G, gate=True, rest=True):
    g = torch.Generator().manual_seed(T + D)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(x=r(N, T, D), dt=r(N, T, D), A_log=0.3 * r(D, S), b=r(N, T, G, S), c=r(N, T, G, S),
                h0=r(N, D, S) if rest else None, D_skip=r(D) if rest else None,
                gate=r(N, T, D) if gate else None, dt_bias=r(D) - 1 if rest else None), \
        r(N, T, D), r(N, D, S)


def near(a, b):
    assert float((a - b).norm()) <= 1e-12 * float(b.norm()) + 1e-30


@pytest.mark.parametrize("gate,rest,softplus", [(True, True, True), (False, False, False),
                                                (True, False, True), (False, True, False)])
def test_as_autograd(gate, rest, softplus):
    i, d_y, d_last = inputs(3, 7, 8, 4, 2, gate, rest)
    if not softplus:
        i["dt"] = i["dt"].abs()
    y, last, g = O.scan_grads(i, d_y, d_last, softplus=softplus)
    how = dict(dt_softplus=softplus)
    ry, rl = O.scan(**{**i, "h0": i["h0"]}, cu=None, **how)
    near(y, ry)
    near(last, rl)
    for n, t in O.grads(O.scan, i, (d_y, d_last), **how).items():
        near(g[NAMES[n]], t)


def test_ragged_rows():
    lens = [5, 1, 0, 7]
    i, d_y, d_last = inputs(4, 7, 8, 4, 1)
    mask = (torch.arange(7) < torch.tensor(lens)[:, None]).double()
    y, last, g = O.scan_grads(i, d_y, d_last, mask)
    cu = [sum(lens[:n]) for n in range(5)]
    pack = lambda t: torch.cat([t[n, :k] for n, k in enumerate(lens)])[None]  # noqa: E731
    rows = ("x", "dt", "b", "c", "gate")
    j = {n: pack(t) if n in rows else t for n, t in i.items()}
    ry, rl = O.scan(**j, cu=cu, dt_softplus=True)
    near(pack(y), ry)
    near(last, rl)
    for n, t in O.grads(O.scan, j, (pack(d_y), d_last), cu=cu, dt_softplus=True).items():
        if n == "D_skip":   # (rows that are no tokens have d_y = 0)
            near(g["dD_skip"], t)
        else:
            near(pack(g[NAMES[n]]) if n in rows else g[NAMES[n]], t)
