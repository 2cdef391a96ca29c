"""dweight and dbias over many rows whose terms are all the same, where the roundings of
a long plain sum go the same way.

Bound.  A sum of terms of one sign is off by at most 2^-24 of itself for each addition
that a term passes through.  A thread adds up to 128 rows, and the results of these
blocks; a CTA its rows of threads (64 or fewer at these sizes), and the call its CTAs by
up to 64 rows of threads: fewer than 512 additions, 2^-15.  Adding one
constant again and again is off by the same amount each time while the sum stays within
a binade, so that the last binade of a stage (half its additions) decides, with an error
that is a quarter of the largest in the mean: 2^-17 = 7.6e-6, and twice that is asked
for.  A term itself, silu or xh, is off by a few 2^-24: 2^-21 more."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -16 + 2.0 ** -21


# a group in a warp's registers; groups wider than that; samples of two rows and, many of
# them, of more than a thread sums at once; slabs with 16-byte vectors and without; the
# sums of many slabs
@pytest.mark.parametrize("N,S,C,groups", [
    (1 << 19, 1, 4096, 32), (1 << 21, 1, 516, 1), (1 << 21, 2, 64, 4), (1 << 16, 11000, 3, 1),
    (1, 1 << 22, 512, 8), (1, 1 << 25, 20, 2), (65535, 16, 1024, 8)])
@pytest.mark.parametrize("z", [0.7, 1.3])
def test_terms_that_are_the_same(N, S, C, groups, z):
    """x is the same in every row, so a channel's xh is too; with one d_y and one gate a
    channel's sum is N S times a number."""
    row = torch.randn(C, generator=torch.Generator().manual_seed(C)).bfloat16().float()
    x = row.cuda().expand(N, S, C).contiguous()
    d_y, gate = torch.ones_like(x), torch.full_like(x, z)
    v = row.double().numpy().reshape(groups, -1)
    m, rs = v.mean(1), 1 / np.sqrt(v.var(1) + 1e-5)
    xh = ((v - m[:, None]) * rs[:, None]).reshape(-1)
    mean, rstd = (torch.tensor(t).float().cuda().expand(N, groups).contiguous() for t in (m, rs))
    gr = G.gdn_group_norm_bwd(x, None, None, groups, mean, rstd, d_y, gate=gate)
    z = float(gate[0, 0, 0])
    du = z / (1 + np.exp(-z))
    for name, want in (("dbias", np.full(C, du)), ("dweight", du * xh)):
        got = gr[name].double().cpu().numpy() / (N * S)
        big = np.abs(want) > 0.5 * np.abs(want).max()
        assert np.abs(got / want - 1)[big].max() <= BOUND, name
        assert np.abs(got - want).max() <= BOUND * np.abs(want).max(), name
