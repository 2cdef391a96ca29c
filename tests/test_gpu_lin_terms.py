"""The returned state of a tensor-core scan whose tokens all lie some way before the end.

Bound.  Weighted values enter the state as bf16 terms; what the terms leave out is at
most 2^-24 of what a token wrote, once it has decayed to the end of the sequence (the
decayed value's own fp32 rounding is far below that).  Every token writes to rows and
columns of its own here, so each element of the state is one token's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("reach", [2.0, 4.5, 5.2, 6.0, 7.0, 7.9, 9.0, 12.0])
def test_tokens_before_the_end(D, reach):
    """`reach`: halvings of a token's contribution over the tokens that follow its tile."""
    T, C = 1024, 128
    tile = 2
    rest = T - (tile + 1) * C
    rate = -reach * np.log(2.0) / rest
    g = torch.Generator().manual_seed(D)
    for back in (False, True):
        x = {n: torch.zeros(1, T, 1, D).bfloat16() for n in "abc"}
        lam = np.exp(np.float64(np.float32(rate)))
        want, wrote = np.zeros((D, D)), np.zeros((D, D))
        for i in range(D):
            j = i % C
            t = T - 1 - (tile * C + j) if back else tile * C + j
            b = torch.randn((), generator=g).bfloat16()
            c = torch.randn(D, generator=g).bfloat16()
            x["b"][0, t, 0, i], x["c"][0, t, 0] = b, c
            n = t + 1 if back else T - 1 - t
            wrote[i] = float(b) * c.double().numpy()
            want[i] = lam ** n * wrote[i]
        ld = torch.tensor([rate], dtype=torch.float32, device="cuda")
        a, b, c = (x[n].cuda() for n in "abc")
        if back:   # the gradient of the first state: rows q, values d_o
            got = G.gdn_lin_bwd(b, a, c, ld, c, check=True)["dh0"]
        else:
            got = G.gdn_lin_fwd(a, b, c, ld, check=True)[1]
        err = np.abs(got[0, 0].double().cpu().numpy() - want)
        assert (err <= 2.0 ** -24 * np.abs(wrote).max()).all(), (back, np.max(err / np.abs(wrote).max()))
