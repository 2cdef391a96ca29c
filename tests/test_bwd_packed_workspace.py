"""The workspace of a packed gdn_bwd call: sized by the tokens of all sequences together, not by
num_seqs rows of that many (host checks; fake device addresses, never dereferenced)."""
import ctypes

import pytest

from linear_attention_recurrence_gated_gb300 import build as gbuild
from linear_attention_recurrence_gated_gb300 import gdn as G

vp = ctypes.c_void_p


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


@pytest.mark.parametrize("n,tokens,heads,dk,dv", [(32, 140000, 16, 64, 64), (32, 140000, 16, 128, 128),
                                                  (128, 131072, 16, 128, 128), (128, 131072, 16, 64, 64)])
def test_size_is_that_of_the_tokens(n, tokens, heads, dk, dv):
    one = G.gdn_bwd_workspace_size(1, tokens, heads, dk, dv)
    scratch = n * 2 * heads * (dv // 32) * 8 * (dk // 32 * 4 * 256) * 4   # a few states a CTA
    assert G.gdn_bwd_workspace_size(n, tokens, heads, dk, dv, packed=True) <= 1.1 * one + scratch


@pytest.mark.parametrize("n,tokens", [(1, 1), (3, 40), (5, 1000), (100, 100), (7, 64 * 7)])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 96)])
def test_within_the_dense_size(n, tokens, dk, dv):
    packed = G.gdn_bwd_workspace_size(n, tokens, 4, dk, dv, packed=True)
    assert 256 < packed <= G.gdn_bwd_workspace_size(n, tokens, 4, dk, dv)
    # a call asks for what it is told to bring: one byte less is refused, nothing is launched
    at = lambda i: vp((1 << 40) + i * (1 << 34))  # noqa: E731
    f = G.lib().gdn_bwd
    args = [at(i) for i in range(15)] + [1, tokens, 4, dk, dv, n, G.GDN_F32, 0, at(20)]
    assert f(*args, packed - 1, vp(0)) == 3
    args[6] = None   # dense rows: the dense size
    args[15] = n
    dense = G.gdn_bwd_workspace_size(n, tokens, 4, dk, dv)
    assert f(*args, dense - 1, vp(0)) == 3


def test_sizes_that_no_call_has():
    for sizes in ((0, 9, 2, 64, 64), (2, -1, 2, 64, 64), (2, 9, 0, 64, 64), (2, 9, 2, 64, 40)):
        assert G.gdn_bwd_workspace_size(*sizes) == G.gdn_bwd_workspace_size(*sizes, packed=True) == 0
