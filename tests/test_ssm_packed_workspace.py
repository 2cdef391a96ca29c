"""The workspaces of packed calls of the scan: sized by the tokens of all sequences together,
not by num_seqs rows of that many."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import build as gbuild
from linear_attention_recurrence_gated_gb300 import gdn as G


@pytest.fixture(scope="module", autouse=True)
def built():
    gbuild.build()


# (sequences, tokens together, channels, states): training batches of ragged and equal lengths
PACKED = [(8, 65536, 1280, 16), (32, 140000, 1280, 16), (32, 131072, 2048, 16),
          (128, 131072, 2048, 16), (32, 131072, 1024, 64)]


@pytest.mark.parametrize("n,tokens,channels,states", PACKED)
def test_backward_size_is_that_of_the_tokens(n, tokens, channels, states):
    one = G.gdn_ssm_bwd_workspace_size(1, tokens, channels, states)
    packed = G.gdn_ssm_bwd_workspace_size(n, tokens, channels, states, packed=True)
    assert 0.9 * one <= packed <= 1.1 * one


def test_many_short_sequences():
    """16384 sequences of one token: what n rows of one token need, but for partial sums."""
    n = 16384
    rows = G.gdn_ssm_bwd_workspace_size(n, 1, 24, 8)
    assert G.gdn_ssm_bwd_workspace_size(n, n, 24, 8, packed=True) <= 1.1 * rows < 1 << 27


@pytest.mark.parametrize("n,tokens,channels,states", PACKED + [(46, 131072, 1280, 16), (5, 40, 64, 8)])
def test_packed_sizes_are_within_the_others(n, tokens, channels, states):
    for f in (G.gdn_ssm_workspace_size, G.gdn_ssm_bwd_workspace_size):
        assert 256 <= f(n, tokens, channels, states, packed=True) <= f(n, tokens, channels, states)


@pytest.mark.parametrize("sizes", [(0, 9, 64, 16, 1), (2, -1, 64, 16, 1), (2, 9, 0, 16, 1),
                                   (2, 9, 64, 24, 1), (2, 9, 64, 16, 0), (2, 9, 63, 16, 2)])
def test_sizes_that_no_call_has(sizes):
    for f in (G.gdn_ssm_workspace_size, G.gdn_ssm_bwd_workspace_size):
        assert f(*sizes) == f(*sizes, packed=True) == 0


class Reached(Exception):
    pass


class Device(torch.Tensor):
    is_cuda = property(lambda self: True)


def test_the_binding_asks_for_the_packed_size(monkeypatch):
    """(tensors that say they are on a CUDA device; the call ends where it would make the
    workspace)"""
    sizes = []

    def made(stream, like, given, size, status):
        sizes.append(size)
        raise Reached

    monkeypatch.setattr(G, "_workspace", made)
    zeros = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype).as_subclass(Device)  # noqa: E731
    n, T, D, S = 40, 2000, 64, 16
    x, b, A = zeros(1, T, D), zeros(1, T, 1, S), zeros(D, S, dtype=torch.float32)
    cu = zeros(n + 1, dtype=torch.int32)
    for packed in (True, False):
        with pytest.raises(Reached):
            G.gdn_ssm_fwd(x, x, A, b, b, None, cu if packed else None)
        with pytest.raises(Reached):
            G.gdn_ssm_bwd(x, x, A, b, b, x, None, cu if packed else None)
    assert sizes == [G.gdn_ssm_workspace_size(n, T, D, S, packed=True),
                     G.gdn_ssm_bwd_workspace_size(n, T, D, S, packed=True),
                     G.gdn_ssm_workspace_size(1, T, D, S), G.gdn_ssm_bwd_workspace_size(1, T, D, S)]
