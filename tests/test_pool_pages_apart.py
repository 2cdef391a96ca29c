"""Pools whose pages lie on top of one another (an expanded tensor, stride 0) are refused by
every call on pages: the library takes a page stride of 0 for densely packed pages, behind the
tensor's memory.  The tensors say that they are on a CUDA device; nothing reaches the library."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

BF, I32 = torch.bfloat16, torch.int32


class Reached(Exception):
    pass


class Device(torch.Tensor):
    is_cuda = property(lambda self: True)


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def entry(name):
        def call(*args):
            raise Reached(name)
        return call
    monkeypatch.setattr(G, "_call", entry)
    monkeypatch.setattr(G, "_raw_stream", lambda stream, device: 0)


def zeros(*s, dtype=torch.float32):
    return torch.zeros(*s, dtype=dtype).as_subclass(Device)


z = lambda *s: zeros(*s, dtype=BF)  # noqa: E731
PAGES = zeros(3, dtype=I32)
CALLS = {
    "gdn_ssm_step": (lambda pool, **kw: G.gdn_ssm_step(
        z(3, 16), z(3, 16), zeros(16, 8), z(3, 1, 8), z(3, 1, 8), pool, PAGES, **kw), (16, 8), torch.float32),
    "gdn_conv_step": (lambda pool, **kw: G.gdn_conv_step(z(3, 16), zeros(16, 4), pool, None, PAGES, **kw),
                      (3, 16), BF),
    "gdn_lin_decode": (lambda pool, **kw: G.gdn_lin_decode(
        z(3, 2, 32), z(3, 2, 32), z(3, 2, 32), zeros(2), pool, PAGES, **kw), (2, 32, 32), torch.float32),
}


@pytest.mark.parametrize("name", CALLS)
def test_expanded_pools(name):
    call, page, dtype = CALLS[name]
    for pool in (zeros(5, *page, dtype=dtype), zeros(5, 2, *page, dtype=dtype)[:, 1],
                 zeros(1, *page, dtype=dtype), zeros(1, 2, *page, dtype=dtype)[:, 1]):
        with pytest.raises(Reached):
            call(pool)
    one = zeros(1, *page, dtype=dtype)
    for pool in (one.expand(5, *page), one[0].expand(5, *page)):
        with pytest.raises(ValueError, match="contiguous pages at one stride"):
            call(pool)
    if name != "gdn_conv_step":   # ... also of the states that are only read
        with pytest.raises(ValueError, match="contiguous pages at one stride"):
            call(one.expand(5, *page), state_out=zeros(5, *page))
        with pytest.raises(ValueError, match="contiguous pages at one stride"):
            call(zeros(5, *page), state_out=one.expand(5, *page))
        with pytest.raises(ValueError, match="contiguous pages at one stride"):
            call(None, state_out=one.expand(5, *page))
