"""The Python binding of the scan, the convolution and the q/k norm refuses what does not
fit before anything reaches the library.  The tensors say that they are on a CUDA device,
and the library's entry points are replaced: a call that passes every check ends in
``Reached``."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

BF = torch.bfloat16


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


def plain(t):
    return t.as_subclass(torch.Tensor)


def refused(call, *kinds):
    with pytest.raises(kinds or (ValueError, TypeError)) as e:
        call()
    return str(e.value)


def reaches(call):
    with pytest.raises(Reached):
        call()


def ssm(dtype=BF, B=2, T=4, D=16, S=8, G_=1):
    z = lambda *s: zeros(*s, dtype=dtype)  # noqa: E731
    return dict(x=z(B, T, D), dt=z(B, T, D), A_log=zeros(D, S), b=z(B, T, G_, S), c=z(B, T, G_, S))


def test_ssm_fwd_and_bwd():
    a = ssm()
    d_y = zeros(2, 4, 16, dtype=BF)
    fwd = lambda **kw: G.gdn_ssm_fwd(**{**a, **kw})  # noqa: E731
    bwd = lambda **kw: G.gdn_ssm_bwd(**{**a, "d_y": d_y, **kw})  # noqa: E731
    for call in (fwd, bwd):
        reaches(lambda: call())
        reaches(lambda: call(gate=d_y, D_skip=zeros(16), dt_bias=zeros(16), initial_state=zeros(2, 16, 8)))
        assert "dt" in refused(lambda: call(dt=a["dt"].float()), TypeError)
        refused(lambda: call(x=a["x"].half()), TypeError)
        refused(lambda: call(dt=a["dt"][:, :3]), ValueError)
        refused(lambda: call(x=a["x"][0]), ValueError)
        refused(lambda: call(b=a["b"][:, :3], c=a["c"][:, :3]), ValueError)
        refused(lambda: call(c=zeros(2, 4, 2, 8, dtype=BF)), ValueError)
        refused(lambda: call(A_log=zeros(16, 16)), ValueError)
        refused(lambda: call(A_log=zeros(16, 8, dtype=torch.float64)), ValueError)
        refused(lambda: call(D_skip=zeros(8)), ValueError)
        refused(lambda: call(gate=zeros(2, 4, 8, dtype=BF)), ValueError)
        refused(lambda: call(initial_state=zeros(1, 16, 8)), ValueError)
        refused(lambda: call(initial_state=zeros(2, 8, 16).transpose(1, 2)), ValueError)
        refused(lambda: call(cu_seqlens=zeros(3, dtype=torch.int64)), TypeError)
        refused(lambda: call(cu_seqlens=zeros(1, dtype=torch.int32)), ValueError)
        assert "CUDA" in refused(lambda: call(c=plain(a["c"])), ValueError)
        assert "CUDA" in refused(lambda: call(dt_bias=torch.zeros(16)), ValueError)
        # slices of a projection are taken, other strides refused
        wide = zeros(2, 4, 48, dtype=BF)
        reaches(lambda: call(x=wide[..., 16:32]))
        refused(lambda: call(x=zeros(2, 4, 33, dtype=BF)[..., :16]), ValueError)
        refused(lambda: call(x=zeros(2, 16, 4, dtype=BF).transpose(1, 2)), ValueError)
        refused(lambda: call(x=zeros(2, 8, 16, dtype=BF)[:, ::2][:, :4].transpose(0, 1).contiguous()
                             .transpose(0, 1)), ValueError)
    refused(lambda: fwd(y=zeros(2, 4, 16)), ValueError)
    refused(lambda: fwd(final_state=zeros(2, 16, 16)), ValueError)
    refused(lambda: bwd(d_y=d_y.float()), ValueError)
    refused(lambda: bwd(d_final_state=zeros(3, 16, 8)), ValueError)
    refused(lambda: bwd(grads=dict(dx=d_y)), ValueError)
    refused(lambda: bwd(grads=dict(dz=d_y)), ValueError)
    refused(lambda: bwd(grads=dict(dx=d_y, ddt=d_y, db=a["b"], dc=a["c"], dA_log=zeros(16))), ValueError)


def test_ssm_step():
    z = lambda *s: zeros(*s, dtype=BF)  # noqa: E731
    a = dict(x=z(3, 16), dt=z(3, 16), A_log=zeros(16, 8), b=z(3, 1, 8), c=z(3, 1, 8), state=zeros(5, 16, 8))
    call = lambda **kw: G.gdn_ssm_step(**{**a, **kw})  # noqa: E731
    reaches(lambda: call())
    reaches(lambda: call(state=zeros(5, 2, 16, 8)[:, 1], pages=zeros(3, dtype=torch.int32)))
    refused(lambda: call(state=zeros(5, 8, 16).transpose(1, 2)), ValueError)
    refused(lambda: call(state=zeros(5, 16, 16)), ValueError)
    refused(lambda: call(state=zeros(5, 16, 8, dtype=BF)), ValueError)
    refused(lambda: call(state=None), ValueError)
    refused(lambda: call(state=zeros(5, 2, 16, 8)[:, 1], state_out=zeros(5, 16, 8)), ValueError)
    refused(lambda: call(state=plain(a["state"])), ValueError)
    refused(lambda: call(pages=zeros(2, dtype=torch.int32)), ValueError, TypeError)
    refused(lambda: call(x=z(3, 32)[:, :16]), ValueError)
    refused(lambda: call(b=z(2, 1, 8)), ValueError)
    refused(lambda: call(x=z(3, 1, 16)), ValueError)
    refused(lambda: call(dt=zeros(3, 16)), ValueError)


def test_conv():
    z = lambda *s: zeros(*s, dtype=BF)  # noqa: E731
    a = dict(x=z(2, 5, 16), w=zeros(16, 4))
    fwd = lambda **kw: G.gdn_conv_fwd(**{**a, **kw})  # noqa: E731
    bwd = lambda **kw: G.gdn_conv_bwd(**{**a, "d_y": z(2, 5, 16), **kw})  # noqa: E731
    for call in (fwd, bwd):
        reaches(lambda: call())
        reaches(lambda: call(bias=zeros(16), x_prev=z(2, 3, 16)))
        refused(lambda: call(x=z(5, 16)), ValueError)
        refused(lambda: call(x=z(2, 5, 16).half()), TypeError)
        refused(lambda: call(w=zeros(16, 4, dtype=BF)), ValueError)
        refused(lambda: call(w=zeros(8, 4)), ValueError)
        refused(lambda: call(bias=zeros(8)), ValueError)
        refused(lambda: call(x_prev=z(2, 4, 16)), ValueError)
        refused(lambda: call(x_prev=zeros(2, 3, 16)), ValueError)
        refused(lambda: call(cu_seqlens=zeros(3, dtype=torch.int64)), TypeError)
        refused(lambda: call(x=plain(a["x"])), ValueError)
    refused(lambda: fwd(y=zeros(2, 5, 16)), ValueError)
    refused(lambda: fwd(x_tail=z(1, 3, 16)), ValueError)
    refused(lambda: bwd(d_y=z(2, 4, 16)), ValueError)
    refused(lambda: bwd(d_x_tail=z(2, 2, 16)), ValueError)
    refused(lambda: bwd(grads=dict(dw=zeros(16, 4))), ValueError)
    step = lambda **kw: G.gdn_conv_step(**{**dict(x=z(3, 16), w=zeros(16, 4), state=z(5, 3, 16)), **kw})  # noqa: E731
    reaches(lambda: step())
    reaches(lambda: step(state=z(5, 2, 3, 16)[:, 0]))
    refused(lambda: step(state=z(5, 4, 16)), ValueError)
    refused(lambda: step(state=zeros(5, 3, 16)), ValueError)
    refused(lambda: step(x=z(3, 1, 16)), ValueError)
    refused(lambda: step(bias=zeros(4)), ValueError)


def test_qk_norm():
    z = lambda *s: zeros(*s, dtype=BF)  # noqa: E731
    a = dict(q=z(2, 5, 4, 16), k=z(2, 5, 2, 16))
    fwd = lambda **kw: G.gdn_qk_norm(**{**a, **kw})  # noqa: E731
    bwd = lambda **kw: G.gdn_qk_norm_bwd(**{**a, "d_q_out": a["q"], "d_k_out": a["k"], **kw})  # noqa: E731
    for call in (fwd, bwd):
        reaches(lambda: call())
        reaches(lambda: call(inv_freq=zeros(8), positions=zeros(2, 5, dtype=torch.int32)))
        wide = z(2, 5, 8 * 16)
        reaches(lambda: call(q=wide[..., :64].view(2, 5, 4, 16), k=wide[..., 64:96].view(2, 5, 2, 16)))
        refused(lambda: call(k=z(2, 4, 2, 16)), ValueError)
        refused(lambda: call(k=z(2, 5, 2, 8)), ValueError)
        refused(lambda: call(k=zeros(2, 5, 2, 16)), TypeError)
        refused(lambda: call(q=z(2, 5, 64)), ValueError)
        refused(lambda: call(q_weight=zeros(8)), ValueError)
        refused(lambda: call(k_weight=z(16)), ValueError)
        refused(lambda: call(inv_freq=zeros(9)), ValueError)
        refused(lambda: call(inv_freq=zeros(8, dtype=torch.float64)), ValueError)
        refused(lambda: call(positions=zeros(2, 5, dtype=torch.int32)), ValueError)
        refused(lambda: call(inv_freq=zeros(8), positions=zeros(2, 5, dtype=torch.int64)), TypeError)
        refused(lambda: call(inv_freq=zeros(8), positions=zeros(5, dtype=torch.int32)), ValueError, TypeError)
        refused(lambda: call(q=a["q"].transpose(1, 2).contiguous().transpose(1, 2)), ValueError)
        refused(lambda: call(q=plain(a["q"])), ValueError)
    refused(lambda: fwd(q_out=zeros(2, 5, 4, 16)), ValueError)
    refused(lambda: bwd(d_q_out=z(2, 5, 4, 32)[..., :16]), ValueError)
    refused(lambda: bwd(grads=dict(dq=a["q"])), ValueError)
