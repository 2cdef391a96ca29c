"""The Python binding of linear attention, group norm and state pages refuses
what does not fit before anything reaches the library.  The tensors say that they
are on a CUDA device, and the library's entry points are replaced: a call that
passes every check ends in ``Reached``."""
from __future__ import annotations

import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G


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


def qkv(dtype=torch.float32, B=1, T=4, H=2, dk=32, dv=32):
    z = lambda d: zeros(B, T, H, d, dtype=dtype)  # noqa: E731
    return z(dk), z(dk), z(dv), zeros(H)


def refused(call, *kinds):
    with pytest.raises(kinds or (ValueError, TypeError)) as e:
        call()
    return str(e.value)


def test_lin_fwd_and_bwd():
    q, k, v, ld = qkv()
    both = (lambda *a, **kw: G.gdn_lin_fwd(*a, **kw),
            lambda q, k, v, ld, *a, **kw: G.gdn_lin_bwd(q, k, v, ld, v, *a, **kw))
    for call in both:
        refused(lambda: call(q, k[:, :3], v, ld))
        refused(lambda: call(q, k, v[..., :1, :], ld))
        refused(lambda: call(q, k.double(), v, ld), TypeError, ValueError)
        refused(lambda: call(q.half(), k.half(), v.half(), ld), TypeError, ValueError)
        refused(lambda: call(q, k, v, ld.double()))
        refused(lambda: call(q, k, v, ld[:1]))
        refused(lambda: call(q[0], k[0], v[0], ld))
        refused(lambda: call(q, k, v, ld, zeros(1, 2, 32, 33)))
        refused(lambda: call(q, k, v[..., ::2], ld))
        refused(lambda: call(q[..., :16].transpose(1, 2), k[..., :16].transpose(1, 2), v, ld))
        assert "CUDA" in refused(lambda: call(q, plain(k), v, ld))
        assert "CUDA" in refused(lambda: call(q, k, v, plain(ld)))
        with pytest.raises(Reached):
            call(q, k, v, ld)


def test_lin_decode():
    q, k, v, ld = qkv(T=1)
    q, k, v = (t[:, 0] for t in (q, k, v))
    state = zeros(1, 2, 32, 32)
    assert "state" in refused(lambda: G.gdn_lin_decode(q, k, v, ld, None))
    refused(lambda: G.gdn_lin_decode(q, k[:, :1], v, ld, state))
    refused(lambda: G.gdn_lin_decode(q, k, v.double(), ld, state), TypeError, ValueError)
    refused(lambda: G.gdn_lin_decode(q, k, v, ld, state[..., :16]))
    refused(lambda: G.gdn_lin_decode(q, k, v, ld, state, zeros(1, dtype=torch.int64)))
    assert "CUDA" in refused(lambda: G.gdn_lin_decode(q, k, v, ld, plain(state)))
    assert "pages" in refused(lambda: G.gdn_lin_decode(q, k, v, ld, state.transpose(2, 3)))
    with pytest.raises(Reached):
        G.gdn_lin_decode(q, k, v, ld, state)


def test_group_norm():
    x, w = zeros(3, 2, 8), zeros(8)
    m = zeros(3, 4)
    fwd = lambda *a, **kw: G.gdn_group_norm(*a, **kw)  # noqa: E731
    refused(lambda: fwd(x[0], w, None, 4))
    refused(lambda: fwd(x, w[:7], None, 4))
    refused(lambda: fwd(x, w.double(), None, 4))
    refused(lambda: fwd(x.half(), w, None, 4), TypeError, ValueError)
    refused(lambda: fwd(x, w, None, 4, gate=x[:2]))
    refused(lambda: fwd(x, w, None, 4, mean=m[:, :3]))
    assert "CUDA" in refused(lambda: fwd(plain(x), w, None, 4))
    assert "contiguous" in refused(lambda: fwd(x.transpose(0, 1), w, None, 4))
    with pytest.raises(Reached):
        fwd(x, w, None, 4)
    refused(lambda: G.gdn_group_norm_bwd(x, w, None, 4, m[:2], m, x))
    refused(lambda: G.gdn_group_norm_bwd(x, w, None, 4, m, m, x[:, :1]))
    assert "CUDA" in refused(lambda: G.gdn_group_norm_bwd(x, w, None, 4, plain(m), m, x))
    with pytest.raises(Reached):
        G.gdn_group_norm_bwd(x, w, None, 4, m, m, x)


def test_pages():
    i32 = lambda *s: zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, table, counts, refs, rows = zeros(6, 16), i32(4, 2), i32(4), i32(6), i32(3)
    calls = (lambda *a: G.gdn_pages_fork(*a, rows, rows), lambda *a: G.gdn_pages_compact(*a),
             lambda p, t, c, r: G.gdn_pages_free(t, c, r, rows))
    for call in calls:
        refused(lambda: call(pool, table.long(), counts, refs))
        refused(lambda: call(pool, table, counts[:3], refs))
        refused(lambda: call(pool, table, counts, refs.long()))
        assert "CUDA" in refused(lambda: call(pool, plain(table), counts, refs))
        assert "contiguous" in refused(lambda: call(pool, i32(2, 4).t(), counts, refs))
        with pytest.raises(Reached):
            call(pool, table, counts, refs)
    refused(lambda: G.gdn_pages_fork(pool, table, counts, refs[:5], rows, rows))
    refused(lambda: G.gdn_pages_fork(pool, table, counts, refs, rows, rows[:2]))
    refused(lambda: G.gdn_pages_free(table, counts, refs, rows.long()))
    refused(lambda: G.gdn_pages_copy(pool, rows, rows[:2]))
    assert "CUDA" in refused(lambda: G.gdn_pages_copy(plain(pool), rows, rows))
    with pytest.raises(Reached):
        G.gdn_pages_copy(pool, rows, rows)
