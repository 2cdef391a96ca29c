"""Tensors on several devices and streams of another one, in the binding of linear
attention, group norm and pages.  As in test_lin_binding nothing reaches the library; the
tensors say which device they are on, and the current device is a stand-in."""
from __future__ import annotations

import contextlib

import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G


class Device(torch.Tensor):
    index = 1
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.index

    @classmethod
    def __torch_function__(cls, func, types, args=(), kwargs=None):
        out = super().__torch_function__(func, types, args, kwargs or {})
        for a in args:
            if isinstance(a, Device) and isinstance(out, Device):
                out.index = a.index
        return out


class Stream:
    def __init__(self, index):
        self.device_index, self.cuda_stream = index, 7


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The calls that were made: (name, the device current then)."""
    made, current = [], [0]

    @contextlib.contextmanager
    def device(i):
        was, current[0] = current[0], i
        try:
            yield
        finally:
            current[0] = was

    def entry(name):
        return lambda *args: made.append((name, current[0])) or 0
    monkeypatch.setattr(G, "_call", entry)
    monkeypatch.setattr(G, "_current_device", lambda: current[0], raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 100 + d, raising=False)
    monkeypatch.setattr(G, "_empty", lambda stream, like, shape, dtype: zeros(*shape, dtype=dtype,
                                                                             index=like.get_device()))
    monkeypatch.setattr(G, "_like_new", lambda stream, t: zeros(*t.shape, dtype=t.dtype,
                                                                index=t.get_device()))
    for name in ("gdn_lin_workspace_size", "gdn_group_norm_workspace_size", "gdn_pages_workspace_size"):
        monkeypatch.setattr(G, name, lambda *a: 512)
    yield made
    assert current[0] == 0


def zeros(*s, dtype=torch.float32, index=1):
    t = torch.zeros(*s, dtype=dtype).as_subclass(Device)
    t.index = index
    return t


def jobs():
    """name -> (tensors, call of them)."""
    f, i32 = zeros, lambda *s: zeros(*s, dtype=torch.int32)
    q = lambda: f(1, 4, 2, 32)  # noqa: E731
    one = lambda: f(1, 2, 32)  # noqa: E731
    state = lambda: f(1, 2, 32, 32)  # noqa: E731
    book = lambda: dict(table=i32(4, 2), counts=i32(4), refs=i32(6))  # noqa: E731
    return {
        "gdn_lin_fwd": (dict(q=q(), k=q(), v=q(), log_decay=f(2), initial_state=state(),
                             cu_seqlens=i32(2), o=q(), final_state=state()), G.gdn_lin_fwd),
        "gdn_lin_bwd": (dict(q=q(), k=q(), v=q(), log_decay=f(2), d_o=q(), initial_state=state(),
                             cu_seqlens=i32(2), d_final_state=state()), G.gdn_lin_bwd),
        "gdn_lin_decode": (dict(q=one(), k=one(), v=one(), log_decay=f(2), state=state(),
                                pages=i32(1), o=one(), state_out=state()), G.gdn_lin_decode),
        "gdn_group_norm": (dict(x=f(3, 2, 8), weight=f(8), bias=f(8), gate=f(3, 2, 8), y=f(3, 2, 8),
                                mean=f(3, 4), rstd=f(3, 4)),
                           lambda **t: G.gdn_group_norm(groups=4, **t)),
        "gdn_group_norm_bwd": (dict(x=f(3, 2, 8), weight=f(8), bias=f(8), gate=f(3, 2, 8),
                                    mean=f(3, 4), rstd=f(3, 4), d_y=f(3, 2, 8)),
                               lambda **t: G.gdn_group_norm_bwd(groups=4, **t)),
        "gdn_pages_copy": (dict(pool=f(6, 16), src=i32(2), dst=i32(2)), G.gdn_pages_copy),
        "gdn_pages_fork": (dict(pool=f(6, 16), **book(), parents=i32(2), children=i32(2),
                                fresh=i32(2)), G.gdn_pages_fork),
        "gdn_pages_free": (dict(**book(), rows=i32(2), table_out=i32(4, 2)), G.gdn_pages_free),
        "gdn_pages_compact": (dict(pool=f(6, 16), **book(), num_live=i32(1)), G.gdn_pages_compact),
    }


JOBS = list(jobs())


@pytest.mark.parametrize("name", JOBS)
def test_the_tensors_device_is_current_during_the_call(calls, name):
    tensors, call = jobs()[name]
    call(**tensors)
    call(**tensors, stream=Stream(1))
    assert calls == [(name, 1)] * 2


@pytest.mark.parametrize("name", JOBS)
def test_a_tensor_of_another_device_is_refused(calls, name):
    tensors, call = jobs()[name]
    for other in tensors:
        if other == "q" or other == "x":
            continue
        t = {n: x for n, x in tensors.items()}
        t[other] = zeros(*t[other].shape, dtype=t[other].dtype, index=0)
        with pytest.raises(ValueError, match="device"):
            call(**t)
    assert calls == []


@pytest.mark.parametrize("name", JOBS)
def test_a_stream_of_another_device_is_refused(calls, name):
    tensors, call = jobs()[name]
    with pytest.raises(ValueError, match="stream"):
        call(**tensors, stream=Stream(0))
    assert calls == []


@pytest.mark.parametrize("name", JOBS)
def test_a_workspace_must_be_on_the_device(calls, name):
    tensors, call = jobs()[name]
    wide = zeros(1024, dtype=torch.uint8)
    for ws in (torch.zeros(512, dtype=torch.uint8), zeros(512, dtype=torch.uint8, index=0), wide[::2]):
        with pytest.raises(ValueError, match="workspace"):
            call(**tensors, workspace=ws)
    assert calls == []
    call(**tensors, workspace=wide)
    assert calls == [(name, 1)]


def test_decode_on_an_empty_pool_is_refused():
    """As any other state that does not fit, not by an IndexError."""
    t, call = jobs()["gdn_lin_decode"]
    with pytest.raises(ValueError):
        call(**{**t, "state": zeros(0, 2, 32, 32), "state_out": zeros(0, 2, 32, 31)})
