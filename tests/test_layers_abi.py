"""CPU tests of the host-side checks of the scan, convolution and q/k-norm entry points
(fake device addresses, never dereferenced; nothing is launched)."""
import ctypes

import pytest

from linear_attention_recurrence_gated_gb300 import build as gbuild
from linear_attention_recurrence_gated_gb300 import gdn as G

vp = ctypes.c_void_p
BASE = 1 << 40


def at(i):
    return BASE + i * (1 << 34)


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return G.lib()


def call(f, order, values, over):
    a = dict(values)
    a.update(over)
    pointers = set(order.split()[:a["_pointers"]]) | {"ws"}
    args = [vp(a[n]) if n in pointers else a[n] for n in order.split()]
    return f(*args, vp(0))


SSM = "x dt A b c D gate bias h0 cu y hT B T C S G N sx sdt sb sc sg dtype flags ws bytes"


def ssm_fwd(L, **over):
    v = dict(x=at(0), dt=at(1), A=at(2), b=at(3), c=at(4), D=at(5), gate=at(6), bias=at(7), h0=at(8),
             cu=None, y=at(9), hT=at(10), B=2, T=100, C=48, S=16, G=2, N=2, sx=0, sdt=0, sb=0, sc=0,
             sg=0, dtype=G.GDN_BF16, flags=G.GDN_DT_SOFTPLUS, ws=at(11), bytes=1 << 30, _pointers=12)
    return call(L.gdn_ssm_fwd, SSM, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(S=24), 2), (dict(S=128), 2), (dict(S=4), 2), (dict(C=40), 2), (dict(C=50), 2),
    (dict(N=20000, B=20000), 2), (dict(C=1 << 21), 2), (dict(C=49), 1), (dict(B=0), 1),
    (dict(T=-1), 1), (dict(C=0), 1), (dict(S=0), 1), (dict(G=0), 1), (dict(N=3), 1), (dict(dtype=2), 1),
    (dict(flags=1), 1), (dict(flags=1 << 8), 1), (dict(cu=at(12), N=3), 1), (dict(sx=47), 1),
    (dict(sx=52), 1), (dict(sb=24), 1), (dict(sg=-48), 1), (dict(x=None), 1), (dict(dt=None), 1),
    (dict(A=None), 1), (dict(b=None), 1), (dict(c=None), 1), (dict(y=None), 1), (dict(x=at(0) + 8), 1),
    (dict(h0=at(8) + 4), 1), (dict(ws=None), 3), (dict(bytes=255), 3), (dict(ws=at(11) + 4), 1),
    (dict(y=at(0)), 1), (dict(y=at(6) + 64), 1), (dict(hT=at(2)), 1), (dict(hT=at(8) + 16), 1),
    (dict(y=at(8)), 1), (dict(hT=at(9)), 1), (dict(ws=at(8)), 1), (dict(ws=at(3)), 1),
    (dict(y=at(11)), 1), (dict(T=0, hT=at(8) + 16), 1)])
def test_ssm_fwd_refuses(L, over, code):
    assert ssm_fwd(L, **over) == code


SSM_BWD = ("x dt A b c D gate bias h0 cu dy dhT dx ddt dA db dc dD dgate dbias dh0 B T C S G N sx sdt "
           "sb sc sg dtype flags ws bytes")


def ssm_bwd(L, **over):
    names = SSM_BWD.split()[:21]
    v = {n: at(i) for i, n in enumerate(names)}
    v.update(cu=None, B=2, T=100, C=48, S=16, G=2, N=2, sx=0, sdt=0, sb=0, sc=0, sg=0,
             dtype=G.GDN_F32, flags=G.GDN_DT_SOFTPLUS, ws=at(30), bytes=1 << 33, _pointers=21)
    return call(L.gdn_ssm_bwd, SSM_BWD, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(S=20), 2), (dict(N=1), 1), (dict(flags=4), 1), (dict(dy=None), 1), (dict(dx=None), 1),
    (dict(ddt=None), 1), (dict(db=None), 1), (dict(dc=None), 1), (dict(dgate=None), 1),
    (dict(gate=None), 1), (dict(dx=at(12) + 8), 1), (dict(ws=None), 3), (dict(bytes=4096), 3),
    (dict(dx=at(0)), 1), (dict(ddt=at(12)), 1), (dict(dh0=at(8)), 1), (dict(dA=at(2)), 1),
    (dict(dbias=at(17)), 1), (dict(ws=at(10)), 1), (dict(dc=at(30)), 1), (dict(sdt=40), 1)])
def test_ssm_bwd_refuses(L, over, code):
    assert ssm_bwd(L, **over) == code


STEP = "x dt A b c D gate bias si so pages y N C S G P stride dtype flags ws bytes"


def ssm_step(L, **over):
    v = {n: at(i) for i, n in enumerate(STEP.split()[:12])}
    v.update(so=v["si"], N=4, C=48, S=16, G=1, P=9, stride=0, dtype=G.GDN_BF16, flags=0, ws=None, bytes=0,
             _pointers=12)
    return call(L.gdn_ssm_step, STEP, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(S=12), 2), (dict(N=0), 1), (dict(P=0), 1), (dict(pages=None, P=3), 1), (dict(stride=700), 1),
    (dict(stride=770), 1), (dict(flags=2), 1), (dict(so=None), 1), (dict(x=None), 1), (dict(y=None), 1),
    (dict(y=at(11) + 8), 1), (dict(ws=at(20), bytes=100), 3), (dict(y=at(0)), 1), (dict(so=at(0)), 1),
    (dict(so=at(8) + 16), 1), (dict(y=at(8)), 1), (dict(y=at(10)), 1)])
def test_ssm_step_refuses(L, over, code):
    assert ssm_step(L, **over) == code


CONV = "x w bias prev cu y tail B T C K N sx dtype flags ws bytes"


def conv_fwd(L, **over):
    v = {n: at(i) for i, n in enumerate(CONV.split()[:7])}
    v.update(cu=None, B=2, T=100, C=48, K=4, N=2, sx=0, dtype=G.GDN_BF16, flags=G.GDN_CONV_SILU, ws=at(9),
             bytes=256, _pointers=7)
    return call(L.gdn_conv_fwd, CONV, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(K=5), 2), (dict(C=44), 2), (dict(N=20000, B=20000), 2), (dict(K=0), 1), (dict(C=0), 1),
    (dict(B=0), 1), (dict(T=-1), 1), (dict(N=3), 1), (dict(cu=at(8), N=3), 1), (dict(flags=1), 1),
    (dict(dtype=7), 1), (dict(sx=40), 1), (dict(sx=52), 1), (dict(x=None), 1), (dict(w=None), 1),
    (dict(y=None), 1), (dict(x=at(0) + 2), 1), (dict(ws=None), 3), (dict(bytes=16), 3), (dict(y=at(0)), 1),
    (dict(tail=at(3)), 1), (dict(tail=at(5)), 1), (dict(y=at(9)), 1), (dict(ws=at(0)), 1),
    (dict(T=0, tail=at(3) + 16), 1)])
def test_conv_fwd_refuses(L, over, code):
    assert conv_fwd(L, **over) == code


CONV_BWD = "x w bias prev cu dy dtail dx dw dbias dprev B T C K N sx dtype flags ws bytes"


def conv_bwd(L, **over):
    v = {n: at(i) for i, n in enumerate(CONV_BWD.split()[:11])}
    v.update(cu=None, B=2, T=100, C=48, K=4, N=2, sx=0, dtype=G.GDN_F32, flags=0, ws=at(15),
             bytes=1 << 24, _pointers=11)
    return call(L.gdn_conv_bwd, CONV_BWD, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(K=6), 2), (dict(N=1), 1), (dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=at(8) + 4), 1),
    (dict(ws=None), 3), (dict(bytes=300), 3), (dict(dx=at(0)), 1), (dict(dw=at(1)), 1),
    (dict(dprev=at(3)), 1), (dict(dbias=at(8)), 1), (dict(ws=at(5)), 1), (dict(dx=at(15)), 1),
    (dict(T=0, dprev=at(6) + 16), 1)])
def test_conv_bwd_refuses(L, over, code):
    assert conv_bwd(L, **over) == code


CONV_STEP = "x w bias state pages y N C K P stride dtype flags ws bytes"


def conv_step(L, **over):
    v = {n: at(i) for i, n in enumerate(CONV_STEP.split()[:6])}
    v.update(N=4, C=48, K=4, P=9, stride=0, dtype=G.GDN_BF16, flags=0, ws=None, bytes=0, _pointers=6)
    return call(L.gdn_conv_step, CONV_STEP, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(K=5), 2), (dict(C=12), 2), (dict(N=0), 1), (dict(P=0), 1), (dict(pages=None, P=2), 1),
    (dict(stride=100), 1), (dict(stride=148), 1), (dict(state=None), 1), (dict(x=None), 1),
    (dict(y=at(0)), 1), (dict(y=at(3)), 1), (dict(state=at(1)), 1), (dict(ws=at(8), bytes=8), 3)])
def test_conv_step_refuses(L, over, code):
    assert conv_step(L, **over) == code


QK = "q k qw kw pos freq qo ko B T Hq Hk D R sq sk scale eps dtype flags"


def qk(L, **over):
    v = {n: at(i) for i, n in enumerate(QK.split()[:8])}
    v.update(B=2, T=100, Hq=4, Hk=2, D=64, R=64, sq=0, sk=0, scale=1.0, eps=1e-6, dtype=G.GDN_BF16,
             flags=0, ws=None, _pointers=8)
    return call(L.gdn_qk_norm, QK, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(D=264), 2), (dict(D=60, R=0), 2), (dict(Hq=5000), 2), (dict(B=0), 1), (dict(T=-1), 1),
    (dict(Hk=0), 1), (dict(R=66), 1), (dict(R=7), 1), (dict(R=-2), 1), (dict(flags=2), 1),
    (dict(dtype=3), 1), (dict(sq=255), 1), (dict(sk=132), 1), (dict(q=None), 1), (dict(freq=None), 1),
    (dict(ko=None), 1), (dict(pos=at(4) + 4), 1), (dict(qo=at(0)), 1), (dict(ko=at(6)), 1),
    (dict(qo=at(2)), 1)])
def test_qk_norm_refuses(L, over, code):
    assert qk(L, **over) == code


QK_BWD = "q k qw kw pos freq dqo dko dq dk dqw dkw B T Hq Hk D R sq sk scale eps dtype flags ws bytes"


def qk_bwd(L, **over):
    v = {n: at(i) for i, n in enumerate(QK_BWD.split()[:12])}
    v.update(B=2, T=100, Hq=4, Hk=2, D=64, R=64, sq=0, sk=0, scale=1.0, eps=1e-6, dtype=G.GDN_F32,
             flags=0, ws=at(20), bytes=1 << 24, _pointers=12)
    return call(L.gdn_qk_norm_bwd, QK_BWD, v, over)


@pytest.mark.parametrize("over,code", [
    (dict(D=300), 2), (dict(dqo=None), 1), (dict(dk=None), 1), (dict(ws=None), 3), (dict(bytes=1024), 3),
    (dict(dq=at(0)), 1), (dict(dkw=at(10)), 1), (dict(dk=at(20)), 1), (dict(ws=at(7)), 1),
    (dict(sq=100), 1)])
def test_qk_norm_bwd_refuses(L, over, code):
    assert qk_bwd(L, **over) == code


def test_workspace_sizes(L):
    assert G.gdn_ssm_workspace_size(1, 256, 64, 16) >= 256
    assert L.gdn_ssm_workspace_size(1, 256, 64, 24, 1) == 0      # no such state size
    assert L.gdn_ssm_workspace_size(0, 256, 64, 16, 1) == 0
    assert L.gdn_ssm_bwd_workspace_size(1, 256, 63, 16, 2) == 0
    assert L.gdn_ssm_bwd_workspace_size(2, 100, 64, 16, 1) > 256
    assert L.gdn_conv_workspace_size(2, 100, 64, 4) > 256
    assert L.gdn_conv_workspace_size(2, 100, 64, 0) == 0
    assert L.gdn_qk_norm_workspace_size(2, 100, 64) > 0 and L.gdn_qk_norm_workspace_size(0, 1, 64) == 0
    # many short sequences: the scan's backward pass keeps no state of each
    many = L.gdn_ssm_bwd_workspace_size(16384, 1, 1280, 16, 1)
    assert many < 1 << 31
