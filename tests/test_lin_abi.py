"""CPU tests of the host-side checks of the linear-attention, group-norm and
page entry points (fake device addresses, never dereferenced; nothing is
launched)."""
import ctypes

import pytest

from linear_attention_recurrence_gated_gb300 import build as gbuild
from linear_attention_recurrence_gated_gb300 import gdn as G

vp = ctypes.c_void_p
BASE = 1 << 40


def at(i):
    return BASE + i * (1 << 32)


@pytest.fixture(scope="module")
def L():
    gbuild.build()
    return G.lib()


def lin_fwd(L, **over):
    a = dict(q=at(0), k=at(1), v=at(2), ld=at(3), s0=at(4), cu=None, o=at(5), sN=at(6), B=2, T=100,
             H=3, dk=64, dv=64, N=2, sq=0, sk=0, sv=0, dtype=G.GDN_BF16, flags=0, ws=at(7),
             ws_bytes=1 << 30)
    a.update(over)
    return L.gdn_lin_fwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["ld"]), vp(a["s0"]), vp(a["cu"]),
                         vp(a["o"]), vp(a["sN"]), a["B"], a["T"], a["H"], a["dk"], a["dv"], a["N"],
                         a["sq"], a["sk"], a["sv"], a["dtype"], a["flags"], vp(a["ws"]),
                         a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(dk=48), 2), (dict(dk=288), 2), (dict(dv=16), 2), (dict(dv=320), 2), (dict(N=20000, B=20000), 2),
    (dict(B=0), 1), (dict(T=-1), 1), (dict(H=0), 1), (dict(N=3), 1), (dict(dtype=5), 1),
    (dict(flags=1), 1), (dict(cu=at(9), N=3), 1), (dict(sq=191), 1), (dict(sk=196), 1),
    (dict(sv=-192), 1), (dict(q=None), 1), (dict(v=None), 1), (dict(ld=None), 1),
    (dict(o=None), 1), (dict(q=at(0) + 8), 1), (dict(sN=at(6) + 4), 1), (dict(ws=None), 3),
    (dict(ws_bytes=255), 3), (dict(ws=at(7) + 8), 1), (dict(o=at(0)), 1), (dict(o=at(2) + 64), 1),
    (dict(sN=at(1)), 1), (dict(sN=at(4) + 16), 1), (dict(o=at(4)), 1), (dict(ws=at(4)), 1),
    (dict(T=0, sN=at(4) + 16), 1)])
def test_lin_fwd_refuses(L, over, code):
    assert lin_fwd(L, **over) == code


def lin_bwd(L, **over):
    a = dict(q=at(0), k=at(1), v=at(2), ld=at(3), s0=at(4), cu=None, do=at(5), ds=at(6), dq=at(7),
             dk_=at(8), dv_=at(9), dh0=at(10), B=2, T=100, H=3, dk=64, dv=64, N=2, sq=0, sk=0, sv=0,
             dtype=G.GDN_BF16, flags=0, ws=at(11), ws_bytes=1 << 30)
    a.update(over)
    return L.gdn_lin_bwd(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["ld"]), vp(a["s0"]), vp(a["cu"]),
                         vp(a["do"]), vp(a["ds"]), vp(a["dq"]), vp(a["dk_"]), vp(a["dv_"]),
                         vp(a["dh0"]), a["B"], a["T"], a["H"], a["dk"], a["dv"], a["N"], a["sq"],
                         a["sk"], a["sv"], a["dtype"], a["flags"], vp(a["ws"]), a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(dk=40), 2), (dict(dv=512), 2), (dict(N=1), 1), (dict(flags=8), 1), (dict(do=None), 1),
    (dict(dq=None), 1), (dict(dk_=at(8) + 2), 1), (dict(ws=None), 3), (dict(ws_bytes=100), 3),
    (dict(dq=at(0)), 1), (dict(dv_=at(5)), 1), (dict(dk_=at(7)), 1), (dict(dh0=at(4)), 1),
    (dict(dh0=at(6)), 1), (dict(dh0=at(8)), 1), (dict(ws=at(5)), 1), (dict(sq=100), 1)])
def test_lin_bwd_refuses(L, over, code):
    assert lin_bwd(L, **over) == code


def lin_decode(L, **over):
    a = dict(q=at(0), k=at(1), v=at(2), ld=at(3), si=at(4), so=at(4), pages=at(5), o=at(6), N=4,
             H=2, dk=64, dv=64, P=9, stride=0, dtype=G.GDN_BF16, flags=0, ws=None, ws_bytes=0)
    a.update(over)
    return L.gdn_lin_decode(vp(a["q"]), vp(a["k"]), vp(a["v"]), vp(a["ld"]), vp(a["si"]),
                            vp(a["so"]), vp(a["pages"]), vp(a["o"]), a["N"], a["H"], a["dk"],
                            a["dv"], a["P"], a["stride"], a["dtype"], a["flags"], vp(a["ws"]),
                            a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(dk=33), 2), (dict(dv=288), 2), (dict(N=70000), 2), (dict(N=0), 1), (dict(P=0), 1),
    (dict(flags=1), 1), (dict(dtype=2), 1), (dict(stride=8191), 1), (dict(stride=8194), 1),
    (dict(so=None), 1), (dict(pages=None, P=3), 1), (dict(pages=at(5) + 4), 1), (dict(o=at(4)), 1),
    (dict(si=at(4) + 32), 1), (dict(o=at(2)), 1), (dict(so=at(1)), 1), (dict(ws=at(7), ws_bytes=100), 3)])
def test_lin_decode_refuses(L, over, code):
    assert lin_decode(L, **over) == code


def norm(L, **over):
    a = dict(x=at(0), w=at(1), b=at(2), gate=at(3), y=at(4), mean=at(5), rstd=at(6), N=4, S=10, C=64,
             G=4, eps=1e-5, dtype=G.GDN_BF16, flags=0, ws=at(7), ws_bytes=1 << 30)
    a.update(over)
    return L.gdn_group_norm(vp(a["x"]), vp(a["w"]), vp(a["b"]), vp(a["gate"]), vp(a["y"]),
                            vp(a["mean"]), vp(a["rstd"]), a["N"], a["S"], a["C"], a["G"], a["eps"],
                            a["dtype"], a["flags"], vp(a["ws"]), a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(C=66), 1), (dict(G=0), 1), (dict(N=-1), 1), (dict(C=8256), 2), (dict(dtype=3), 1),
    (dict(flags=1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(x=None), 1),
    (dict(y=None), 1), (dict(y=at(4) + 2), 1), (dict(ws=None), 3), (dict(ws_bytes=10), 3),
    (dict(y=at(0)), 1), (dict(y=at(3)), 1), (dict(mean=at(6)), 1), (dict(mean=at(1)), 1),
    (dict(ws=at(0)), 1), (dict(N=0), 0), (dict(S=0), 0)])
def test_norm_refuses(L, over, code):
    assert norm(L, **over) == code


def norm_bwd(L, **over):
    a = dict(x=at(0), w=at(1), b=at(2), gate=at(3), mean=at(4), rstd=at(5), dy=at(6), dx=at(7),
             dgate=at(8), dw=at(9), db=at(10), N=4, S=10, C=64, G=4, dtype=G.GDN_BF16, flags=0,
             ws=at(11), ws_bytes=1 << 30)
    a.update(over)
    return L.gdn_group_norm_bwd(*(vp(a[n]) for n in ("x", "w", "b", "gate", "mean", "rstd", "dy",
                                                     "dx", "dgate", "dw", "db")),
                                a["N"], a["S"], a["C"], a["G"], a["dtype"], a["flags"], vp(a["ws"]),
                                a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(C=70), 1), (dict(C=16384), 2), (dict(flags=2), 1), (dict(dy=None), 1), (dict(mean=None), 1),
    (dict(dgate=None), 1), (dict(dx=None), 1), (dict(ws=None), 3), (dict(dx=at(0)), 1),
    (dict(dgate=at(7)), 1), (dict(dw=at(1)), 1), (dict(db=at(9)), 1), (dict(ws=at(6)), 1)])
def test_norm_bwd_refuses(L, over, code):
    assert norm_bwd(L, **over) == code


def fork(L, **over):
    a = dict(pool=at(0), bytes=64, P=100, t=at(1), c=at(2), r=at(3), R=10, M=4, par=at(4), ch=at(5),
             n=3, fresh=at(6), to=at(1), co=at(2), ro=at(3), ws=at(7), ws_bytes=1 << 20)
    a.update(over)
    return L.gdn_pages_fork(vp(a["pool"]), a["bytes"], a["P"], vp(a["t"]), vp(a["c"]), vp(a["r"]),
                            a["R"], a["M"], vp(a["par"]), vp(a["ch"]), a["n"], vp(a["fresh"]),
                            vp(a["to"]), vp(a["co"]), vp(a["ro"]), vp(a["ws"]), a["ws_bytes"], vp(0))


@pytest.mark.parametrize("over,code", [
    (dict(bytes=8), 2), (dict(bytes=0), 1), (dict(P=0), 1), (dict(M=0), 1), (dict(n=-1), 1),
    (dict(P=1 << 25), 2), (dict(ws=None), 3), (dict(ws_bytes=300), 3), (dict(pool=None), 1),
    (dict(par=None), 1), (dict(fresh=None), 1), (dict(t=at(1) + 4), 1), (dict(fresh=at(4)), 1),
    (dict(to=at(1) + 16), 1), (dict(co=at(1)), 1), (dict(ro=at(2)), 1), (dict(pool=at(5)), 1),
    (dict(ws=at(0)), 1), (dict(R=0), 1)])
def test_fork_refuses(L, over, code):
    assert fork(L, **over) == code


def test_the_other_page_calls_refuse(L):
    copy = lambda pool=at(0), b=64, P=9, s=at(1), d=at(2), n=3, ws=at(3), wb=1 << 20: \
        L.gdn_pages_copy(vp(pool), b, P, vp(s), vp(d), n, vp(ws), wb, vp(0))  # noqa: E731
    assert copy(b=24) == 2 and copy(P=0) == 1 and copy(s=None) == 1 and copy(d=at(0)) == 1
    assert copy(ws=None) == 3 and copy(wb=256) == 3 and copy(ws=at(1)) == 1 and copy(n=0) == 0
    free = lambda t=at(0), c=at(1), r=at(2), R=9, rows=at(3), n=2, to=at(0), co=at(1), ro=at(2), \
        ws=at(4), wb=1 << 20: L.gdn_pages_free(vp(t), vp(c), vp(r), 50, R, 4, vp(rows), n, vp(to),
                                               vp(co), vp(ro), vp(ws), wb, vp(0))  # noqa: E731
    assert free(rows=None) == 1 and free(R=0) == 1 and free(to=at(1)) == 1 and free(ws=None) == 3
    assert free(ro=at(3)) == 1 and free(c=None) == 1 and free(ws=at(3)) == 1 and free(R=-1) == 1
    compact = lambda pool=at(0), b=64, t=at(1), c=at(2), r=at(3), num=at(4), to=at(1), ro=at(3), \
        ws=at(5), wb=1 << 20: L.gdn_pages_compact(vp(pool), b, 50, vp(t), vp(c), vp(r), 9, 4,
                                                  vp(num), vp(to), vp(ro), vp(ws), wb,
                                                  vp(0))  # noqa: E731
    assert compact(b=40) == 2 and compact(num=None) == 1 and compact(num=at(2)) == 1
    assert compact(to=at(2)) == 1 and compact(pool=at(3)) == 1 and compact(wb=1) == 3
    assert compact(ro=at(1)) == 1


def test_workspace_sizes(L):
    assert G.gdn_lin_workspace_size(8, 4096, 16, 64, 64) >= 256
    assert G.gdn_lin_workspace_size(0, 4096, 16, 64, 64) == 0
    assert G.gdn_group_norm_workspace_size(4, 4096, 1280, 40) > 0
    assert G.gdn_group_norm_workspace_size(0, 4096, 1280, 40) == 0
    assert G.gdn_pages_workspace_size(100, 10, 5) > 256
    assert G.gdn_pages_workspace_size(0, 10, 5) == 0
