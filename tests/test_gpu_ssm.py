"""Selective scan (gdn_ssm_fwd, gdn_ssm_bwd, gdn_ssm_step) on the GPU against the fp64
oracle.

Tolerances, relative L2 of a tensor: every factor exp(delta A) is off by at most 2^-22 (two
units of the exponential's last place and the rounding of its argument) and each of a
token's four operations by 2^-24; a state adds up at most T tokens, so fp32 results may be
off by T 2^-22 + 2^-20 (delta's own error).  Storage in bf16 adds its half step, 2^-8."""
import itertools

import pytest
import torch

import oracle.ssm as O
from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu
NAMES = ("x", "dt", "A_log", "b", "c", "h0", "D_skip", "gate", "dt_bias")


def inputs(B, T, D, S, G_, dtype, N=None, seed=0, gate=True, skip=True, bias=True, init=True,
           slices=False):
    g = torch.Generator().manual_seed(1000 * T + 10 * D + S + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = B if N is None else N
    i = dict(x=r(B, T, D).to(dtype), dt=(0.5 * r(B, T, D)).to(dtype),
             A_log=torch.log(torch.arange(1.0, S + 1)) + 0.2 * r(D, S),
             b=r(B, T, G_, S).to(dtype), c=r(B, T, G_, S).to(dtype),
             h0=r(N, D, S) if init else None, D_skip=1 + 0.2 * r(D) if skip else None,
             gate=r(B, T, D).to(dtype) if gate else None,
             dt_bias=r(D) - 3 if bias else None)
    i["d_y"] = r(B, T, D).to(dtype)
    i["d_hT"] = r(N, D, S) if init else None
    if slices:   # rows of wider tensors
        for n in ("x", "dt", "b", "c", "gate"):
            if i[n] is not None:
                t = i[n]
                wide = torch.full((B, T, t[0, 0].numel() + 24), float("nan"), dtype=dtype).cuda()
                wide[..., 8:8 + t[0, 0].numel()] = t.flatten(2).cuda()
                i[n] = wide[..., 8:8 + t[0, 0].numel()].view(t.shape)
    return {n: None if t is None else t.cuda() for n, t in i.items()}


def call(i, cu=None, **kw):
    return G.gdn_ssm_fwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], i["h0"], cu,
                         D_skip=i["D_skip"], gate=i["gate"], dt_bias=i["dt_bias"],
                         **{"dt_softplus": True, "check": True, **kw})


def call_bwd(i, cu=None, **kw):
    return G.gdn_ssm_bwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], i["d_y"], i["h0"], cu,
                         i["d_hT"], D_skip=i["D_skip"], gate=i["gate"], dt_bias=i["dt_bias"],
                         **{"dt_softplus": True, "check": True, **kw})


def want(i, cu=None, softplus=True):
    y, last = O.scan(*(O._d(i[n]) for n in NAMES[:5]), O._d(i["h0"]), cu, O._d(i["D_skip"]),
                     O._d(i["gate"]), O._d(i["dt_bias"]), softplus)
    return y, last


def want_bwd(i, cu=None, softplus=True):
    g = O.grads(O.scan, {n: i[n] for n in NAMES}, (i["d_y"], i["d_hT"]), cu=cu,
                dt_softplus=softplus)
    names = dict(x="dx", dt="ddt", A_log="dA_log", b="db", c="dc", h0="dh0", D_skip="dD_skip",
                 gate="dgate", dt_bias="ddt_bias")
    return {names[n]: t for n, t in g.items()}


def close(got, ref, T, what=""):
    tol = T * 2.0 ** -22 + 2.0 ** -20 + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    d = got.detach().cpu().double() - ref
    assert torch.isfinite(got.float()).all(), what
    err, size = float(d.norm()), float(ref.norm())
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.2e} > {tol:.2e}"


def check_bwd(got, ref, T):
    for n, t in ref.items():
        close(got[n], t, T, n)


# every state size, groups, lengths around tiles (8, 16, 32 tokens) and pieces (32), channels
# that fill a CTA's and such that do not
SIZES = [(1, 1, 8, 8, 1), (2, 7, 24, 16, 1), (1, 8, 64, 32, 1), (3, 17, 32, 64, 2),
         (1, 33, 136, 16, 1), (2, 64, 48, 8, 3), (1, 100, 264, 8, 1), (1, 300, 40, 16, 1),
         (2, 129, 72, 32, 1), (1, 257, 40, 64, 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, dtype):
    i = inputs(*size, dtype)
    y, last = call(i)
    ry, rl = want(i)
    close(y, ry, size[1], "y")
    close(last, rl, size[1], "state")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", SIZES)
def test_backward(size, dtype):
    i = inputs(*size, dtype, seed=1)
    check_bwd(call_bwd(i), want_bwd(i), size[1])


@pytest.mark.parametrize("gate,skip,bias,init,softplus",
                         list(itertools.product([False, True], repeat=5))[::3])
def test_parts(gate, skip, bias, init, softplus):
    i = inputs(2, 41, 24, 16, 1, torch.float32, gate=gate, skip=skip, bias=bias, init=init)
    if not softplus:   # steps that are given as they are
        i["dt"] = i["dt"].abs() * 0.2
        i["dt_bias"] = None if i["dt_bias"] is None else i["dt_bias"].abs() * 0.1
    y, last = call(i, dt_softplus=softplus)
    ry, rl = want(i, softplus=softplus)
    close(y, ry, 41, "y")
    close(last, rl, 41, "state")
    check_bwd(call_bwd(i, dt_softplus=softplus), want_bwd(i, softplus=softplus), 41)


PACKED = [[5], [0, 3, 0, 0, 40, 1], [1] * 9, [64, 32, 31, 33, 7], [0, 0, 9, 0], [200, 8, 16]]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", PACKED)
def test_packed(lens, dtype):
    cu = [sum(lens[:k]) for k in range(len(lens) + 1)]
    i = inputs(1, cu[-1], 40, 16, 1, dtype, N=len(lens))
    dev = torch.tensor(cu, dtype=torch.int32).cuda()
    y, last = call(i, dev)
    ry, rl = want(i, cu)
    close(y, ry, max(lens), "y")
    close(last, rl, max(lens), "state")
    check_bwd(call_bwd(i, dev), want_bwd(i, cu), max(lens))


def test_slices_of_projections():
    i = inputs(2, 37, 48, 16, 2, torch.bfloat16, slices=True)
    dense = {n: None if t is None else t.contiguous() for n, t in i.items()}
    for a, b in zip(call(i), call(dense)):
        assert torch.equal(a, b)
    for n, t in call_bwd(i).items():
        assert torch.equal(t, call_bwd(dense)[n]), n


def test_cut_along_time_and_not():
    """A workspace of 256 bytes leaves sequences whole."""
    i = inputs(1, 1500, 32, 16, 1, torch.float32)
    small = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert G.gdn_ssm_workspace_size(1, 1500, 32, 16) > 256
    whole, cut = call(i, workspace=small), call(i)
    for a, b in zip(whole, cut):
        close(a, b.double().cpu(), 1500)
    ry, rl = want(i)
    close(cut[0], ry, 1500)
    close(cut[1], rl, 1500)
    check_bwd(call_bwd(i), want_bwd(i), 1500)


def test_state_in_place_and_chained():
    for T in (40, 1500):   # one piece, several
        i = inputs(2, T, 24, 16, 1, torch.float32)
        y, last = call(i)
        h = i["h0"].clone()
        y2, last2 = call({**i, "h0": h}, final_state=h)
        assert last2 is h and torch.equal(y, y2) and torch.equal(last, h)
        cut = T // 3
        part = lambda a, b: {n: t[:, a:b] if t is not None and t.dim() > 2 and n != "h0" and n != "d_hT"  # noqa: E731
                             else t for n, t in i.items()}
        first = {n: t.contiguous() if t is not None else t for n, t in part(0, cut).items()}
        rest = {n: t.contiguous() if t is not None else t for n, t in part(cut, T).items()}
        y1, mid = call(first)
        y3, end = call({**rest, "h0": mid})
        close(torch.cat([y1, y3], 1), y.double().cpu(), T)
        close(end, last.double().cpu(), T)


def test_results_are_reproducible():
    i = inputs(2, 700, 136, 16, 1, torch.bfloat16)
    a, b = call_bwd(i), call_bwd(i)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_long_sums_of_equal_terms():
    """3449 tokens of equal gradients: the sums over tokens keep fp32's precision."""
    T, D = 3449, 8
    i = inputs(1, T, D, 8, 1, torch.float32, init=False)
    i["x"].fill_(0.3)
    i["d_y"].fill_(0.7)
    i["gate"] = None
    g = call_bwd(i)
    want_skip = T * float(i["x"][0, 0, 0]) * float(i["d_y"][0, 0, 0])
    # sums of 16, of blocks of them, over CTAs: at most some 60 additions in a row
    assert (g["dD_skip"].double() - want_skip).abs().max() <= 64 * 2.0 ** -24 * want_skip


def test_not_finite_values_stay_behind():
    """NaN and infinity reach their token, their channel's later ones, and nothing else."""
    for T in (60, 1500):
        i = inputs(2, T, 24, 16, 1, torch.float32)
        y, last = call(i)
        for name, bad in (("x", float("nan")), ("gate", float("inf")), ("dt", float("nan"))):
            j = {n: None if t is None else t.clone() for n, t in i.items()}
            j[name][1, 50, 5] = bad
            y2, last2 = call(j)
            assert torch.equal(y2[0], y[0]) and torch.equal(y2[1, :50], y[1, :50])
            keep = [c for c in range(24) if c != 5]
            assert torch.equal(y2[1][:, keep], y[1][:, keep])
            assert torch.equal(last2[0], last[0]) and torch.equal(last2[1, keep], last[1, keep])
            assert not torch.isfinite(y2[1, 50, 5])
        j = {n: None if t is None else t.clone() for n, t in i.items()}
        j["d_y"][1, 50, 5] = float("nan")
        g, h = call_bwd(i), call_bwd(j)
        assert torch.equal(g["dx"][0], h["dx"][0]) and torch.equal(g["dx"][1, 51:], h["dx"][1, 51:])
        assert torch.equal(g["db"][1, 51:], h["db"][1, 51:])


def test_extreme_steps():
    """Steps of zero, of a thousand (the state is replaced), huge negative logits."""
    i = inputs(1, 24, 16, 16, 1, torch.float32, bias=False, gate=False)
    i["dt"][0, 3] = 1000.0
    i["dt"][0, 9] = -1000.0
    i["dt"][0, 15] = 0.0
    y, last = call(i)
    ry, rl = want(i)
    close(y, ry, 24)
    close(last, rl, 24)
    check_bwd(call_bwd(i), want_bwd(i), 24)


def test_gradients_are_differences():
    i = inputs(1, 50, 16, 8, 1, torch.float32)
    g = call_bwd(i)
    names = dict(x="dx", dt="ddt", A_log="dA_log", b="db", c="dc", h0="dh0", D_skip="dD_skip",
                 gate="dgate", dt_bias="ddt_bias")

    def value(j):
        y, last = call(j)
        return float((y.double() * i["d_y"].double()).sum() +
                     (last.double() * i["d_hT"].double()).sum())

    gen = torch.Generator().manual_seed(5)
    scale = float(call(i)[0].double().norm() * i["d_y"].double().norm())
    for n, d in names.items():
        v = torch.randn(i[n].shape, generator=gen).cuda()
        e = 2.0 ** -7
        diff = (value({**i, n: i[n] + e * v}) - value({**i, n: i[n] - e * v})) / (2 * e)
        exact = float((g[d].double() * v.double()).sum())
        # the third derivative's share, e^2, and the outputs' rounding over e
        assert abs(diff - exact) <= 30 * e * e * (abs(exact) + 1) + 100 * 2.0 ** -22 * scale / e, n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,D,S,G_", [(1, 8, 8, 1), (3, 136, 16, 1), (5, 48, 32, 2), (9, 40, 64, 1),
                                      (300, 1280, 16, 1), (257, 72, 16, 3)])
def test_step(N, D, S, G_, dtype):
    i = inputs(N, 1, D, S, G_, dtype)
    P = N + 5
    pool = torch.randn(P, 2, D, S, generator=torch.Generator().manual_seed(3)).cuda()
    pages = torch.randperm(P, generator=torch.Generator().manual_seed(4))[:N].to(torch.int32).cuda()
    pages[N // 2] = -1
    before = pool.clone()
    layer = pool[:, 1]
    one = lambda n: None if i[n] is None else i[n][:, 0].contiguous()  # noqa: E731
    y, out = G.gdn_ssm_step(one("x"), one("dt"), i["A_log"], one("b"), one("c"), layer, pages,
                            D_skip=i["D_skip"], gate=one("gate"), dt_bias=i["dt_bias"],
                            dt_softplus=True, check=True)
    h0 = before[pages.clamp(min=0).long(), 1]
    ry, rl = want({**i, "h0": h0})
    live = (pages >= 0).cpu()
    close(y[live], ry[live, 0], 1)
    assert (y[~live] == 0).all()
    close(out[pages[live].long()], rl[live], 1)
    rest = torch.ones(P, dtype=torch.bool)
    rest[pages[live].long().cpu()] = False
    assert torch.equal(pool[rest], before[rest]) and torch.equal(pool[:, 0], before[:, 0])


def test_step_by_step_is_the_scan():
    i = inputs(3, 20, 40, 16, 1, torch.float32)
    y, last = call(i)
    pool = i["h0"].clone()
    for t in range(20):
        one = lambda n: i[n][:, t].contiguous()  # noqa: E731
        yt, _ = G.gdn_ssm_step(one("x"), one("dt"), i["A_log"], one("b"), one("c"), pool,
                               D_skip=i["D_skip"], gate=one("gate"), dt_bias=i["dt_bias"],
                               dt_softplus=True)
        close(yt, y[:, t].double().cpu(), 20)
    close(pool, last.double().cpu(), 20)


def test_bad_pages_and_offsets_are_recorded():
    i = inputs(3, 1, 16, 16, 1, torch.float32)
    one = lambda n: i[n][:, 0].contiguous()  # noqa: E731
    pool = i["h0"].clone()
    step = lambda pages: G.gdn_ssm_step(one("x"), one("dt"), i["A_log"], one("b"), one("c"), pool,  # noqa: E731
                                        pages, check=True)
    with pytest.raises(G.GdnError) as e:
        step(torch.tensor([0, 7, 2], dtype=torch.int32).cuda())
    assert e.value.status == G.GDN_ERR_DEVICE_CHECK
    i = inputs(1, 20, 16, 16, 1, torch.float32, N=3)
    for cu in ([0, 12, 8, 20], [0, 5, 9, 21], [1, 5, 9, 20], [0, 5, 9, 19], [0, -3, 9, 20]):
        dev = torch.tensor(cu, dtype=torch.int32).cuda()
        for f in (call, call_bwd):
            with pytest.raises(G.GdnError) as e:
                f(i, dev)
            assert e.value.status == G.GDN_ERR_BAD_SEQLENS


def test_no_tokens():
    i = inputs(2, 0, 16, 16, 1, torch.float32)
    y, last = call(i)
    assert y.shape == (2, 0, 16) and torch.equal(last, i["h0"])
    g = call_bwd(i)
    assert torch.equal(g["dh0"], i["d_hT"])
    assert all((g[n] == 0).all() for n in ("dA_log", "dD_skip", "ddt_bias"))


def test_streams_and_graphs():
    """On a stream of its own, and captured twice with one workspace, replayed on new inputs."""
    i = inputs(2, 600, 40, 16, 1, torch.bfloat16)
    y, last = call(i)
    g = call_bwd(i)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, last2 = call(i, stream=side)
    g2 = call_bwd(i, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(last, last2)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    n = max(G.gdn_ssm_workspace_size(2, 600, 40, 16), G.gdn_ssm_bwd_workspace_size(2, 600, 40, 16))
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    graphs, outs = [], []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append((call(i, workspace=ws, check=False), call_bwd(i, workspace=ws, check=False)))
        graphs.append(graph)
    other = inputs(2, 600, 40, 16, 1, torch.bfloat16, seed=9)
    for k, t in other.items():
        i[k].copy_(t)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    y, last = call(other)
    g = call_bwd(other)
    for (fy, fl), gr in outs:
        assert torch.equal(fy, y) and torch.equal(fl, last)
        assert all(torch.equal(gr[k], g[k]) for k in g)
