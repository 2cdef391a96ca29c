"""Short convolution (gdn_conv_fwd, gdn_conv_bwd, gdn_conv_step) on the GPU against the fp64
oracle.  Tolerances, relative L2 of a tensor: an output is a handful of fp32 operations
and one sigmoid (2^-21 together); sums over T tokens are taken in blocks, at most some 200
additions in a row, each off by 2^-24 of the sum of magnitudes (a hundred times the sum
for random terms of 10^4 tokens: 2^-24 200 sqrt(T) is allowed).  bf16 adds 2^-8."""
import pytest
import torch

import oracle.ssm as O
from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


def inputs(B, T, C, K, dtype, N=None, seed=0, init=True, bias=True):
    g = torch.Generator().manual_seed(100 * T + C + K + seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    N = B if N is None else N
    i = dict(x=r(B, T, C).to(dtype), w=r(C, K) / K ** 0.5, bias=0.1 * r(C) if bias else None,
             x_prev=r(N, K - 1, C).to(dtype) if init else None, d_y=r(B, T, C).to(dtype),
             d_tail=r(N, K - 1, C).to(dtype))
    return {n: None if t is None else t.cuda() for n, t in i.items()}


def close(got, ref, tol, what=""):
    tol = tol + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    err, size = float((got.detach().cpu().double() - ref).norm()), float(ref.norm())
    assert err <= tol * size + 1e-30, f"{what}: {err / max(size, 1e-300):.2e} > {tol:.2e}"


def check(i, cu=None, silu=True, tail=True):
    dev = None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda()
    T = i["x"].shape[1]
    y, xt = G.gdn_conv_fwd(i["x"], i["w"], i["bias"], i["x_prev"], dev, silu=silu, check=True)
    ry, rt = O.conv(O._d(i["x"]), O._d(i["w"]), O._d(i["bias"]), O._d(i["x_prev"]), cu, silu)
    close(y, ry, 2.0 ** -20, "y")
    assert torch.equal(xt.cpu().double(), rt)
    d_tail = i["d_tail"] if tail else None
    g = G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"], i["x_prev"], dev, d_tail, silu=silu,
                       check=True)
    ref = O.grads(O.conv, {n: i[n] for n in ("x", "w", "bias", "x_prev")}, (i["d_y"], d_tail),
                  cu=cu, silu=silu)
    for n, t in ref.items():
        if t.numel():
            tol = 2.0 ** -20 if n in ("x", "x_prev") else 2.0 ** -20 + 200 * T ** 0.5 * 2.0 ** -24
            close(g["d" + n], t, tol, "d" + n)
    return y, xt, g


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 2, 3, 4])
@pytest.mark.parametrize("B,T,C", [(1, 1, 8), (2, 3, 16), (3, 17, 40), (1, 64, 264), (2, 100, 24),
                                   (1, 1000, 520)])
def test_dense(B, T, C, K, dtype):
    check(inputs(B, T, C, K, dtype))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("lens", [[5], [0, 3, 0, 0, 40, 1], [1] * 40, [2, 1, 3, 2, 1, 64, 9], [0, 9, 0],
                                  [200, 8, 16], [7, 8, 9, 1, 8, 0, 65]])
def test_packed(lens, dtype):
    cu = [sum(lens[:k]) for k in range(len(lens) + 1)]
    for K in (2, 4):
        check(inputs(1, cu[-1], 40, K, dtype, N=len(lens)), cu)


@pytest.mark.parametrize("silu", [False, True])
def test_without_parts(silu):
    i = inputs(2, 50, 32, 4, torch.float32, init=False, bias=False)
    y, tail, g = check(i, silu=silu, tail=False)
    assert g["dbias"] is None and g["dx_prev"] is None


def test_same_as_the_fixed_prologue():
    i = inputs(2, 90, 64, 4, torch.bfloat16, bias=False)
    y, _ = G.gdn_conv_fwd(i["x"], i["w"], None, i["x_prev"])
    other = G.gdn_conv_silu(i["x"], i["w"], i["x_prev"])
    close(y, other.double().cpu(), 2.0 ** -20)


def test_slices_of_projections():
    i = inputs(2, 70, 48, 4, torch.bfloat16)
    wide = torch.full((2, 70, 96), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[..., 24:72] = i["x"]
    x = wide[..., 24:72]
    for a, b in zip(G.gdn_conv_fwd(x, i["w"], i["bias"]), G.gdn_conv_fwd(i["x"], i["w"], i["bias"])):
        assert torch.equal(a, b)
    a = G.gdn_conv_bwd(x, i["w"], i["d_y"], i["bias"])
    b = G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"])
    assert all(a[n] is None or torch.equal(a[n], b[n]) for n in a)


def test_not_finite_values_stay_behind():
    i = inputs(1, 40, 16, 4, torch.float32, N=2)
    cu = torch.tensor([0, 21, 40], dtype=torch.int32).cuda()
    f = lambda x: G.gdn_conv_fwd(x, i["w"], i["bias"], i["x_prev"], cu)[0]  # noqa: E731
    b = lambda x, d: G.gdn_conv_bwd(x, i["w"], d, i["bias"], i["x_prev"], cu)["dx"]  # noqa: E731
    y, dx = f(i["x"]), b(i["x"], i["d_y"])
    x = i["x"].clone()
    x[0, 20, 3] = float("nan")   # the last token of the first sequence
    y2 = f(x)
    same = torch.ones(40, 16, dtype=torch.bool)
    same[20, 3] = False
    assert torch.equal(y2[0].cpu()[same], y[0].cpu()[same])
    d = i["d_y"].clone()
    d[0, 21, 3] = float("inf")   # the first of the second
    dx2 = b(i["x"], d)
    same[20, 3] = True
    same[21, 3] = False
    assert torch.equal(dx2[0].cpu()[same], dx[0].cpu()[same])


def test_long_sums_of_equal_terms():
    i = inputs(1, 30000, 8, 4, torch.float32, init=False)
    i["x"].fill_(0.3)
    i["d_y"].fill_(0.7)
    g = G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"], silu=False)
    want = 30000 * float(i["d_y"][0, 0, 0])
    # 64 tokens, a CTA's rows of threads (256), its segments and the CTAs: 1000 in a row at most
    assert (g["dbias"].double() - want).abs().max() <= 400 * 2.0 ** -24 * want


def test_results_are_reproducible_on_streams_and_in_graphs():
    i = inputs(2, 700, 136, 4, torch.bfloat16)
    run = lambda **kw: (*G.gdn_conv_fwd(i["x"], i["w"], i["bias"], i["x_prev"], **kw),  # noqa: E731
                        *G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"], i["x_prev"],
                                        **kw).values())
    a = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = run(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c = run()
    graph.replay()
    torch.cuda.synchronize()
    for other in (b, c):
        assert all(torch.equal(u, v) for u, v in zip(a, other))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 2, 4])
def test_step_by_step_is_the_convolution(K, dtype):
    i = inputs(3, 9, 40, K, dtype)
    y, tail = G.gdn_conv_fwd(i["x"], i["w"], i["bias"], i["x_prev"])
    P = 6
    pool = torch.randn(P, 2, K - 1, 40, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    pages = torch.tensor([4, 0, 3], dtype=torch.int32).cuda()
    pool[pages.long(), 1] = i["x_prev"]
    before = pool.clone()
    for t in range(9):
        yt, _ = G.gdn_conv_step(i["x"][:, t].contiguous(), i["w"], pool[:, 1], i["bias"], pages,
                                check=True)
        assert torch.equal(yt, y[:, t])
    assert torch.equal(pool[pages.long(), 1], tail)
    rest = [1, 2, 5]
    assert torch.equal(pool[rest], before[rest]) and torch.equal(pool[:, 0], before[:, 0])


def test_padded_and_bad_pages():
    i = inputs(3, 1, 16, 4, torch.float32)
    x = i["x"][:, 0].contiguous()
    pool = i["x_prev"].clone()
    y, _ = G.gdn_conv_step(x, i["w"], pool, i["bias"], torch.tensor([-1, 1, -1], dtype=torch.int32).cuda(),
                           check=True)
    assert (y[[0, 2]] == 0).all() and torch.equal(pool[[0, 2]], i["x_prev"][[0, 2]])
    with pytest.raises(G.GdnError) as e:
        G.gdn_conv_step(x, i["w"], pool, i["bias"], torch.tensor([0, 3, 1], dtype=torch.int32).cuda(),
                        check=True)
    assert e.value.status == G.GDN_ERR_DEVICE_CHECK


def test_bad_offsets_write_nothing():
    i = inputs(1, 20, 16, 4, torch.float32, N=3)
    for cu in ([0, 5, 9, 21], [1, 5, 9, 20], [0, 5, 9, 19], [0, -3, 9, 20], [0, 12, 8, 20]):
        dev = torch.tensor(cu, dtype=torch.int32).cuda()
        for f in (lambda **k: G.gdn_conv_fwd(i["x"], i["w"], i["bias"], i["x_prev"], dev, **k),
                  lambda **k: G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"], i["x_prev"], dev, **k)):
            with pytest.raises(G.GdnError) as e:
                f(check=True)
            assert e.value.status == G.GDN_ERR_BAD_SEQLENS
    y = torch.full_like(i["x"], 7.0)
    G.gdn_conv_fwd(i["x"], i["w"], i["bias"], None, torch.tensor([0, 5, 9, 19], dtype=torch.int32).cuda(), y=y)
    assert (y[0, 9:] == 7).all() and (y[0, :9] != 7).all()


def test_no_tokens():
    i = inputs(2, 0, 16, 4, torch.float32)
    y, tail = G.gdn_conv_fwd(i["x"], i["w"], i["bias"], i["x_prev"])
    assert torch.equal(tail, i["x_prev"])
    g = G.gdn_conv_bwd(i["x"], i["w"], i["d_y"], i["bias"], i["x_prev"], None, i["d_tail"])
    assert torch.equal(g["dx_prev"], i["d_tail"]) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()
