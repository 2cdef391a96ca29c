"""The scan's backward pass over many tiles on the GPU, against the fp64 oracle: sequences left
whole in CTAs that pass the 16 tiles after which sums move to the workspace many times, CTAs
with several sequences, and segments of more than 128 tokens; slow decays and steps of zero.

Tolerances, relative L2 of a tensor.  A state (or its gradient) remembers K = min(T, 1 / r)
steps, r the smallest delta |A|: its mean over channels and states decides how many errors of
single steps add up.  A step's own errors (exp2, two products, a sum) are below 2^-22, of both
signs once exp2's mean is taken away to 5e-9: 2^-22 sqrt(K) + 5e-9 K, and 2^-20 for delta and
what a result adds.  Products of a state and a gradient have it twice.  Sums over n additions
in a row add 2^-24 n of their terms.  bf16 adds 2^-8."""
import pytest
import torch

import oracle.ssm as O
from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu
WEIGHTS = ("dA_log", "dD_skip", "ddt_bias")


def inputs(N, T, D, S, dtype, groups=1, seed=0):
    g = torch.Generator(device="cuda").manual_seed(100 * T + D + S + seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    rows = lambda *s: r(*s).to(dtype)  # noqa: E731
    i = dict(x=rows(N, T, D), dt=0.5 * rows(N, T, D), A_log=torch.log(torch.arange(1.0, S + 1)).cuda() +
             0.2 * r(D, S), b=rows(N, T, groups, S), c=rows(N, T, groups, S), h0=r(N, D, S),
             D_skip=1 + 0.2 * r(D), gate=rows(N, T, D), dt_bias=r(D) - 3)
    return i, rows(N, T, D), r(N, D, S)


def run(i, d_y, d_last, cu=None, **kw):
    return G.gdn_ssm_bwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], d_y, i["h0"], cu, d_last,
                         D_skip=i["D_skip"], gate=i["gate"], dt_bias=i["dt_bias"],
                         **{"dt_softplus": True, "check": True, **kw})


def memory(i, T):
    """K: at most T, the mean over channels and states of 1 / (delta |A|)."""
    delta = torch.nn.functional.softplus(i["dt"].float() + i["dt_bias"]).mean((0, 1))
    return min(T, float((1 / (delta[:, None] * torch.exp(i["A_log"]))).mean()))


def close(got, ref, tol, what):
    tol = tol + (2.0 ** -8 if got.dtype == torch.bfloat16 else 0)
    err, size = float((got.double() - ref).norm()), float(ref.norm())
    assert err <= tol * size, f"{what}: {err / size:.2e} > {tol:.2e}"


def check(got, ref, i, T, adds):
    K = memory(i, T)
    tol = 2.0 ** -22 * K ** 0.5 + 5e-9 * K + 2.0 ** -20
    for n, t in ref.items():
        close(got[n], t, 2 * tol + (adds * 2.0 ** -24 if n in WEIGHTS else 0), n)


def least_workspace(call, most):
    """The smallest workspace that the call takes (its sequences are left whole then)."""
    ws = torch.zeros(most, dtype=torch.uint8, device="cuda")
    low, high = 0, most // 16
    while high - low > 1:
        mid = (low + high) // 2
        try:
            call(ws[:16 * mid])
            high = mid
        except G.GdnError as e:
            assert e.status == 3
            low = mid
    return ws[:16 * high]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("T", [301, 1500])
def test_whole_sequences(T, S, dtype):
    """2 CTAs of a channel block, one sequence each: 38 or 188 tiles."""
    N, D = 2, 40
    i, d_y, d_last = inputs(N, T, D, S, dtype)
    full = G.gdn_ssm_bwd_workspace_size(N, T, D, S)
    ws = least_workspace(lambda w: run(i, d_y, d_last, workspace=w, check=False), full)
    assert ws.numel() < full
    _, _, ref = O.scan_grads(i, d_y, d_last)
    # 128 tokens of A (16 of the others), a join for each 16 tiles, a CTA's rows of threads
    check(run(i, d_y, d_last, workspace=ws), ref, i, T, 128 + T // 128 + 32 + 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 64])
def test_many_sequences_a_cta(S, dtype):
    """3000 sequences of 5 to 6 tiles: three or four of them a CTA; as rows and packed, the
    packed ones also of ragged lengths, empty ones among them."""
    N, T, D = 3000, 44, 8
    i, d_y, d_last = inputs(N, T, D, S, dtype)
    _, _, ref = O.scan_grads(i, d_y, d_last)
    adds = 128 + 2 + 32 + 912 // 8 + 8
    check(run(i, d_y, d_last), ref, i, T, adds)
    lens = torch.tensor([T - n * 7 % 13 if n % 50 else 0 for n in range(N)])
    at = torch.arange(T)
    mask = (at < lens[:, None]).cuda()
    pack = lambda t: t[mask][None].contiguous()  # noqa: E731
    rows = ("x", "dt", "b", "c", "gate")
    j = {n: pack(t) if n in rows else t for n, t in i.items()}
    cu = torch.cat([torch.zeros(1), lens.cumsum(0)]).to(torch.int32).cuda()
    got = run(j, pack(d_y), d_last, cu)
    _, _, ref = O.scan_grads(i, d_y, d_last, mask.double())
    check(got, {n: pack(t) if t.dim() > 2 and n != "dh0" else t for n, t in ref.items()}, i, T, adds)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_long_segments(S, dtype):
    """8192 tokens, ten channel blocks: cut into some 30 or 43 segments of 192 tokens and more."""
    N, T, D = 1, 8192, 10 * 2048 // S
    i, d_y, d_last = inputs(N, T, D, S, dtype)
    y, last, ref = O.scan_grads(i, d_y, d_last)
    check(run(i, d_y, d_last), ref, i, T, 128 + 3 + 32 + 8 + 8)
    K = memory(i, T)
    tol = 2.0 ** -22 * K ** 0.5 + 5e-9 * K + 2.0 ** -20
    got = G.gdn_ssm_fwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], i["h0"], D_skip=i["D_skip"],
                        gate=i["gate"], dt_bias=i["dt_bias"], dt_softplus=True, check=True)
    close(got[0], y, tol, "y")
    close(got[1], last, tol, "state")


def test_most_sequences_weights():
    """16384 sequences of one token, 18 of them a CTA: the sums over all."""
    N, D, S = 16384, 24, 8
    i, d_y, d_last = inputs(N, 1, D, S, torch.bfloat16)
    _, _, ref = O.scan_grads(i, d_y, d_last)
    adds = 128 + 2 + 32 + 912 // 8 + 8
    check(run(i, d_y, d_last), ref, i, 1, adds)
    flat = {n: t.view(1, N, *t.shape[2:]) if n in ("x", "dt", "b", "c", "gate") else t for n, t in i.items()}
    cu = torch.arange(N + 1, dtype=torch.int32, device="cuda")
    got = run(flat, d_y.view(1, N, D), d_last, cu)
    check({n: got[n] for n in WEIGHTS}, {n: ref[n] for n in WEIGHTS}, i, 1, adds)


@pytest.mark.parametrize("S", [8, 64])
def test_long_sums_of_equal_terms_in_one_cta(S):
    """3449 tokens of equal gradients in one CTA: 16 tiles' terms of a thread (two a tile for S =
    8), 27 joins, up to 32 rows of threads: 92 additions in a row at most."""
    N, T, D = 1, 3449, 8
    i, d_y, d_last = inputs(N, T, D, S, torch.float32)
    i["x"].fill_(0.3)
    d_y.fill_(0.7)
    i["gate"] = None
    ws = least_workspace(lambda w: run(i, d_y, d_last, workspace=w, check=False),
                         G.gdn_ssm_bwd_workspace_size(N, T, D, S))
    got = run(i, d_y, d_last, workspace=ws)
    want = T * float(i["x"][0, 0, 0]) * float(d_y[0, 0, 0])
    assert (got["dD_skip"].double() - want).abs().max() <= 92 * 2.0 ** -24 * want


def slow(T, D, S, low, high, seed=0):
    """Steps and rates with delta |A| log2(e) spread over [low, high], positive terms."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda *s: torch.rand(*s, generator=g, device="cuda")  # noqa: E731
    rate = low * (high / low) ** 0.5 / 1.4426950408889634
    spread = (high / low) ** 0.5
    i = dict(x=0.5 + u(1, T, D), dt=spread ** (u(1, T, D) - 0.5), A_log=torch.log(rate * spread ** (u(D, S) - 0.5)),
             b=0.5 + u(1, T, 1, S), c=0.5 + u(1, T, 1, S), h0=None, D_skip=None, gate=None, dt_bias=None)
    return i, 0.5 + u(1, T, D), 0.5 + u(1, D, S)


def forward(i, **kw):
    return G.gdn_ssm_fwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], check=True, **kw)


@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("whole", [False, True])
def test_slow_decays(S, whole):
    """K = 500 to 3000 steps remembered, all terms of one sign: nothing cancels."""
    T, D = 4000, 16
    i, d_y, d_last = slow(T, D, S, 2.0 ** -10, 2.0 ** -8.5, S)
    y, last, ref = O.scan_grads(i, d_y, d_last, softplus=False)
    args = dict(workspace=torch.zeros(256, dtype=torch.uint8, device="cuda")) if whole else {}
    got, state = forward(i, **args)
    K = min(T, 1.4426950408889634 * 2.0 ** 9.25)
    tol = 2.0 ** -22 * K ** 0.5 + 5e-9 * K + 2.0 ** -20
    close(got, y, tol, "y")
    close(state, last, tol, "state")
    back = lambda ws: run(i, d_y, d_last, dt_softplus=False, workspace=ws, check=ws is None)  # noqa: E731
    ws = least_workspace(back, G.gdn_ssm_bwd_workspace_size(1, T, D, S)) if whole else None
    grads = back(ws)
    for n in ("dx", "ddt", "db", "dc", "dA_log"):
        close(grads[n], ref[n], 2 * tol + 200 * 2.0 ** -24, n)


@pytest.mark.parametrize("S", [8, 16, 32, 64])
def test_mean_of_exp2_is_taken_away(S):
    """delta |A| log2(e) spread over 2^-7 to 2^-5, where the hardware's exp2 is 2.2e-8 low on
    average: states, and the gradient of the first one, are not off by half of what that would
    make of them, on average over channels and states."""
    T, D = 400, 64
    i, d_y, d_last = slow(T, D, S, 2.0 ** -7, 2.0 ** -5, 7 * S)
    _, last, ref = O.scan_grads(i, d_y, d_last, softplus=False)
    # the same with every exp(delta A) lower by 2.2e-8: delta A more by that
    delta, A = i["dt"].double(), -torch.exp(i["A_log"].double())
    h, product = torch.zeros_like(last), torch.ones_like(last)
    for t in range(T):
        a = torch.exp(delta[:, t, :, None] * A) * (1 - 2.2e-8)
        h = a * h + (delta[:, t] * i["x"][:, t].double())[..., None] * i["b"].double()[:, t]
    drop = float(((h - last) / last).mean())
    assert -3e-6 < drop < -4e-7
    for ws in (None, torch.zeros(256, dtype=torch.uint8, device="cuda")):
        _, state = forward(i, workspace=ws)
        off = float(((state.double() - last) / last).mean())
        assert abs(off) < -drop / 2, (off, drop)
    # a first state's gradient, through 100 tokens: 2.2e-6 of exp2's mean
    j, d_y, d_last = slow(100, D, S, 2.0 ** -7, 2.0 ** -5, 7 * S)
    d_y.zero_()
    ws = least_workspace(lambda w: run(j, d_y, d_last, dt_softplus=False, workspace=w, check=False),
                         G.gdn_ssm_bwd_workspace_size(1, 100, D, S))
    _, _, ref = O.scan_grads(j, d_y, d_last, softplus=False)
    got = run(j, d_y, d_last, dt_softplus=False, workspace=ws)["dh0"]
    assert abs(float(((got.double() - ref["dh0"]) / ref["dh0"]).mean())) < 1.1e-6


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("softplus", [False, True])
def test_steps_of_zero_change_nothing(S, softplus, dtype):
    """A token with a large step, then steps of zero to the end of the tile and beyond: the
    states, and the gradients that come back through them, are those of the one token alone,
    bit for bit; where the backward pass cuts the sequence, which takes dh0's factor from the
    sum of delta over a segment, within what the two exponentials may differ: each off by 2^-22
    and its argument's rounding, |delta A| 2^-24, and one of them lifted by 3.1e-8."""
    D = 24
    none = -1000.0 if softplus else 0.0
    for T in (2, 8, 13, 32, 50, 700):
        i, d_y, d_last = inputs(2, T, D, S, dtype)
        i["gate"] = i["dt_bias"] = None
        i["dt"].fill_(none)
        i["dt"][:, 0] = 0.5
        d_y.zero_()
        one = {n: t[:, :1].contiguous() if n in ("x", "dt", "b", "c") else t for n, t in i.items()}
        f = lambda j: G.gdn_ssm_fwd(j["x"], j["dt"], j["A_log"], j["b"], j["c"], j["h0"], D_skip=j["D_skip"],  # noqa: E731
                                    dt_softplus=softplus, check=True)
        assert torch.equal(f(i)[1], f(one)[1])
        back = lambda j, d, **kw: run(j, d, d_last, dt_softplus=softplus, **kw)["dh0"]  # noqa: E731
        want = back(one, d_y[:, :1].contiguous())
        ws = least_workspace(lambda w: back(i, d_y, workspace=w, check=False),
                             G.gdn_ssm_bwd_workspace_size(2, T, D, S))
        ws.zero_()
        assert torch.equal(back(i, d_y, workspace=ws), want), T
        arg = (0.97407698 if softplus else 0.5) * torch.exp(i["A_log"])   # (softplus(0.5))
        far = 2 * (2.0 ** -22 + arg * 2.0 ** -24) + 3.1e-8
        assert ((back(i, d_y) - want).abs() <= far * want.abs() + 2.0 ** -125).all(), T
        i["dt"].fill_(none)
        assert torch.equal(f(i)[1], i["h0"])
        assert torch.equal(back(i, d_y), d_last)
        pool = i["h0"].clone()
        G.gdn_ssm_step(i["x"][:, 0].contiguous(), i["dt"][:, 0].contiguous(), i["A_log"], i["b"][:, 0].contiguous(),
                       i["c"][:, 0].contiguous(), pool, dt_softplus=softplus)
        assert torch.equal(pool, i["h0"])
