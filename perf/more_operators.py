"""Cases of the selective scan, its short convolution, and the q/k norm with rotation.

``run`` computes one pass of a case: with ``own`` false in elementary torch
operations in 32 bits, with ``own`` true through the library's entry points.

The operators:

- selective state space scan, h_t = exp(delta_t A) h_{t-1} + delta_t x_t b_t and
  y_t = (c_t . h_t + D x_t) silu(gate_t), with delta = softplus(dt + dt_bias) and
  A = -exp(A_log): x, dt, gate [B, T, D], b, c [B, T, G, S], A_log [D, S]; prompts
  (forward; packed with cu_seqlens), training (backward), single tokens on a pool
  of state pages (step);
- short causal depthwise convolution with a bias and SiLU: forward (packed sequences
  too), backward, single tokens on a pool of pages that hold the last inputs;
- norm of each head of q and k (root mean square with a weight, or l2), then the
  rotation of its first R elements by the token's position, forward and backward.
"""
import math
import random

import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # a short prompt on a narrow layer: latency (the tiny_fp32 workload's width and length)
        dict(name="ssm_fwd_tiny_fp32", op="ssm_fwd", dtype="fp32", B=1, T=256, D=64, S=16, G=1,
             num_seqs=0, lens=0, init=False, gate=False),
        # a training or prefill batch (the conv_hymo_bf16 workload's shape)
        dict(name="ssm_fwd_hymo_bf16", op="ssm_fwd", dtype="bf16", B=4, T=4096, D=1280, S=16, G=1,
             num_seqs=0, lens=0, init=False, gate=True),
        # prefill of one long document: few channels, a long axis (the long_bf16 workload's shape)
        dict(name="ssm_fwd_long_bf16", op="ssm_fwd", dtype="bf16", B=1, T=65536, D=2048, S=16, G=1,
             num_seqs=0, lens=0, init=False, gate=True),
        # training step of a small batch in fp32: odd length, two groups, the pages' 32 states
        dict(name="ssm_bwd_small_fp32", op="ssm_bwd", dtype="fp32", B=2, T=333, D=96, S=32, G=2,
             num_seqs=0, lens=0, init=True, gate=True),
        # training step (the conv_hymo_bf16 workload's shape)
        dict(name="ssm_bwd_hymo_bf16", op="ssm_bwd", dtype="bf16", B=4, T=4096, D=1280, S=16, G=1,
             num_seqs=0, lens=0, init=False, gate=True),
        # generation for a full server (decode_hymo_bf16's number of sequences), states in a pool
        dict(name="ssm_step_full_bf16", op="ssm_step", dtype="bf16", N=1024, D=1280, S=16, G=1,
             P=1280, gate=True),
        # the convolution over packed prompts of ragged lengths (varlen_bf16's lengths)
        dict(name="conv_fwd_varlen_bf16", op="conv_fwd", dtype="bf16", B=1, T=0, C=1280, K=4,
             num_seqs=32, lens=8192, init=True, silu=True),
        # training step of the convolution (the conv_hymo_bf16 workload's shape)
        dict(name="conv_bwd_hymo_bf16", op="conv_bwd", dtype="bf16", B=4, T=4096, C=1280, K=4,
             num_seqs=0, lens=0, init=False, silu=True),
        # generation for a handful of users: latency
        dict(name="conv_step_few_bf16", op="conv_step", dtype="bf16", N=8, C=1280, K=4, P=64,
             silu=True),
        # q and k of a training or prefill batch (the hymo_bf16 workload's shape), slices of a projection
        dict(name="qk_fwd_hymo_bf16", op="qk_fwd", dtype="bf16", B=8, T=4096, Hq=16, Hk=16, D=64,
             R=64, l2=False, inter=False),
        # training step of the wide layer (the wide_bf16 workload's shape), half of a head rotated
        dict(name="qk_bwd_wide_bf16", op="qk_bwd", dtype="bf16", B=4, T=8192, Hq=16, Hk=16, D=128,
             R=64, l2=False, inter=True),
        # one token for each of 128 users at far positions, shared key heads: latency
        dict(name="qk_token_bf16", op="qk_fwd", dtype="bf16", B=128, T=1, Hq=16, Hk=4, D=128, R=128,
             l2=False, inter=False),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def _sequences_of(rng, most, longest):
    """Dense rows or packed sequences of at most `most` tokens together."""
    if rng.random() < 0.4:
        n = _log(rng, 1, 24)
        return dict(B=1, T=0, num_seqs=n, lens=_log(rng, 4, max(4, min(longest, most // n))))
    B = _log(rng, 1, 16)
    return dict(B=B, T=_log(rng, 1, max(1, min(longest, most // B))), num_seqs=0, lens=0)


def draw(rng):
    op = rng.choice(["ssm_fwd", "ssm_fwd", "ssm_bwd", "ssm_bwd", "ssm_step", "conv_fwd", "conv_bwd",
                     "conv_step", "qk_fwd", "qk_bwd"])
    dtype = rng.choice(["fp32", "bf16", "bf16"])
    if op in ("ssm_fwd", "ssm_bwd", "ssm_step"):
        S, G = rng.choice([8, 16, 16, 32, 64]), rng.choice([1, 1, 2, 4])
        D = 8 * G * _log(rng, 1, 512 // G)
        if op == "ssm_step":
            N = _log(rng, 1, 1024)
            N = max(1, min(N, (32 << 20) // (D * S)))
            return dict(op=op, dtype=dtype, N=N, D=D, S=S, G=G, P=N + _log(rng, 1, 256),
                        gate=rng.random() < 0.5)
        most = max(16, ((1 << 30) if op == "ssm_fwd" else (1 << 28)) // (D * S))
        return dict(op=op, dtype=dtype, D=D, S=S, G=G, init=rng.random() < 0.5,
                    gate=rng.random() < 0.5, **_sequences_of(rng, most, 16384))
    if op in ("conv_fwd", "conv_bwd", "conv_step"):
        C, K, silu = 8 * _log(rng, 1, 512), rng.choice([2, 3, 4, 4]), rng.random() < 0.7
        if op == "conv_step":
            N = _log(rng, 1, 1024)
            return dict(op=op, dtype=dtype, N=N, C=C, K=K, P=N + _log(rng, 1, 256), silu=silu)
        return dict(op=op, dtype=dtype, C=C, K=K, init=rng.random() < 0.5, silu=silu,
                    **_sequences_of(rng, max(64, (64 << 20) // C), 32768))
    D = rng.choice([32, 64, 80, 96, 128, 256])
    Hq = _log(rng, 1, 32)
    Hk = rng.choice([h for h in (1, 2, 4, 8, 16, 32, Hq) if h <= Hq and Hq % h == 0])
    B = _log(rng, 1, 128)
    return dict(op=op, dtype=dtype, B=B, T=_log(rng, 1, max(1, (64 << 20) // (B * (Hq + Hk) * D))),
                Hq=Hq, Hk=Hk, D=D, R=rng.choice([D, D // 2, 16, 0]), l2=rng.random() < 0.3,
                inter=rng.random() < 0.5)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _lens(case):
    r = random.Random(case["num_seqs"] * 100003 + case["lens"])
    return [r.randint(max(1, case["lens"] // 64), case["lens"]) for _ in range(case["num_seqs"])]


def _tokens(case):
    return sum(_lens(case)) if case["num_seqs"] else case["B"] * case["T"]


def _seq(case):
    """(T, sequences, cu_seqlens or None) of a case."""
    if not case["num_seqs"]:
        return case["T"], case["B"], None
    off = [0]
    for n in _lens(case):
        off.append(off[-1] + n)
    return off[-1], case["num_seqs"], torch.tensor(off, dtype=torch.int32, device="cuda")


def _ssm_weights(case, rand):
    """A_log = log(1 .. S) with some spread (the usual start, after some training); dt_bias with
    softplus(dt_bias) spread over the logarithm of [1e-3, 0.1]."""
    D, S = case["D"], case["S"]
    dt0 = torch.exp(torch.rand(D, generator=rand.gen, device="cuda") * math.log(100.0) + math.log(1e-3))
    return dict(A_log=torch.log(torch.arange(1.0, S + 1, device="cuda")) + 0.2 * rand(D, S),
                dt_bias=dt0 + torch.log(-torch.expm1(-dt0)), D_skip=1.0 + 0.2 * rand(D))


def _randn(seed):
    g = _gen(seed)

    def rand(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    rand.gen = g
    return rand


def _ssm_inputs(case, seed):
    rand, dt = _randn(seed), _DT[case["dtype"]]
    B, D, S, G = case["B"], case["D"], case["S"], case["G"]
    T, N, cu = _seq(case)
    s = dict(case=case, cu=cu, **_ssm_weights(case, rand))
    s["x"] = rand(B, T, D).to(dt)
    s["dt"] = (0.5 * rand(B, T, D)).to(dt)
    # b and c are slices of one projection, the gate one of the layer's input projection
    bc = rand(B, T, 2 * G * S).to(dt)
    s["b"], s["c"] = (t.view(B, T, G, S) for t in (bc[..., :G * S], bc[..., G * S:]))
    s["gate"] = rand(B, T, 2 * D).to(dt)[..., D:] if case["gate"] else None
    s["h0"] = rand(N, D, S) if case["init"] else None
    if case["op"] == "ssm_bwd":
        s["d_y"] = rand(B, T, D).to(dt)
        s["d_hT"] = rand(N, D, S) if case["init"] else None
    return s


def _ssm_step_inputs(case, seed):
    rand, dt = _randn(seed), _DT[case["dtype"]]
    N, D, S, G, P = case["N"], case["D"], case["S"], case["G"], case["P"]
    s = dict(case=case, **_ssm_weights(case, rand), x=rand(N, D).to(dt), dt=(0.5 * rand(N, D)).to(dt),
             b=rand(N, G, S).to(dt), c=rand(N, G, S).to(dt),
             gate=rand(N, D).to(dt) if case["gate"] else None, pool=rand(P, D, S))
    s["pages"] = torch.randperm(P, generator=rand.gen, device="cuda")[:N].to(torch.int32)
    return s


def _conv_inputs(case, seed):
    rand, dt = _randn(seed), _DT[case["dtype"]]
    B, C, K = case["B"], case["C"], case["K"]
    T, N, cu = _seq(case)
    s = dict(case=case, cu=cu, x=rand(B, T, C).to(dt), w=rand(C, K) / K ** 0.5, bias=0.1 * rand(C),
             x_prev=rand(N, K - 1, C).to(dt) if case["init"] else None)
    if case["op"] == "conv_bwd":
        s["d_y"] = rand(B, T, C).to(dt)
    return s


def _conv_step_inputs(case, seed):
    rand, dt = _randn(seed), _DT[case["dtype"]]
    N, C, K, P = case["N"], case["C"], case["K"], case["P"]
    s = dict(case=case, x=rand(N, C).to(dt), w=rand(C, K) / K ** 0.5, bias=0.1 * rand(C),
             pool=rand(P, K - 1, C).to(dt))
    s["pages"] = torch.randperm(P, generator=rand.gen, device="cuda")[:N].to(torch.int32)
    return s


def _qk_inputs(case, seed):
    rand, dt = _randn(seed), _DT[case["dtype"]]
    B, T, Hq, Hk, D, R = (case[n] for n in ("B", "T", "Hq", "Hk", "D", "R"))
    p = rand(B, T, (Hq + 2 * Hk) * D).to(dt)   # the projection to q, k and v
    s = dict(case=case, q=p[..., :Hq * D].view(B, T, Hq, D),
             k=p[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D),
             q_weight=None if case["l2"] else 1.0 + 0.2 * rand(D),
             k_weight=None if case["l2"] else 1.0 + 0.2 * rand(D), q_scale=D ** -0.5, positions=None,
             inv_freq=None)
    if R:
        # positions of prompts that continue contexts of up to 128k tokens
        start = torch.randint(0, 131072, (B, 1), generator=rand.gen, device="cuda")
        s["positions"] = (start + torch.arange(T, device="cuda")).to(torch.int32)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()
    if case["op"] == "qk_bwd":
        s["d_q"], s["d_k"] = rand(B, T, Hq, D).to(dt), rand(B, T, Hk, D).to(dt)
    return s


def prepare(case, seed):
    return {"ssm_fwd": _ssm_inputs, "ssm_bwd": _ssm_inputs, "ssm_step": _ssm_step_inputs,
            "conv_fwd": _conv_inputs, "conv_bwd": _conv_inputs, "conv_step": _conv_step_inputs,
            "qk_fwd": _qk_inputs, "qk_bwd": _qk_inputs}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------
def _padded(s, *tensors):
    """fp32 [N, T, ...] of each tensor (zero rows past a sequence's end), the mask of the rows that
    are tokens [N, T], and the way back to the tensors' own rows."""
    if s["cu"] is None:
        t = next(x for x in tensors if x is not None)
        inside = torch.ones(t.shape[:2], dtype=torch.bool, device=t.device)
        return [None if x is None else x.float() for x in tensors], inside, lambda y: y
    cu = s["cu"].long()
    lens = _lens(s["case"])
    at = torch.arange(max(lens), device=cu.device)
    inside = at < (cu[1:] - cu[:-1])[:, None]
    idx = torch.where(inside, cu[:-1, None] + at, 0)

    def pick(x):
        y = x[0].float()[idx]
        return y * inside.view(*inside.shape, *[1] * (y.dim() - 2))

    return [None if x is None else pick(x) for x in tensors], inside, lambda y: y[inside][None]


def _silu(z):
    return z / (1 + torch.exp(-z))


def _softplus(v):
    """log(1 + exp(v)) without overflow."""
    return v.clamp(min=0) + torch.log1p(torch.exp(-v.abs()))


def _chunks(t, L):
    """[N, T, ...] as [N, chunks, L, ...], zeros behind the end."""
    N, T = t.shape[:2]
    n = max(1, -(-T // L))
    out = t.new_zeros(N, n * L, *t.shape[2:])
    out[:, :T] = t
    return out.view(N, n, L, *t.shape[2:])


def _plain_scan(s):
    """(terms, h of every chunk's start, last h) of the padded scan: chunks of about sqrt(T) tokens
    side by side, from zero; then their starts in order."""
    c = s["case"]
    G, S = c["G"], c["S"]
    Dg = c["D"] // G
    (x, dt, b, cc, gate), inside, back = _padded(s, s["x"], s["dt"], s["b"], s["c"], s["gate"])
    T = x.shape[1]
    L = max(1, math.isqrt(T))
    v = dt + s["dt_bias"]
    delta = _softplus(v) * inside[..., None]
    A = -torch.exp(s["A_log"])
    heads = lambda t: _chunks(t, L).reshape(t.shape[0], -1, L, G, Dg)  # noqa: E731
    d, u = heads(delta), heads(delta * x)
    bc, ccc = _chunks(b, L), _chunks(cc, L)
    Ag = A.view(G, Dg, S)
    h = x.new_zeros(*d.shape[:2], G, Dg, S)
    for i in range(L):
        h = h * torch.exp(d[:, :, i, ..., None] * Ag) + u[:, :, i, ..., None] * bc[:, :, i, :, None]
    decay = torch.exp(d.sum(2)[..., None] * Ag)
    at = x.new_zeros(x.shape[0], G, Dg, S) if s["h0"] is None else s["h0"].view(-1, G, Dg, S)
    starts = []
    for j in range(h.shape[1]):
        starts.append(at)
        at = at * decay[:, j] + h[:, j]
    terms = dict(x=x, v=v, delta=delta, gate=gate, d=d, u=u, b=bc, c=ccc, A=A, Ag=Ag, L=L, T=T, Dg=Dg,
                 inside=inside, back=back, decay=decay)
    return terms, torch.stack(starts, 1), at


def _rows(y, t):
    """[N, chunks, L, G, Dg] to [N, T, D]."""
    return y.reshape(y.shape[0], -1, y.shape[-2] * y.shape[-1])[:, :t["T"]]


def _plain_ssm_fwd(s):
    t, h, last = _plain_scan(s)
    y = torch.empty_like(t["u"])
    for i in range(t["L"]):
        h = h * torch.exp(t["d"][:, :, i, ..., None] * t["Ag"]) + \
            t["u"][:, :, i, ..., None] * t["b"][:, :, i, :, None]
        y[:, :, i] = (h * t["c"][:, :, i, :, None]).sum(-1)
    y = _rows(y, t) + s["D_skip"] * t["x"]
    if t["gate"] is not None:
        y = y * _silu(t["gate"])
    D, S = s["A_log"].shape
    return t["back"](y).to(s["x"].dtype), last.reshape(-1, D, S)


def _plain_ssm_bwd(s):
    t, h, _ = _plain_scan(s)
    c, (D, S), L = s["case"], s["A_log"].shape, t["L"]
    (dy,), _, back = _padded(s, s["d_y"])
    ds = dy if t["gate"] is None else dy * _silu(t["gate"])
    shape = t["u"].shape
    dsc = _chunks(ds, L).reshape(shape)
    # the state before each token, and y's sum (for the gate's gradient)
    before, sums = [], torch.empty_like(t["u"])
    for i in range(L):
        before.append(h)
        h = h * torch.exp(t["d"][:, :, i, ..., None] * t["Ag"]) + \
            t["u"][:, :, i, ..., None] * t["b"][:, :, i, :, None]
        sums[:, :, i] = (h * t["c"][:, :, i, :, None]).sum(-1)
    before.append(h)
    # the gradient that each chunk receives at its end: the chunks from zero, then in order
    g = torch.zeros_like(h)
    for i in range(L - 1, -1, -1):
        g = (g + dsc[:, :, i, ..., None] * t["c"][:, :, i, :, None]) * \
            torch.exp(t["d"][:, :, i, ..., None] * t["Ag"])
    at = torch.zeros_like(g[:, 0]) if s["d_hT"] is None else s["d_hT"].view(g[:, 0].shape)
    ends = []
    for j in range(g.shape[1] - 1, -1, -1):
        ends.append(at)
        at = at * t["decay"][:, j] + g[:, j]
    dh0, g = at, torch.stack(ends[::-1], 1)
    bg, dd = torch.empty_like(t["u"]), torch.empty_like(t["u"])
    db, dc = torch.empty_like(t["b"]), torch.empty_like(t["b"])
    dA = torch.zeros_like(t["Ag"])
    for i in range(L - 1, -1, -1):
        g = g + dsc[:, :, i, ..., None] * t["c"][:, :, i, :, None]
        dc[:, :, i] = (dsc[:, :, i, ..., None] * before[i + 1]).sum(-2)
        db[:, :, i] = (t["u"][:, :, i, ..., None] * g).sum(-2)
        bg[:, :, i] = (g * t["b"][:, :, i, :, None]).sum(-1)
        g = g * torch.exp(t["d"][:, :, i, ..., None] * t["Ag"])
        w = g * before[i]
        dd[:, :, i] = (w * t["Ag"]).sum(-1)
        dA += (w * t["d"][:, :, i, ..., None]).sum((0, 1))
    x, bg = t["x"], _rows(bg, t)
    ddt = (x * bg + _rows(dd, t)) / (1 + torch.exp(-t["v"])) * t["inside"][..., None]
    dt_ = s["x"].dtype
    flat = lambda y: y.reshape(y.shape[0], -1, c["G"], S)[:, :t["T"]]  # noqa: E731
    out = {"dx": back(t["delta"] * bg + s["D_skip"] * ds).to(dt_), "ddt": back(ddt).to(dt_),
           "db": back(flat(db)).to(dt_), "dc": back(flat(dc)).to(dt_),
           "dA_log": dA.view(D, S) * t["A"], "dD_skip": (ds * x).sum((0, 1)),
           "ddt_bias": ddt.sum((0, 1)), "dh0": dh0.reshape(-1, D, S)}
    if t["gate"] is not None:
        sig = 1 / (1 + torch.exp(-t["gate"]))
        out["dgate"] = back(dy * (_rows(sums, t) + s["D_skip"] * x) * sig *
                            (1 + t["gate"] * (1 - sig))).to(dt_)
    return out


def _plain_ssm_step(s):
    G, S = s["case"]["G"], s["case"]["S"]
    idx = s["pages"].long()
    x, b, c = (s[n].float() for n in "xbc")
    delta = _softplus(s["dt"].float() + s["dt_bias"])
    N, D = x.shape
    h = s["pool"][idx].view(N, G, D // G, S)
    h = h * torch.exp(delta[..., None] * -torch.exp(s["A_log"])).view(h.shape) + \
        (delta * x).view(N, G, D // G, 1) * b[:, :, None]
    s["pool"][idx] = h.view(N, D, S)
    y = (h * c[:, :, None]).sum(-1).view(N, D) + s["D_skip"] * x
    if s["gate"] is not None:
        y = y * _silu(s["gate"].float())
    return y.to(s["x"].dtype), s["pool"]


def _plain_conv_z(s):
    """(inputs behind their prefix [N, T + K - 1, C], the sum z, and so on)."""
    K = s["case"]["K"]
    (x, dy), inside, back = _padded(s, s["x"], s.get("d_y"))
    N, T, C = x.shape
    prev = x.new_zeros(N, K - 1, C) if s["x_prev"] is None else s["x_prev"].float()
    xp = torch.cat([prev, x], 1)
    z = s["bias"].expand(N, T, C).clone()
    for k in range(K):
        z += s["w"][:, k] * xp[:, k:k + T]
    return xp, z, dy, inside, back


def _plain_conv_fwd(s):
    c, K = s["case"], s["case"]["K"]
    xp, z, _, inside, back = _plain_conv_z(s)
    y = back(_silu(z) if c["silu"] else z).to(s["x"].dtype)
    at = inside.sum(1)[:, None] + torch.arange(K - 1, device=xp.device)   # the last K - 1 rows of each
    return y, xp[torch.arange(xp.shape[0], device=xp.device)[:, None], at].to(s["x"].dtype)


def _plain_conv_bwd(s):
    c, K, T = s["case"], s["case"]["K"], None
    xp, z, dy, inside, back = _plain_conv_z(s)
    T = z.shape[1]
    if c["silu"]:
        sig = 1 / (1 + torch.exp(-z))
        dy = dy * sig * (1 + z * (1 - sig))
    dy = dy * inside[..., None]
    dxp = torch.zeros_like(xp)
    for k in range(K):
        dxp[:, k:k + T] += s["w"][:, k] * dy
    out = {"dx": back(dxp[:, K - 1:]).to(s["x"].dtype), "dbias": dy.sum((0, 1)),
           "dw": torch.stack([(dy * xp[:, k:k + T]).sum((0, 1)) for k in range(K)], 1)}
    if s["x_prev"] is not None:
        out["dx_prev"] = dxp[:, :K - 1].to(s["x"].dtype)
    return out


def _plain_conv_step(s):
    idx = s["pages"].long()
    xp = torch.cat([s["pool"][idx], s["x"][:, None]], 1)
    s["pool"][idx] = xp[:, 1:]
    z = (xp.float() * s["w"].t()).sum(1) + s["bias"]
    return (_silu(z) if s["case"]["silu"] else z).to(s["x"].dtype), s["pool"]


def _angles(s):
    """cos and sin [B, T, 1, R / 2]: far positions in 64 bits."""
    a = s["positions"].double()[..., None] * s["inv_freq"].double()
    return torch.cos(a).float().unsqueeze(2), torch.sin(a).float().unsqueeze(2)


def _halves(x, R, inter):
    if inter:
        return x[..., 0:R:2], x[..., 1:R:2]
    return x[..., :R // 2], x[..., R // 2:R]


def _joined(a, b, rest, inter):
    r = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _plain_unit(x, l2):
    x = x.float()
    m = (x * x).sum(-1, keepdim=True) if l2 else (x * x).mean(-1, keepdim=True)
    return x, 1 / torch.sqrt(m + 1e-6)


def _plain_qk_fwd(s):
    c, out = s["case"], []
    R = c["R"]
    cs = _angles(s) if R else None
    for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x, r = _plain_unit(s[n], c["l2"])
        u = x * r * scale
        if s[n + "_weight"] is not None:
            u = u * s[n + "_weight"]
        if R:
            a, b = _halves(u, R, c["inter"])
            u = _joined(a * cs[0] - b * cs[1], a * cs[1] + b * cs[0], u[..., R:], c["inter"])
        out.append(u.to(s[n].dtype))
    return tuple(out)


def _plain_qk_bwd(s):
    c, out = s["case"], {}
    R = c["R"]
    cs = _angles(s) if R else None
    for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x, r = _plain_unit(s[n], c["l2"])
        d = s["d_" + n].float() * scale
        if R:
            a, b = _halves(d, R, c["inter"])
            d = _joined(a * cs[0] + b * cs[1], b * cs[0] - a * cs[1], d[..., R:], c["inter"])
        if s[n + "_weight"] is not None:
            out[f"d{n}_weight"] = (d * x * r).sum((0, 1, 2))
            d = d * s[n + "_weight"]
        m = (x * d).sum(-1, keepdim=True) / (1 if c["l2"] else c["D"])
        out["d" + n] = (r * (d - x * r * r * m)).to(s[n].dtype)
    return out


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"ssm_fwd": _plain_ssm_fwd, "ssm_bwd": _plain_ssm_bwd, "ssm_step": _plain_ssm_step,
                "conv_fwd": _plain_conv_fwd, "conv_bwd": _plain_conv_bwd,
                "conv_step": _plain_conv_step, "qk_fwd": _plain_qk_fwd, "qk_bwd": _plain_qk_bwd}[op](s)
    from linear_attention_recurrence_gated_gb300 import gdn
    c = s["case"]
    if op == "ssm_fwd":
        return gdn.gdn_ssm_fwd(s["x"], s["dt"], s["A_log"], s["b"], s["c"], s["h0"], s["cu"],
                               D_skip=s["D_skip"], gate=s["gate"], dt_bias=s["dt_bias"],
                               dt_softplus=True)
    if op == "ssm_bwd":
        g = gdn.gdn_ssm_bwd(s["x"], s["dt"], s["A_log"], s["b"], s["c"], s["d_y"], s["h0"], s["cu"],
                            s["d_hT"], D_skip=s["D_skip"], gate=s["gate"], dt_bias=s["dt_bias"],
                            dt_softplus=True)
        return {k: v for k, v in g.items() if v is not None}
    if op == "ssm_step":
        return gdn.gdn_ssm_step(s["x"], s["dt"], s["A_log"], s["b"], s["c"], s["pool"], s["pages"],
                                D_skip=s["D_skip"], gate=s["gate"], dt_bias=s["dt_bias"],
                                dt_softplus=True)
    if op == "conv_fwd":
        return gdn.gdn_conv_fwd(s["x"], s["w"], s["bias"], s["x_prev"], s["cu"], silu=c["silu"])
    if op == "conv_bwd":
        g = gdn.gdn_conv_bwd(s["x"], s["w"], s["d_y"], s["bias"], s["x_prev"], s["cu"],
                             silu=c["silu"])
        return {k: v for k, v in g.items() if v is not None}
    if op == "conv_step":
        return gdn.gdn_conv_step(s["x"], s["w"], s["pool"], s["bias"], s["pages"], silu=c["silu"])
    how = dict(q_scale=s["q_scale"], l2norm=c["l2"], interleaved=c["inter"])
    if op == "qk_fwd":
        return gdn.gdn_qk_norm(s["q"], s["k"], s["q_weight"], s["k_weight"], s["positions"],
                               s["inv_freq"], **how)
    g = gdn.gdn_qk_norm_bwd(s["q"], s["k"], s["d_q"], s["d_k"], s["q_weight"], s["k_weight"],
                            s["positions"], s["inv_freq"], **how)
    return {k: v for k, v in g.items() if v is not None}


def work(case):
    op = case["op"]
    e = 2 if case["dtype"] == "bf16" else 4
    if op in ("ssm_fwd", "ssm_bwd"):
        n, D, S, G, gate = _tokens(case), case["D"], case["S"], case["G"], int(case["gate"])
        state = 4 * (case["num_seqs"] or case["B"]) * D * S
        if op == "ssm_fwd":   # an exp2 counted as one operation, a multiply-add as two
            return {"bytes": n * e * (D * (3 + gate) + 2 * G * S) + state * (1 + case["init"]),
                    "flops": n * D * (7 * S + 6)}
        return {"bytes": n * e * (D * (5 + 2 * gate) + 4 * G * S) + state * (1 + 2 * case["init"]),
                "flops": n * D * (22 * S + 20)}
    if op == "ssm_step":
        N, D, S, gate = case["N"], case["D"], case["S"], int(case["gate"])
        return {"bytes": N * (8 * D * S + e * (D * (3 + gate) + 2 * case["G"] * S)) + 4 * D * S,
                "flops": N * D * (7 * S + 6)}
    if op in ("conv_fwd", "conv_bwd"):
        n, C, K = _tokens(case), case["C"], case["K"]
        tails = (case["num_seqs"] or case["B"]) * (K - 1) * C * e
        if op == "conv_fwd":
            return {"bytes": 2 * n * C * e + tails * (1 + case["init"]), "flops": n * C * (2 * K + 4)}
        return {"bytes": 3 * n * C * e + 2 * tails * case["init"], "flops": n * C * (6 * K + 8)}
    if op == "conv_step":
        N, C, K = case["N"], case["C"], case["K"]
        return {"bytes": N * C * e * (2 + 2 * (K - 1)) + 4 * C * (K + 1), "flops": N * C * (2 * K + 4)}
    n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
    if op == "qk_fwd":
        return {"bytes": 2 * n * e, "flops": 7 * n}
    return {"bytes": 3 * n * e, "flops": 14 * n}


# ---------------------------------------------------------------------------
# the definitions in 64 bits: token by token, gradients by the chain rule or autograd
# ---------------------------------------------------------------------------
def _tokens_of(s):
    """rows(t): (sequences that have a token t, its rows among all tokens)."""
    x = s["x"]
    if s["cu"] is None:
        B, T = x.shape[:2]
        start = torch.arange(B, device="cuda") * T
        return T, B, lambda t: (slice(None), start + t)
    cu = s["cu"].tolist()
    lens = [b - a for a, b in zip(cu, cu[1:])]

    def rows(t):
        on = [i for i, n in enumerate(lens) if n > t]
        return (torch.tensor(on, device="cuda"), torch.tensor([cu[i] + t for i in on], device="cuda"))

    return max(lens), len(lens), rows


def _exact_ssm(s, backward):
    c = s["case"]
    D, S, per = c["D"], c["S"], c["D"] // c["G"]
    flat = lambda n: s[n].double().flatten(0, 1)  # noqa: E731
    x, dt = flat("x"), flat("dt")
    wide = lambda t: t.repeat_interleave(per, -2)  # noqa: E731  (rows of a group to its channels)
    b, cc = flat("b"), flat("c")
    rate = -s["A_log"].double().exp()
    skip, pre = s["D_skip"].double(), dt + s["dt_bias"].double()
    step = torch.where(pre > 30, pre, torch.log1p(pre.clamp(max=30).exp()))
    gate = None if s["gate"] is None else flat("gate")
    sig = None if gate is None else torch.sigmoid(gate)
    T, N, rows = _tokens_of(s)
    h = torch.zeros(N, D, S, dtype=torch.float64, device="cuda")
    if s["h0"] is not None:
        h += s["h0"].double()
    if not backward:
        y = skip * x
        for t in range(T):
            on, r = rows(t)
            new = h[on] * (step[r].unsqueeze(-1) * rate).exp() + \
                (step[r] * x[r]).unsqueeze(-1) * wide(b[r])
            h[on] = new
            y[r] += torch.einsum("nds,nds->nd", new, wide(cc[r]))
        if gate is not None:
            y = y * gate * sig
        return y.view(s["x"].shape), h
    before = torch.empty(x.shape[0], D, S, dtype=torch.float64, device="cuda")
    total = skip * x
    for t in range(T):
        on, r = rows(t)
        before[r] = h[on]
        new = h[on] * (step[r].unsqueeze(-1) * rate).exp() + (step[r] * x[r]).unsqueeze(-1) * wide(b[r])
        h[on] = new
        total[r] += torch.einsum("nds,nds->nd", new, wide(cc[r]))
    dy = flat("d_y")
    out = {}
    if gate is not None:
        out["dgate"] = (dy * total * (sig + gate * sig * (1 - sig))).view(s["x"].shape)
        dy = dy * gate * sig
    g = torch.zeros_like(h)
    if s["d_hT"] is not None:
        g += s["d_hT"].double()
    dx, dstep = skip * dy, torch.empty_like(x)
    db, dc, drate = torch.empty_like(b), torch.empty_like(cc), torch.zeros_like(rate)
    for t in range(T - 1, -1, -1):
        on, r = rows(t)
        wb, a = wide(b[r]), (step[r].unsqueeze(-1) * rate).exp()
        now = before[r] * a + (step[r] * x[r]).unsqueeze(-1) * wb
        mine = g[on] + dy[r].unsqueeze(-1) * wide(cc[r])
        split = lambda z: z.view(z.shape[0], c["G"], per, S).sum(2)  # noqa: E731
        dc[r] = split(dy[r].unsqueeze(-1) * now)
        db[r] = split((step[r] * x[r]).unsqueeze(-1) * mine)
        through = (mine * wb).sum(-1)
        dx[r] += step[r] * through
        kept = mine * a * before[r]
        dstep[r] = x[r] * through + (kept * rate).sum(-1)
        drate += (kept * step[r].unsqueeze(-1)).sum(0)
        g[on] = mine * a
    dpre = dstep * torch.sigmoid(pre)
    out.update(dx=dx.view(s["x"].shape), ddt=dpre.view(s["x"].shape), db=db.view(s["b"].shape),
               dc=dc.view(s["c"].shape), dA_log=drate * rate, dD_skip=(dy * x).sum(0),
               ddt_bias=dpre.sum(0), dh0=g)
    return out


def _exact_ssm_step(s):
    c, idx = s["case"], s["pages"].long()
    per = c["D"] // c["G"]
    pool, x = s["pool"].double(), s["x"].double()
    pre = s["dt"].double() + s["dt_bias"].double()
    step = torch.where(pre > 30, pre, torch.log1p(pre.clamp(max=30).exp()))
    b, cc = (s[n].double().repeat_interleave(per, 1) for n in "bc")
    h = pool[idx] * torch.exp(torch.einsum("nd,ds->nds", step, -s["A_log"].double().exp())) + \
        torch.einsum("nd,nds->nds", step * x, b)
    pool[idx] = h
    y = torch.einsum("nds,nds->nd", h, cc) + s["D_skip"].double() * x
    if s["gate"] is not None:
        y = y * torch.nn.functional.silu(s["gate"].double())
    return y, pool


def _exact_conv(s, backward):
    """Sequence by sequence, gradients by autograd."""
    c, K = s["case"], s["case"]["K"]
    leaf = {n: s[n].double().requires_grad_(backward) for n in ("x", "w", "bias", "x_prev")
            if s[n] is not None}
    x, prev = leaf["x"], leaf.get("x_prev")
    cu = None if s["cu"] is None else s["cu"].tolist()
    seqs = [x[i] for i in range(x.shape[0])] if cu is None else \
        [x[0, a:b] for a, b in zip(cu, cu[1:])]
    ys, tails = [], []
    for i, rows in enumerate(seqs):
        head = rows.new_zeros(K - 1, rows.shape[1]) if prev is None else prev[i]
        full = torch.cat([head, rows])
        z = torch.einsum("tck,ck->tc", full.unfold(0, K, 1), leaf["w"]) + leaf["bias"]
        ys.append(torch.nn.functional.silu(z) if c["silu"] else z)
        tails.append(full[len(rows):])
    y = (torch.stack(ys) if cu is None else torch.cat(ys)[None])
    if not backward:
        return y, torch.stack(tails)
    y.backward(s["d_y"].double())
    names = {"x": "dx", "w": "dw", "bias": "dbias", "x_prev": "dx_prev"}
    return {names[n]: t.grad for n, t in leaf.items()}


def _exact_conv_step(s):
    pool, idx = s["pool"].double(), s["pages"].long()
    window = torch.cat([pool[idx], s["x"].double()[:, None]], 1)
    pool[idx] = window[:, 1:]
    z = torch.einsum("nkc,ck->nc", window, s["w"].double()) + s["bias"].double()
    return (torch.nn.functional.silu(z) if s["case"]["silu"] else z), pool


def _exact_qk(s, backward):
    """Rotation as a product of complex numbers; gradients by autograd."""
    c, outs, grads = s["case"], [], {}
    R = c["R"]
    for n, scale in (("q", s["q_scale"]), ("k", 1.0)):
        x = s[n].double().requires_grad_(backward)
        w = s[n + "_weight"]
        w = None if w is None else w.double().requires_grad_(backward)
        sq = x.square().sum(-1, keepdim=True)
        u = x * torch.rsqrt((sq if c["l2"] else sq / c["D"]) + 1e-6) * scale
        if w is not None:
            u = u * w
        if R:
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                               s["positions"].double().unsqueeze(-1) * s["inv_freq"].double())
            pairs = u[..., :R].unflatten(-1, (R // 2, 2)) if c["inter"] else \
                u[..., :R].unflatten(-1, (2, R // 2)).transpose(-1, -2)
            z = torch.view_as_real(torch.complex(pairs[..., 0], pairs[..., 1]) * turn.unsqueeze(2))
            u = torch.cat([(z if c["inter"] else z.transpose(-1, -2)).flatten(-2), u[..., R:]], -1)
        if backward:
            u.backward(s["d_" + n].double())
            grads["d" + n] = x.grad
            if w is not None:
                grads[f"d{n}_weight"] = w.grad
        else:
            outs.append(u)
    return grads if backward else tuple(outs)


def exact(case, seed):
    op = case["op"]
    if op == "ssm_bwd" and _tokens(case) * case["D"] * case["S"] > 6e8:
        return None
    s = prepare(case, seed)
    if op in ("ssm_fwd", "ssm_bwd"):
        return _exact_ssm(s, op == "ssm_bwd")
    if op == "ssm_step":
        return _exact_ssm_step(s)
    if op in ("conv_fwd", "conv_bwd"):
        return _exact_conv(s, op == "conv_bwd")
    if op == "conv_step":
        return _exact_conv_step(s)
    return _exact_qk(s, op == "qk_bwd")
