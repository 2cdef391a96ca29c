"""Cases of the linear-attention, group-norm and state-page operators.

``run`` computes one pass of a case: with ``own`` false in elementary torch
operations in 32 bits, with ``own`` true through the library's entry points.

The operators:

- linear attention with a decay lam_h = exp(log_decay[h]) for each head,
  S_t = lam_h S_{t-1} + k_t v_t^T, o_t = S_t^T q_t (q, k [B, T, H, dk],
  v [B, T, H, dv]; packed sequences with cu_seqlens): prompts (forward),
  training (backward), and single tokens on a pool of state pages (decode);
- group norm over [N, S, C] with SiLU on the normalised value and / or a
  SiLU gate beside it, forward and backward;
- pages of a state cache: fork of sequences, and free followed by compaction.
"""
import random

import numpy as np
import torch

own = False

_DT = {"fp32": torch.float32, "bf16": torch.bfloat16}
_C = 128  # tokens per chunk of the plain form


def listed():
    return [
        # a short prompt on two small heads: latency (the tiny_fp32 workload's shape)
        dict(name="lin_fwd_tiny_fp32", op="lin_fwd", dtype="fp32", B=1, T=256, H=2, dk=32, dv=32,
             init=False, num_seqs=0, lens=0),
        # a training or prefill batch of the HyMo-shaped layer (the hymo_bf16 workload's shape)
        dict(name="lin_fwd_hymo_bf16", op="lin_fwd", dtype="bf16", B=8, T=4096, H=16, dk=64, dv=64,
             init=False, num_seqs=0, lens=0),
        # prefill of one long document: few units, a long axis (the long_bf16 workload's shape)
        dict(name="lin_fwd_long_bf16", op="lin_fwd", dtype="bf16", B=1, T=65536, H=16, dk=128,
             dv=128, init=False, num_seqs=0, lens=0),
        # packed prompts of ragged lengths, continued from states (the varlen_bf16 workload's shape)
        dict(name="lin_fwd_varlen_bf16", op="lin_fwd", dtype="bf16", B=1, T=0, H=8, dk=128, dv=256,
             init=True, num_seqs=32, lens=8192),
        # training step of a small ragged batch in fp32 (odd length, dk != dv)
        dict(name="lin_bwd_small_fp32", op="lin_bwd", dtype="fp32", B=2, T=333, H=3, dk=32, dv=64,
             init=True, num_seqs=0, lens=0),
        # training step of the wide layer (the wide_bf16 workload's shape)
        dict(name="lin_bwd_wide_bf16", op="lin_bwd", dtype="bf16", B=4, T=8192, H=16, dk=128,
             dv=128, init=True, num_seqs=0, lens=0),
        # generation for a handful of users: latency
        dict(name="lin_decode_few_bf16", op="lin_decode", dtype="bf16", N=8, H=16, dk=64, dv=64,
             P=64),
        # generation for a full server (the decode_hymo_bf16 workload's shape), states in a pool
        dict(name="lin_decode_full_bf16", op="lin_decode", dtype="bf16", N=1024, H=16, dk=64, dv=64,
             P=1280),
        # the layer's output norm: one group per head of each token, gated (hymo_bf16's output)
        dict(name="norm_fwd_heads_bf16", op="norm_fwd", dtype="bf16", N=32768, S=1, C=1024, G=16,
             silu=False, gate=True),
        # training step of the norm over feature maps (conv_hymo_bf16's shape), SiLU
        dict(name="norm_bwd_maps_bf16", op="norm_bwd", dtype="bf16", N=4, S=4096, C=1280, G=40,
             silu=True, gate=False),
        # beams or samples branch off: every child gets a page of its own (256 KB pages)
        dict(name="pages_fork", op="pages_fork", P=2048, page=65536, R=640, M=6, live=256, n=192),
        # sequences end, their pages are freed and the pool is packed
        dict(name="pages_compact", op="pages_compact", P=1536, page=65536, R=512, M=4, live=448,
             n=160),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_bwd", "lin_decode", "norm_fwd", "norm_bwd",
                     "pages_fork", "pages_compact"])
    dtype = rng.choice(["fp32", "bf16", "bf16"])
    if op in ("lin_fwd", "lin_bwd"):
        dk, dv = rng.choice([(32, 32), (64, 64), (128, 128), (64, 128), (128, 64)])
        H = _log(rng, 1, 32)
        most = (96 << 20) // (H * (dk + dv))  # tokens, so that q, k, v and o stay within a GB
        case = dict(op=op, dtype=dtype, H=H, dk=dk, dv=dv, init=rng.random() < 0.5)
        if rng.random() < 0.4:
            n = _log(rng, 1, 24)
            case.update(B=1, T=0, num_seqs=n, lens=_log(rng, 8, max(8, min(8192, most // n))))
        else:
            B = _log(rng, 1, 16)
            case.update(B=B, T=_log(rng, 64, max(64, min(32768, most // B))), num_seqs=0, lens=0)
        return case
    if op == "lin_decode":
        dk, dv = rng.choice([(32, 32), (64, 64), (128, 128), (64, 128)])
        H, N = _log(rng, 1, 32), _log(rng, 1, 1024)
        N = max(1, min(N, (64 << 20) // (H * dk * dv)))
        return dict(op=op, dtype=dtype, N=N, H=H, dk=dk, dv=dv, P=N + _log(rng, 1, 256))
    if op in ("norm_fwd", "norm_bwd"):
        D, G = rng.choice([4, 10, 16, 32, 64, 128]), rng.choice([1, 3, 8, 16, 32])
        most = (64 << 20) // (D * G)
        if rng.random() < 0.5:
            N, S = _log(rng, 16, max(16, min(65536, most))), 1
        else:
            N = _log(rng, 1, 16)
            S = _log(rng, 49, max(49, min(16384, most // N)))
        gate = rng.random() < 0.5
        return dict(op=op, dtype=dtype, N=N, S=S, C=D * G, G=G, silu=not gate or rng.random() < 0.3,
                    gate=gate)
    live = _log(rng, 8, 384)
    return dict(op=op, P=4 * live + _log(rng, 1, 64), page=16 * _log(rng, 64, 4096), R=2 * live,
                M=rng.choice([2, 3, 4]), live=live, n=_log(rng, 4, max(4, live // 2)))


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _lens(case):
    r = random.Random(case["num_seqs"] * 100003 + case["lens"])
    return [r.randint(max(1, case["lens"] // 64), case["lens"]) for _ in range(case["num_seqs"])]


def _tokens(case):
    return sum(_lens(case)) if case["num_seqs"] else case["B"] * case["T"]


def _decay(H):
    """Slopes -2^(-8 (h + 1) / H): from fast heads (half a token) to slow ones (256 tokens)."""
    h = torch.arange(1, H + 1, dtype=torch.float64)
    return (-torch.exp2(-8.0 * h / H)).to(torch.float32).cuda()


def _lin_inputs(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    B, T, H, dk, dv = case["B"], case["T"], case["H"], case["dk"], case["dv"]
    s = dict(case=case, cu=None, N=B)
    if case["num_seqs"]:
        off = np.concatenate([[0], np.cumsum(_lens(case))])
        T, s["N"] = int(off[-1]), case["num_seqs"]
        s["cu"] = torch.tensor(off, dtype=torch.int32, device="cuda")
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    s["q"] = (rand(B, T, H, dk) / dk ** 0.5).to(dt)
    s["k"] = rand(B, T, H, dk).to(dt)
    s["v"] = rand(B, T, H, dv).to(dt)
    s["log_decay"] = _decay(H)
    s["s0"] = rand(s["N"], H, dk, dv) if case["init"] else None
    if case["op"] == "lin_bwd":
        s["d_o"] = rand(B, T, H, dv).to(dt)
        s["d_sT"] = rand(s["N"], H, dk, dv) / dk ** 0.5 if case["init"] else None
    return s


def _decode_inputs(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    N, H, dk, dv, P = case["N"], case["H"], case["dk"], case["dv"], case["P"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    return dict(case=case, q=(rand(N, H, dk) / dk ** 0.5).to(dt), k=rand(N, H, dk).to(dt),
                v=rand(N, H, dv).to(dt), log_decay=_decay(H), pool=rand(P, H, dk, dv),
                pages=torch.randperm(P, generator=g, device="cuda")[:N].to(torch.int32))


def _norm_inputs(case, seed):
    g, dt = _gen(seed), _DT[case["dtype"]]
    N, S, C, G = case["N"], case["S"], case["C"], case["G"]
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    # features with a scale and an offset of their own in each channel
    x = (rand(N, S, C) * (0.5 + rand(C).abs()) + 0.5 * rand(C)).to(dt)
    s = dict(case=case, x=x, weight=1.0 + 0.2 * rand(C), bias=0.2 * rand(C),
             gate=rand(N, S, C).to(dt) if case["gate"] else None)
    if case["op"] == "norm_bwd":
        s["d_y"] = rand(N, S, C).to(dt)
        _, s["mean"], s["rstd"] = _plain_norm(s)  # kept from the forward pass
    return s


def _pages_inputs(case, seed):
    """`live` rows of up to M pages, the last of a row its own and the earlier ones shared with
    the row before (snapshots of a common prefix); page numbers in random order."""
    r = random.Random(int(seed) * 7919 + 17)
    P, R, M, live, n = case["P"], case["R"], case["M"], case["live"], case["n"]
    order = list(range(P))
    r.shuffle(order)
    table, counts, refs = np.full((R, M), -1, np.int32), np.zeros(R, np.int32), np.zeros(P, np.int32)
    rows = list(range(R))
    r.shuffle(rows)
    shared = []
    for i in range(live):
        if i % 4 == 0:
            shared = [order.pop() for _ in range(r.randint(0, M - 1))]
        mine = shared[: r.randint(0, len(shared))] + [order.pop()]
        table[rows[i], : len(mine)] = mine
        counts[rows[i]] = len(mine)
        refs[mine] += 1
    pool = torch.randn(P, case["page"], generator=_gen(seed), device="cuda")
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    s = dict(case=case, pool=pool, table=dev(table), counts=dev(counts), refs=dev(refs))
    if case["op"] == "pages_fork":
        s["parents"] = dev([rows[r.randrange(live)] for _ in range(n)])
        s["children"] = dev(rows[live: live + n])
    else:
        s["rows"] = dev(r.sample(rows[:live], n))
    return s


def prepare(case, seed):
    op = case["op"]
    if op in ("lin_fwd", "lin_bwd"):
        return _lin_inputs(case, seed)
    if op == "lin_decode":
        return _decode_inputs(case, seed)
    if op in ("norm_fwd", "norm_bwd"):
        return _norm_inputs(case, seed)
    return _pages_inputs(case, seed)


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------
def _plain_scan(q, k, v, log_decay, s0, lens):
    """o and the final state of the recurrence over dense [N, T, H, *] fp32
    tensors whose rows past lens[n] are zero."""
    N, T, H, dk = q.shape
    dv, nc = v.shape[-1], max(1, -(-T // _C))
    pad = nc * _C - T
    q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(N, nc, _C, H, -1)
               .permute(0, 3, 1, 2, 4) for x in (q, k, v))  # [N, H, nc, C, d]
    i = torch.arange(_C, device=q.device)
    ld = log_decay.view(H, 1, 1)
    back = (i[:, None] - i[None, :]).clamp(min=0)
    weight = torch.exp(ld * back) * (i[:, None] >= i[None, :])              # [H, C, C]
    o = ((q @ k.transpose(-1, -2)) * weight[None, :, None]) @ v
    edge = torch.minimum(torch.arange(nc + 1, device=q.device)[None] * _C, lens[:, None])  # [N, nc+1]
    left = (edge[:, 1:, None] - 1 - (edge[:, :-1, None] + i)).clamp(min=0)    # tokens to the chunk's end
    x = (k * torch.exp(log_decay.view(1, H, 1, 1) * left[:, None]).unsqueeze(-1)).transpose(-1, -2) @ v
    # every chunk's entry state (and the final one) from all chunks before it
    span = edge[:, :, None] - edge[:, None, 1:]                               # [N, nc+1, nc]
    w = torch.exp(log_decay.view(1, H, 1, 1) * span.clamp(min=0)[:, None]) * \
        (torch.arange(nc, device=q.device) < torch.arange(nc + 1, device=q.device)[:, None])
    s = (w @ x.reshape(N, H, nc, dk * dv)).view(N, H, nc + 1, dk, dv)
    if s0 is not None:
        s = s + torch.exp(log_decay.view(1, H, 1) * edge[:, None]).view(N, H, nc + 1, 1, 1) * s0[:, :, None]
    o = o + torch.exp(ld[..., 0] * (i + 1)).view(1, H, 1, _C, 1) * (q @ s[:, :, :nc])
    o = o.permute(0, 2, 3, 1, 4).reshape(N, nc * _C, H, dv)[:, :T]
    return o, s[:, :, nc]


def _dense(s, *tensors):
    """(lens, fp32 [N, T, H, *] of each tensor with zero rows past the lengths, its inverse)."""
    if s["cu"] is None:
        t = tensors[0]
        lens = torch.full((t.shape[0],), t.shape[1], device=t.device)
        return lens, [x.float() for x in tensors], lambda y: y
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    most = max(_lens(s["case"]))
    at = torch.arange(most, device=cu.device)
    inside = at < lens[:, None]
    idx = torch.where(inside, cu[:-1, None] + at, 0)
    dense = [x[0].float()[idx] * inside[..., None, None] for x in tensors]
    row = torch.arange(tensors[0].shape[1], device=cu.device)
    seq = torch.searchsorted(cu[1:], row, right=True)
    return lens, dense, lambda y: y[seq, row - cu[seq]][None]


def _flip(x, lens):
    """Each sequence's rows in reverse order (rows past its length stay zero)."""
    at = lens[:, None] - 1 - torch.arange(x.shape[1], device=x.device)
    y = torch.gather(x, 1, at.clamp(min=0)[..., None, None].expand_as(x))
    return y * (at >= 0)[..., None, None]


def _plain_lin_fwd(s):
    lens, (q, k, v), packed = _dense(s, s["q"], s["k"], s["v"])
    o, sT = _plain_scan(q, k, v, s["log_decay"], s["s0"], lens)
    return packed(o).to(s["q"].dtype), sT


def _plain_lin_bwd(s):
    lens, (q, k, v, do), packed = _dense(s, s["q"], s["k"], s["v"], s["d_o"])
    ld, dt = s["log_decay"], s["q"].dtype
    turn = lambda x: None if x is None else x.transpose(-1, -2)  # noqa: E731
    dq, _ = _plain_scan(do, v, k, ld, turn(s["s0"]), lens)
    lam = torch.exp(ld).view(1, -1, 1, 1)
    end = None if s["d_sT"] is None else s["d_sT"] / lam
    qr, kr, vr, dor = (_flip(x, lens) for x in (q, k, v, do))
    dk, _ = _plain_scan(vr, dor, qr, ld, turn(end), lens)
    dv, g1 = _plain_scan(kr, qr, dor, ld, end, lens)
    return {"dq": packed(dq).to(dt), "dk": packed(_flip(dk, lens)).to(dt),
            "dv": packed(_flip(dv, lens)).to(dt), "dh0": lam * g1}


def _plain_decode(s):
    idx = s["pages"].long()
    q, k, v = (s[n].float() for n in "qkv")
    st = torch.exp(s["log_decay"]).view(1, -1, 1, 1) * s["pool"][idx] + k[..., :, None] * v[..., None, :]
    s["pool"][idx] = st
    return (q[..., :, None] * st).sum(-2).to(s["q"].dtype), s["pool"]


def _silu(z):
    return z / (1 + torch.exp(-z))


def _plain_norm(s):
    c, x = s["case"], s["x"].float()
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    xg = x.view(N, S, G, C // G)
    mean = xg.mean((1, 3))
    d = xg - mean.view(N, 1, G, 1)
    rstd = 1 / torch.sqrt((d * d).mean((1, 3)) + 1e-5)
    y = (d * rstd.view(N, 1, G, 1)).view(N, S, C) * s["weight"] + s["bias"]
    if c["silu"]:
        y = _silu(y)
    if c["gate"]:
        y = y * _silu(s["gate"].float())
    return y.to(s["x"].dtype), mean, rstd


def _plain_norm_bwd(s):
    c, x, dy = s["case"], s["x"].float(), s["d_y"].float()
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    mean, rstd = s["mean"].view(N, 1, G, 1), s["rstd"].view(N, 1, G, 1)
    xh = ((x.view(N, S, G, C // G) - mean) * rstd).view(N, S, C)
    n = xh * s["weight"] + s["bias"]
    sig = 1 / (1 + torch.exp(-n))
    a, da = (n * sig, sig * (1 + n * (1 - sig))) if c["silu"] else (n, torch.ones_like(n))
    out = {}
    dn = dy * da
    if c["gate"]:
        z = s["gate"].float()
        sz = 1 / (1 + torch.exp(-z))
        out["dgate"] = (dy * a * sz * (1 + z * (1 - sz))).to(s["x"].dtype)
        dn = dn * z * sz
    out["dweight"], out["dbias"] = (dn * xh).sum((0, 1)), dn.sum((0, 1))
    dxh, xh = (dn * s["weight"]).view(N, S, G, C // G), xh.view(N, S, G, C // G)
    dx = rstd * (dxh - dxh.mean((1, 3), keepdim=True) - xh * (dxh * xh).mean((1, 3), keepdim=True))
    out["dx"] = dx.view(N, S, C).to(s["x"].dtype)
    return out


def _plain_fork(s):
    table, counts, refs, pool = s["table"], s["counts"], s["refs"], s["pool"]
    parents, children = s["parents"].long(), s["children"].long()
    n, M = parents.numel(), table.shape[1]
    cnt = counts[parents].long()
    fresh = torch.argsort((refs > 0).int(), stable=True)[:n]  # the lowest free pages
    pos = torch.arange(M, device=table.device)
    rows = table[parents]
    keep = pos < cnt[:, None] - 1
    child = torch.where(keep, rows, torch.where(pos == cnt[:, None] - 1, fresh[:, None].int(), -1))
    table_out, counts_out, refs_out = table.clone(), counts.clone(), refs.clone()
    table_out[children] = child
    counts_out[children] = cnt.int()
    refs_out.index_add_(0, rows.clamp(min=0).long().reshape(-1), keep.int().reshape(-1))
    refs_out[fresh] = 1
    pool[fresh] = pool[rows.gather(1, cnt[:, None] - 1)[:, 0].long()]
    return {"fresh": fresh.int(), "table": table_out, "counts": counts_out, "refs": refs_out,
            "pool": pool}


def _plain_free_compact(s):
    table, counts, refs, pool = s["table"].clone(), s["counts"].clone(), s["refs"].clone(), s["pool"]
    rows = s["rows"].long()
    pos = torch.arange(table.shape[1], device=table.device)
    gone = pos < counts[rows][:, None]
    refs.index_add_(0, table[rows].clamp(min=0).long().reshape(-1), -gone.int().reshape(-1))
    table[rows] = -1
    counts[rows] = 0
    live = refs > 0
    num = live.sum()
    at = torch.arange(refs.numel(), device=table.device)
    src, dst = torch.nonzero(live & (at >= num))[:, 0], torch.nonzero(~live & (at < num))[:, 0]
    new = at.clone()
    new[src] = dst
    table = torch.where(pos < counts[:, None], new[table.clamp(min=0).long()].int(), -1)
    pool[dst] = pool[src]
    refs[dst] = refs[src]
    refs[src] = 0
    return {"num_live": num.int().view(1), "table": table, "counts": counts, "refs": refs,
            "pool": pool}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"lin_fwd": _plain_lin_fwd, "lin_bwd": _plain_lin_bwd, "lin_decode": _plain_decode,
                "norm_fwd": _plain_norm, "norm_bwd": _plain_norm_bwd, "pages_fork": _plain_fork,
                "pages_compact": _plain_free_compact}[op](s)
    from linear_attention_recurrence_gated_gb300 import gdn
    c = s["case"]
    if op == "lin_fwd":
        return gdn.gdn_lin_fwd(s["q"], s["k"], s["v"], s["log_decay"], s["s0"], s["cu"])
    if op == "lin_bwd":
        return gdn.gdn_lin_bwd(s["q"], s["k"], s["v"], s["log_decay"], s["d_o"], s["s0"], s["cu"],
                               s["d_sT"])
    if op == "lin_decode":
        return gdn.gdn_lin_decode(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], s["pages"])
    if op == "norm_fwd":
        return gdn.gdn_group_norm(s["x"], s["weight"], s["bias"], c["G"], gate=s["gate"],
                                  silu=c["silu"])
    if op == "norm_bwd":
        g = gdn.gdn_group_norm_bwd(s["x"], s["weight"], s["bias"], c["G"], s["mean"], s["rstd"],
                                   s["d_y"], gate=s["gate"], silu=c["silu"])
        return {k: v for k, v in g.items() if v is not None}
    if op == "pages_fork":
        fresh, table, counts, refs = gdn.gdn_pages_fork(s["pool"], s["table"], s["counts"],
                                                        s["refs"], s["parents"], s["children"])
        return {"fresh": fresh, "table": table, "counts": counts, "refs": refs, "pool": s["pool"]}
    table, counts, refs = gdn.gdn_pages_free(s["table"], s["counts"], s["refs"], s["rows"])
    num, table, refs = gdn.gdn_pages_compact(s["pool"], table, counts, refs, table_out=table,
                                             refs_out=refs)
    return {"num_live": num, "table": table, "counts": counts, "refs": refs, "pool": s["pool"]}


def work(case):
    op = case["op"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if op in ("lin_fwd", "lin_bwd"):
        rows, dk, dv = _tokens(case) * case["H"], case["dk"], case["dv"]
        state = 4 * (case["num_seqs"] or case["B"]) * case["H"] * dk * dv
        if op == "lin_fwd":
            return {"bytes": rows * e * (2 * dk + 2 * dv) + state * (1 + case["init"]),
                    "flops": 4 * rows * dk * dv}
        return {"bytes": rows * e * (4 * dk + 3 * dv) + state * (1 + 2 * case["init"]),
                "flops": 10 * rows * dk * dv}
    if op == "lin_decode":
        rows, dk, dv = case["N"] * case["H"], case["dk"], case["dv"]
        return {"bytes": rows * (8 * dk * dv + e * (2 * dk + 2 * dv)), "flops": 4 * rows * dk * dv}
    if op in ("norm_fwd", "norm_bwd"):
        n, gate = case["N"] * case["S"] * case["C"], int(case["gate"])
        if op == "norm_fwd":
            return {"bytes": n * e * (2 + gate), "flops": n * 8}
        return {"bytes": n * e * (3 + 2 * gate), "flops": n * 20}
    meta = 8 * (case["R"] * (case["M"] + 1) + case["P"])
    if op == "pages_fork":
        return {"bytes": 8 * case["page"] * case["n"] + meta, "flops": 0}
    # a page above the packed end moves; page numbers are random, so that is the free share
    per = (1 + 0.15 * (case["M"] - 1)) * (case["live"] - case["n"])  # pages that stay live
    return {"bytes": 8 * case["page"] * per * (1 - per / case["P"]) + meta, "flops": 0}


# ---------------------------------------------------------------------------
# the definitions in 64 bits: token by token, page by page
# ---------------------------------------------------------------------------
def _sequences(s):
    """[(first token, length)] of every sequence, and one tensor flattened to [tokens, H, d]."""
    if s["cu"] is None:
        B, T = s["q"].shape[:2]
        return [(b * T, T) for b in range(B)]
    cu = s["cu"].tolist()
    return [(a, b - a) for a, b in zip(cu, cu[1:])]


def _exact_lin(s, backward):
    c = s["case"]
    seqs = _sequences(s)
    flat = {n: s[n].double().reshape(-1, c["H"], s[n].shape[-1]) for n in ("q", "k", "v", "d_o") if n in s}
    lam = torch.exp(s["log_decay"].double()).view(1, -1, 1, 1)
    start = torch.tensor([a for a, _ in seqs], device="cuda")
    size = torch.tensor([b for _, b in seqs], device="cuda")
    N, H, dk, dv = len(seqs), c["H"], c["dk"], c["dv"]
    S = torch.zeros(N, H, dk, dv, dtype=torch.float64, device="cuda")
    if s["s0"] is not None:
        S += s["s0"].double()
    longest = max(b for _, b in seqs)
    same = s["cu"] is None
    first = torch.empty_like(flat["q"]) if backward else torch.empty_like(flat["v"])

    def at(t):
        """Rows of token t of every sequence that has one."""
        if same:
            return slice(None), start + t
        on = torch.tensor([i for i, (_, n) in enumerate(seqs) if n > t], device="cuda")
        return on, start[on] + t

    for t in range(longest):
        on, row = at(t)
        S[on] = lam * S[on] + flat["k"][row].unsqueeze(-1) * flat["v"][row].unsqueeze(-2)
        if backward:
            first[row] = (S[on] * flat["d_o"][row].unsqueeze(-2)).sum(-1)
        else:
            first[row] = (S[on] * flat["q"][row].unsqueeze(-1)).sum(-2)
    if not backward:
        return first.view(s["v"].shape), S
    G = torch.zeros_like(S)   # lam times the gradient of the state after the token
    if s["d_sT"] is not None:
        G += s["d_sT"].double()
    dk_, dv_ = torch.empty_like(flat["k"]), torch.empty_like(flat["v"])
    for t in range(longest - 1, -1, -1):
        on, row = at(t)
        g = G[on] + flat["q"][row].unsqueeze(-1) * flat["d_o"][row].unsqueeze(-2)
        dk_[row] = (g * flat["v"][row].unsqueeze(-2)).sum(-1)
        dv_[row] = (g * flat["k"][row].unsqueeze(-1)).sum(-2)
        G[on] = lam * g
    return {"dq": first.view(s["q"].shape), "dk": dk_.view(s["k"].shape),
            "dv": dv_.view(s["v"].shape), "dh0": G}


def _exact_norm(s):
    """Autograd of the formula in 64 bits gives the gradients."""
    c = s["case"]
    leaf = {n: s[n].double().requires_grad_(c["op"] == "norm_bwd")
            for n in ("x", "weight", "bias", "gate") if s[n] is not None}
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    g = leaf["x"].reshape(N, S, G, C // G).permute(0, 2, 1, 3).reshape(N, G, -1)
    mean = g.mean(-1)
    rstd = ((g - mean[..., None]) ** 2).mean(-1).add(1e-5).rsqrt()
    h = ((g - mean[..., None]) * rstd[..., None]).reshape(N, G, S, C // G).permute(0, 2, 1, 3)
    h = h.reshape(N, S, C) * leaf["weight"] + leaf["bias"]
    y = h * torch.sigmoid(h) if c["silu"] else h
    if "gate" in leaf:
        y = y * leaf["gate"] * torch.sigmoid(leaf["gate"])
    if c["op"] == "norm_fwd":
        return y, mean, rstd
    y.backward(s["d_y"].double())
    return {"d" + n: t.grad for n, t in leaf.items()}


def _exact_pages(s):
    table, counts, refs = (s[n].cpu().numpy().copy() for n in ("table", "counts", "refs"))
    pool, moves, out = s["pool"], [], {}
    if s["case"]["op"] == "pages_fork":
        fresh = []
        for p, ch in zip(s["parents"].tolist(), s["children"].tolist()):
            n = int(counts[p])
            page = int(np.flatnonzero(refs == 0)[0])
            moves.append((int(table[p, n - 1]), page))
            refs[page] = 1
            refs[table[p, : n - 1]] += 1
            table[ch] = -1
            table[ch, : n - 1], table[ch, n - 1], counts[ch] = table[p, : n - 1], page, n
            fresh.append(page)
        out["fresh"] = np.array(fresh, np.int32)
    else:
        for r in s["rows"].tolist():
            np.subtract.at(refs, table[r, : counts[r]], 1)
            table[r], counts[r] = -1, 0
        num = int((refs > 0).sum())
        holes = [p for p in range(num) if refs[p] == 0]
        for src in range(num, len(refs)):
            if refs[src] > 0:
                dst = holes.pop(0)
                moves.append((src, dst))
                refs[dst], refs[src] = refs[src], 0
                table[table == src] = dst
        out["num_live"] = np.array([num], np.int32)
    for src, dst in moves:
        pool[dst] = pool[src]
    return {**out, "table": table, "counts": counts, "refs": refs, "pool": pool}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op in ("lin_fwd", "lin_bwd"):
        return _exact_lin(s, op == "lin_bwd")
    if op == "lin_decode":
        pool, idx = s["pool"].double(), s["pages"].long()
        st = torch.exp(s["log_decay"].double())[:, None, None] * pool[idx] + \
            torch.einsum("nhi,nhj->nhij", s["k"].double(), s["v"].double())
        pool[idx] = st
        return torch.einsum("nhi,nhij->nhj", s["q"].double(), st), pool
    if op in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s)
    return _exact_pages(s)
