"""The selective scan, its short convolution and the q/k norm with rotation in fp64 torch
on the CPU, written as their formulas: token by token, head by head.  Gradients by
autograd."""
from __future__ import annotations

import torch


def _d(t):
    return None if t is None else t.detach().cpu().double()


def _seqs(x, cu):
    """Index of every sequence into [B, T, ...]: (row, slice)."""
    B, T = x.shape[:2]
    if cu is None:
        return [(i, slice(0, T)) for i in range(B)]
    cu = [int(v) for v in cu]
    return [(0, slice(a, b)) for a, b in zip(cu, cu[1:])]


def scan(x, dt, A_log, b, c, h0=None, cu=None, D_skip=None, gate=None, dt_bias=None,
         dt_softplus=False):
    """(y, last states) of fp64 tensors."""
    D, S = A_log.shape
    per = D // b.shape[2]
    A = -torch.exp(A_log)
    seqs = _seqs(x, cu)
    rows = [[None] * x.shape[1] for _ in range(x.shape[0])]
    last = []
    for n, (i, span) in enumerate(seqs):
        h = torch.zeros(D, S, dtype=torch.float64) if h0 is None else h0[n]
        for t in range(span.start, span.stop):
            v = dt[i, t] if dt_bias is None else dt[i, t] + dt_bias
            delta = torch.logaddexp(v, torch.zeros_like(v)) if dt_softplus else v
            bt, ct = (m[i, t].repeat_interleave(per, 0) for m in (b, c))
            h = torch.exp(delta[:, None] * A) * h + (delta * x[i, t])[:, None] * bt
            y = (h * ct).sum(-1)
            if D_skip is not None:
                y = y + D_skip * x[i, t]
            if gate is not None:
                y = y * gate[i, t] * torch.sigmoid(gate[i, t])
            rows[i][t] = y
        last.append(h)
    if x.shape[1] == 0:
        return x.clone(), torch.stack(last)
    return torch.stack([torch.stack(r) for r in rows]), torch.stack(last)


def conv(x, w, bias=None, x_prev=None, cu=None, silu=True):
    """(y, last inputs)."""
    K = w.shape[1]
    y, tails = x.clone(), []
    out = []
    for n, (i, span) in enumerate(_seqs(x, cu)):
        head = x.new_zeros(K - 1, x.shape[2]) if x_prev is None else x_prev[n]
        full = torch.cat([head, x[i, span]])
        L = span.stop - span.start
        z = sum(full[k:k + L] * w[:, k] for k in range(K))
        if bias is not None:
            z = z + bias
        out.append(z * torch.sigmoid(z) if silu else z)
        tails.append(full[L:])
    y = torch.stack(out) if cu is None else torch.cat(out)[None]
    return y, torch.stack(tails)


def qk(x, weight=None, positions=None, inv_freq=None, scale=1.0, eps=1e-6, l2norm=False,
       interleaved=False):
    """One of q and k, [B, T, H, D]."""
    sq = (x * x).sum(-1, keepdim=True)
    u = x / torch.sqrt((sq if l2norm else sq / x.shape[-1]) + eps) * scale
    if weight is not None:
        u = u * weight
    if inv_freq is None or inv_freq.numel() == 0:
        return u
    half = inv_freq.numel()
    if positions is None:
        positions = torch.arange(x.shape[1]).expand(x.shape[:2])
    phi = (positions.double()[..., None] * inv_freq.double())[:, :, None]
    first = [2 * i if interleaved else i for i in range(half)]
    second = [2 * i + 1 if interleaved else i + half for i in range(half)]
    a, b = u[..., first], u[..., second]
    out = u.clone()
    out[..., first] = a * torch.cos(phi) - b * torch.sin(phi)
    out[..., second] = a * torch.sin(phi) + b * torch.cos(phi)
    return out


def grads(fn, inputs, d_outs, **how):
    """Gradients of every tensor of ``inputs`` (name -> tensor) under ``fn(**inputs, **how)``,
    whose outputs receive ``d_outs`` (None: none)."""
    leaf = {n: _d(t).requires_grad_() for n, t in inputs.items() if t is not None}
    outs = fn(**{n: leaf.get(n) for n in inputs}, **how)
    outs = outs if isinstance(outs, tuple) else (outs,)
    total = sum((o * _d(d)).sum() for o, d in zip(outs, d_outs) if d is not None)
    total.backward()
    return {n: torch.zeros_like(t) if t.grad is None else t.grad for n, t in leaf.items()}


def scan_grads(i, d_y, d_last=None, mask=None, softplus=True):
    """(y, last states, gradients) of sequences side by side, by the recurrence and its adjoint
    written out, in fp64 on the tensors' device.  ``i``: x, dt, A_log, b, c and h0, D_skip,
    gate, dt_bias (or None) of [N, T, ..] rows; mask [N, T]: which rows are tokens (or None:
    all)."""
    i = {n: None if t is None else t.double() for n, t in i.items()}
    x, (D, S) = i["x"], i["A_log"].shape
    N, T, _ = x.shape
    per = D // i["b"].shape[2]
    wide = lambda t: t.repeat_interleave(per, -2)  # noqa: E731
    A = -torch.exp(i["A_log"])
    v = i["dt"] if i["dt_bias"] is None else i["dt"] + i["dt_bias"]
    delta = v.clamp(min=0) + torch.log1p(torch.exp(-v.abs())) if softplus else v
    skip = x.new_zeros(D) if i["D_skip"] is None else i["D_skip"]
    sig = None if i["gate"] is None else torch.sigmoid(i["gate"])
    silu = x.new_ones(()) if sig is None else i["gate"] * sig
    d_y = d_y.double()
    if mask is not None:
        delta, d_y = delta * mask[..., None], d_y * mask[..., None]
    h = x.new_zeros(N, D, S) if i["h0"] is None else i["h0"]
    states, s = [h], torch.empty_like(x)
    for t in range(T):
        h = torch.exp(delta[:, t, :, None] * A) * h + (delta[:, t] * x[:, t])[..., None] * wide(i["b"][:, t])
        states.append(h)
        s[:, t] = (wide(i["c"][:, t]) * h).sum(-1) + skip * x[:, t]
    last, ds = h, d_y * silu
    g = torch.zeros_like(h) if d_last is None else d_last.double()
    dx, ddelta = skip * ds, torch.empty_like(x)
    db, dc, dA = torch.empty_like(i["b"]), torch.empty_like(i["c"]), torch.zeros_like(A)
    group = lambda t: t.view(N, -1, per, S).sum(2)  # noqa: E731
    for t in range(T - 1, -1, -1):
        bt, step = wide(i["b"][:, t]), delta[:, t, :, None]
        G = g + ds[:, t, :, None] * wide(i["c"][:, t])
        dc[:, t] = group(ds[:, t, :, None] * states[t + 1])
        db[:, t] = group(step * x[:, t, :, None] * G)
        q = (bt * G).sum(-1)
        dx[:, t] += delta[:, t] * q
        g = torch.exp(step * A) * G
        w = g * states[t]
        ddelta[:, t] = x[:, t] * q + (A * w).sum(-1)
        dA += (step * w).sum(0)
    ddt = ddelta * torch.sigmoid(v) if softplus else ddelta
    if mask is not None:
        ddt = ddt * mask[..., None]
    out = dict(dx=dx, ddt=ddt, db=db, dc=dc, dA_log=A * dA, dD_skip=(ds * x).sum((0, 1)),
               ddt_bias=ddt.sum((0, 1)), dh0=g)
    if sig is not None:
        out["dgate"] = d_y * s * sig * (1 + i["gate"] * (1 - sig))
    return s * silu, last, out
