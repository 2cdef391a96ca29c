"""64-bit definitions of the linear-attention, group-norm and state-page
operators, token by token and page by page (numpy; nothing of the CUDA path).

Linear attention with a decay lam = exp(log_decay[h]) for each head:
S_t = lam S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.  Its gradients follow from the
reversed recurrence G_t = q_t do_t^T + lam G_{t+1} (G after the last token:
d_final_state / lam, kept here as lam G = d_final_state).
"""
from __future__ import annotations

import numpy as np


def _np(x):
    return None if x is None else np.asarray(x.double().cpu().numpy() if hasattr(x, "cpu") else x,
                                              np.float64)


def spans(B, T, cu=None):
    """(batch row, first token, length) of every sequence."""
    if cu is None:
        return [(b, 0, T) for b in range(B)]
    cu = [int(c) for c in cu]
    return [(0, a, b - a) for a, b in zip(cu, cu[1:])]


def forward(q, k, v, log_decay, s0=None, cu=None):
    q, k, v, s0 = _np(q), _np(k), _np(v), _np(s0)
    lam = np.exp(_np(log_decay))[:, None, None]
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    seqs = spans(B, T, cu)
    o = np.zeros((B, T, H, dv))
    sT = np.zeros((len(seqs), H, dk, dv))
    for n, (b, a, L) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[n].copy()
        for t in range(a, a + L):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            o[b, t] = np.einsum("hij,hi->hj", S, q[b, t])
        sT[n] = S
    return o, sT


def backward(q, k, v, log_decay, d_o, s0=None, d_sT=None, cu=None):
    q, k, v, d_o, s0, d_sT = (_np(x) for x in (q, k, v, d_o, s0, d_sT))
    lam = np.exp(_np(log_decay))[:, None, None]
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    seqs = spans(B, T, cu)
    out = {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v),
           "dh0": np.zeros((len(seqs), H, dk, dv))}
    for n, (b, a, L) in enumerate(seqs):
        S = np.zeros((H, dk, dv)) if s0 is None else s0[n].copy()
        for t in range(a, a + L):
            S = lam * S + k[b, t][:, :, None] * v[b, t][:, None, :]
            out["dq"][b, t] = np.einsum("hij,hj->hi", S, d_o[b, t])
        R = np.zeros((H, dk, dv)) if d_sT is None else d_sT[n].copy()
        for t in range(a + L - 1, a - 1, -1):
            G = R + q[b, t][:, :, None] * d_o[b, t][:, None, :]
            out["dk"][b, t] = np.einsum("hij,hj->hi", G, v[b, t])
            out["dv"][b, t] = np.einsum("hij,hi->hj", G, k[b, t])
            R = lam * G
        out["dh0"][n] = R
    return out


def _silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def _dsilu(z):
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-z))
    return s * (1.0 + z * (1.0 - s))


def group_norm(x, weight, bias, groups, gate=None, silu=False, eps=1e-5):
    x, weight, bias, gate = _np(x), _np(weight), _np(bias), _np(gate)
    N, S, C = x.shape
    g = x.reshape(N, S, groups, C // groups)
    mean = g.mean((1, 3))
    rstd = 1.0 / np.sqrt(g.var((1, 3)) + eps)
    xh = ((g - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, S, C)
    u = xh * (1.0 if weight is None else weight) + (0.0 if bias is None else bias)
    y = _silu(u) if silu else u
    return (y if gate is None else y * _silu(gate)), mean, rstd


def group_norm_bwd(x, weight, bias, groups, d_y, gate=None, silu=False, eps=1e-5):
    x, weight, bias, gate, d_y = _np(x), _np(weight), _np(bias), _np(gate), _np(d_y)
    N, S, C = x.shape
    w = np.ones(C) if weight is None else weight
    g = x.reshape(N, S, groups, C // groups)
    mean = g.mean((1, 3), keepdims=True)
    rstd = 1.0 / np.sqrt(g.var((1, 3), keepdims=True) + eps)
    xh = ((g - mean) * rstd).reshape(N, S, C)
    u = xh * w + (0.0 if bias is None else bias)
    out = {"dgate": None}
    du = d_y
    if gate is not None:
        out["dgate"] = d_y * (_silu(u) if silu else u) * _dsilu(gate)
        du = d_y * _silu(gate)
    if silu:
        du = du * _dsilu(u)
    out["dweight"], out["dbias"] = (du * xh).sum((0, 1)), du.sum((0, 1))
    dxh, xg = (du * w).reshape(g.shape), xh.reshape(g.shape)
    dx = rstd * (dxh - dxh.mean((1, 3), keepdims=True) - xg * (dxh * xg).mean((1, 3), keepdims=True))
    out["dx"] = dx.reshape(N, S, C)
    return out


class Pages:
    """The page bookkeeping, one job after the other on host integers.  A job
    that breaks a rule is left out and its place kept in ``bad``."""

    def __init__(self, table, counts, refs, pool=None):
        self.table, self.counts, self.refs = (np.array(a, np.int64) for a in (table, counts, refs))
        self.pool = None if pool is None else np.array(pool)
        self.bad, self.short = [], False

    def fork(self, parents, children):
        t0, c0, r0 = self.table.copy(), self.counts.copy(), self.refs.copy()
        R, M = t0.shape
        free = [p for p in range(len(r0)) if r0[p] == 0]
        old = None if self.pool is None else self.pool.copy()
        fresh, seen = [], set()
        for i, (p, c) in enumerate(zip(parents, children)):
            ok = -1 <= p < R and 0 <= c < R and c not in seen
            if 0 <= c < R:
                seen.add(c)
            if ok:
                ok = c0[c] < M if p == c else c0[c] == 0
            if not ok:
                self.bad.append(i)
                fresh.append(-1)
                continue
            have = 0 if p < 0 else c0[p]
            if p >= 0 and have == 0:
                fresh.append(-1)
                continue
            if not free:
                self.short = True
                fresh.append(-1)
                continue
            page = free.pop(0)
            if p == c:
                self.table[c, have] = page
                self.counts[c] = have + 1
            else:
                n = max(int(have), 1)
                self.table[c] = -1
                self.table[c, : n - 1] = t0[p, : n - 1] if p >= 0 else []
                self.table[c, n - 1] = page
                self.counts[c] = n
                for pg in self.table[c, : n - 1]:
                    self.refs[pg] += 1
            self.refs[page] = 1
            if self.pool is not None:
                self.pool[page] = 0 if p < 0 else old[t0[p, have - 1]]
            fresh.append(page)
        return np.array(fresh, np.int64)

    def free(self, rows):
        for i, r in enumerate(rows):
            if not 0 <= r < len(self.counts):
                self.bad.append(i)
                continue
            for pg in self.table[r, : self.counts[r]]:
                self.refs[pg] -= 1
            self.table[r, : self.counts[r]] = -1
            self.counts[r] = 0

    def compact(self):
        live = int((self.refs > 0).sum())
        holes = [p for p in range(live) if self.refs[p] == 0]
        M = self.table.shape[1]
        for src in range(live, len(self.refs)):
            if self.refs[src] > 0:
                dst = holes.pop(0)
                self.refs[dst], self.refs[src] = self.refs[src], 0
                self.table[self.table == src] = dst
                if self.pool is not None:
                    self.pool[dst] = self.pool[src]
        self.table[np.arange(M)[None] >= self.counts[:, None]] = -1
        return live
