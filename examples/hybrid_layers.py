"""Two layers of a hybrid model, trained and served on the framework's kernels.

    selective:  x, z = u Wi;  x = conv(x);  dt, b, c = x Wx;  y = scan(x, dt Wd, b, c) silu(z) Wo
    attention:  q, k, v = u Wqkv;  q, k = norm and rotation of q, k;  y = attention(q, k, v) Wo

each added to its input.  ``train`` runs forward and backward passes of both; ``serve``
reads packed prompts into the pages of three pools (the convolution's last inputs, the
scan's states, the attention's), forks every prompt and extends the branches token by
token.  Run it:  python examples/hybrid_layers.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_recurrence_gated_gb300 import gdn  # noqa: E402


class Conv(torch.autograd.Function):
    """SiLU of the causal convolution of x [B, T, C]."""

    @staticmethod
    def forward(ctx, x, w, bias):
        y, _ = gdn.gdn_conv_fwd(x, w, bias, output_tail=False)
        ctx.save_for_backward(x, w, bias)
        return y

    @staticmethod
    def backward(ctx, d_y):
        x, w, bias = ctx.saved_tensors
        g = gdn.gdn_conv_bwd(x, w, d_y.contiguous(), bias)
        return g["dx"], g["dw"], g["dbias"]


class Scan(torch.autograd.Function):
    """The selective scan of x [B, T, D], gated."""

    @staticmethod
    def forward(ctx, x, dt, A_log, b, c, D_skip, gate, dt_bias):
        y, _ = gdn.gdn_ssm_fwd(x, dt, A_log, b, c, D_skip=D_skip, gate=gate, dt_bias=dt_bias,
                               dt_softplus=True, output_final_state=False)
        ctx.save_for_backward(x, dt, A_log, b, c, D_skip, gate, dt_bias)
        return y

    @staticmethod
    def backward(ctx, d_y):
        x, dt, A_log, b, c, D_skip, gate, dt_bias = ctx.saved_tensors
        g = gdn.gdn_ssm_bwd(x, dt, A_log, b, c, d_y.contiguous(), D_skip=D_skip, gate=gate,
                            dt_bias=dt_bias, dt_softplus=True)
        return (g["dx"], g["ddt"], g["dA_log"], g["db"], g["dc"], g["dD_skip"], g["dgate"],
                g["ddt_bias"])


class QKNorm(torch.autograd.Function):
    """q, k [B, T, H, D] with their heads normalised and rotated; q scaled by 1 / sqrt(D)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, inv_freq):
        ctx.save_for_backward(q, k, q_weight, k_weight, inv_freq)
        return gdn.gdn_qk_norm(q, k, q_weight, k_weight, None, inv_freq, q_scale=q.shape[-1] ** -0.5)

    @staticmethod
    def backward(ctx, d_q, d_k):
        q, k, q_weight, k_weight, inv_freq = ctx.saved_tensors
        g = gdn.gdn_qk_norm_bwd(q, k, d_q.contiguous(), d_k.contiguous(), q_weight, k_weight, None,
                                inv_freq, q_scale=q.shape[-1] ** -0.5)
        return g["dq"], g["dk"], g["dq_weight"], g["dk_weight"], None


class Attention(torch.autograd.Function):
    """Linear attention with a decay for each head, from zero states."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        o, _ = gdn.gdn_lin_fwd(q, k, v, log_decay, output_final_state=False)
        ctx.save_for_backward(q, k, v, log_decay)
        return o

    @staticmethod
    def backward(ctx, d_o):
        q, k, v, log_decay = ctx.saved_tensors
        g = gdn.gdn_lin_bwd(q, k, v, log_decay, d_o.contiguous())
        return g["dq"], g["dk"], g["dv"], None


class Layers:
    """Weights of both layers in ``dtype``; those that the kernels take in fp32."""

    def __init__(self, width=128, inner=256, states=16, rank=8, heads=2, taps=4,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        self.inner, self.states, self.rank, self.heads, self.head = inner, states, rank, heads, 64
        gen = torch.Generator().manual_seed(seed)

        def w(*s, scale=None):
            t = torch.randn(*s, generator=gen) * (s[0] ** -0.5 if scale is None else scale)
            return t.to(device, dtype).requires_grad_()

        def f32(t):
            return t.to(device, torch.float32).requires_grad_()

        self.w_in, self.w_x = w(width, 2 * inner), w(inner, rank + 2 * states)
        self.w_dt, self.w_out = w(rank, inner), w(inner, width)
        self.conv_w = f32(torch.randn(inner, taps, generator=gen) / taps ** 0.5)
        self.conv_b = f32(0.1 * torch.randn(inner, generator=gen))
        self.A_log = f32(torch.log(torch.arange(1.0, states + 1)).expand(inner, states).clone())
        self.D_skip = f32(torch.ones(inner))
        self.dt_bias = f32(torch.randn(inner, generator=gen) - 3)
        self.w_qkv, self.w_o = w(width, 3 * heads * self.head), w(heads * self.head, width)
        self.q_norm, self.k_norm = (f32(1 + 0.1 * torch.randn(self.head, generator=gen)) for _ in range(2))
        self.log_decay = (-torch.exp2(-1.0 - torch.arange(heads).float())).to(device)
        self.inv_freq = (10000.0 ** (-torch.arange(0, self.head, 2) / self.head)).to(device)

    def parameters(self):
        return [self.w_in, self.w_x, self.w_dt, self.w_out, self.conv_w, self.conv_b, self.A_log,
                self.D_skip, self.dt_bias, self.w_qkv, self.w_o, self.q_norm, self.k_norm]

    def steps(self, x):
        """dt, b, c of the convolution's output: dt dense, b and c slices of one projection."""
        p = x @ self.w_x
        S = self.states
        b, c = (p[..., self.rank + i * S:self.rank + (i + 1) * S].unsqueeze(-2) for i in range(2))
        return p[..., :self.rank] @ self.w_dt, b, c

    def train_forward(self, u):
        x, z = (u @ self.w_in).chunk(2, -1)
        x = Conv.apply(x, self.conv_w, self.conv_b)
        dt, b, c = self.steps(x)
        y = Scan.apply(x, dt, self.A_log, b, c, self.D_skip, z, self.dt_bias)
        u = u + y @ self.w_out
        B, T, _ = u.shape
        q, k, v = (u @ self.w_qkv).view(B, T, 3, self.heads, self.head).unbind(2)
        q, k = QKNorm.apply(q, k, self.q_norm, self.k_norm, self.inv_freq)
        o = Attention.apply(q, k, v, self.log_decay)
        return u + o.reshape(B, T, -1) @ self.w_o


def train(steps=20, batch=2, tokens=150, seed=0):
    """Fits a fixed random target; returns the losses."""
    layers = Layers(seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    u, target = (torch.randn(batch, tokens, 128, generator=gen).cuda().bfloat16() for _ in range(2))
    opt = torch.optim.Adam(layers.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = (layers.train_forward(u) - target).float().square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve(lengths=(70, 1, 133), branches=2, steps=6, seed=0):
    """Returns [(inputs of a branch, its outputs of the extended tokens)] and the layers."""
    m = Layers(seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    n, rows = len(lengths), len(lengths) * (branches + 1)
    pages = 2 * rows

    def ints(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def tokens(count):
        return torch.randn(count, 128, generator=gen).cuda().bfloat16()

    # three pools, whose pages of one number belong to one sequence; one table for them
    scans = torch.empty(pages, m.inner, m.states, device="cuda")
    convs = torch.empty(pages, 3, m.inner, device="cuda", dtype=torch.bfloat16)
    attns = torch.empty(pages, m.heads, m.head, m.head, device="cuda")
    table = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    counts, refs = ints(*[0] * rows), ints(*[0] * pages)

    # prompts: packed, every layer once over all of them
    prompts = [tokens(t) for t in lengths]
    cu = ints(*[sum(lengths[:i]) for i in range(n + 1)])
    fresh, *_ = gdn.gdn_pages_fork(scans, table, counts, refs, ints(*[-1] * n), ints(*range(n)),
                                   table_out=table, counts_out=counts, refs_out=refs, check=True)
    u = torch.cat(prompts)[None]
    x, z = (u @ m.w_in).chunk(2, -1)
    x, tails = gdn.gdn_conv_fwd(x, m.conv_w, m.conv_b, None, cu, check=True)
    dt, b, c = m.steps(x)
    y, states = gdn.gdn_ssm_fwd(x, dt, m.A_log, b, c, None, cu, D_skip=m.D_skip, gate=z,
                                dt_bias=m.dt_bias, dt_softplus=True, check=True)
    convs[fresh.long()], scans[fresh.long()] = tails, states
    u = u + y @ m.w_out
    q, k, v = (u @ m.w_qkv).view(1, -1, 3, m.heads, m.head).unbind(2)
    positions = torch.cat([torch.arange(t) for t in lengths]).to(torch.int32).cuda()[None]
    q, k = gdn.gdn_qk_norm(q, k, m.q_norm, m.k_norm, positions, m.inv_freq, q_scale=m.head ** -0.5)
    _, states = gdn.gdn_lin_fwd(q, k, v, m.log_decay, None, cu, check=True)
    attns[fresh.long()] = states

    # branches: copies of the prompts' pages in every pool
    parents = [i for i in range(n) for _ in range(branches)]
    children = list(range(n, n + len(parents)))
    new, *_ = gdn.gdn_pages_fork(scans, table, counts, refs, ints(*parents), ints(*children),
                                 table_out=table, counts_out=counts, refs_out=refs, check=True)
    old = fresh[torch.tensor(parents, device="cuda")].contiguous()
    for pool in (convs, attns):
        gdn.gdn_pages_copy(pool, old, new, check=True)
    seen = [[prompts[p]] for p in parents]
    outputs = [[] for _ in parents]
    at = ints(*[lengths[p] for p in parents])

    for step in range(steps):   # one token for each branch
        u = tokens(len(parents))
        for i in range(len(parents)):
            seen[i].append(u[i:i + 1])
        x, z = (t.contiguous() for t in (u @ m.w_in).chunk(2, -1))
        x, _ = gdn.gdn_conv_step(x, m.conv_w, convs, m.conv_b, new, check=True)
        dt, b, c = (t.contiguous() for t in m.steps(x))
        y, _ = gdn.gdn_ssm_step(x, dt, m.A_log, b, c, scans, new, D_skip=m.D_skip, gate=z,
                                dt_bias=m.dt_bias, dt_softplus=True, check=True)
        u = u + y @ m.w_out
        q, k, v = (u @ m.w_qkv).view(-1, 1, 3, m.heads, m.head).unbind(2)
        q, k = gdn.gdn_qk_norm(q, k, m.q_norm, m.k_norm, (at + step)[:, None], m.inv_freq,
                               q_scale=m.head ** -0.5)
        o, _ = gdn.gdn_lin_decode(q[:, 0], k[:, 0], v[:, 0].contiguous(), m.log_decay, attns, new,
                                  check=True)
        u = u + o.reshape(len(parents), -1) @ m.w_o
        for i in range(len(parents)):
            outputs[i].append(u[i:i + 1])
    return [(torch.cat(s), torch.cat(o)) for s, o in zip(seen, outputs)], m


@torch.no_grad()
def whole(layers, u):
    """The layers' outputs for one sequence in a single pass."""
    return layers.train_forward(u[None])[0]


if __name__ == "__main__":
    losses = train()
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    results, layers = serve()
    worst = 0.0
    for u, y in results:
        want = whole(layers, u)[-len(y):].float()
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    print(f"serving: {len(results)} branches, token by token against one pass: {worst:.1e}")
