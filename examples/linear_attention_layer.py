"""One linear-attention layer, trained and served on the framework's kernels.

    y = group_norm(attention(x Wq, x Wk, x Wv), one group per head) silu(x Wg) Wo

``train`` runs forward and backward passes of the layer and of a norm over its
features; ``serve`` reads packed prompts into the pages of a state cache, forks each
prompt into branches, extends every branch token by token, drops some, compacts the
pool and goes on.  Run it:  python examples/linear_attention_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_recurrence_gated_gb300 import gdn  # noqa: E402


class Attention(torch.autograd.Function):
    """o, last states of q, k, v [B, T, H, D] from zero states."""

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


class GroupNorm(torch.autograd.Function):
    """Group norm of x [N, S, C], times silu(gate), or with SiLU after it."""

    @staticmethod
    def forward(ctx, x, weight, bias, gate, groups, silu):
        y, mean, rstd = gdn.gdn_group_norm(x, weight, bias, groups, gate=gate, silu=silu)
        ctx.save_for_backward(x, weight, bias, gate, mean, rstd)
        ctx.how = groups, silu
        return y

    @staticmethod
    def backward(ctx, d_y):
        x, weight, bias, gate, mean, rstd = ctx.saved_tensors
        groups, silu = ctx.how
        g = gdn.gdn_group_norm_bwd(x, weight, bias, groups, mean, rstd, d_y.contiguous(),
                                   gate=gate, silu=silu)
        return g["dx"], g["dweight"], g["dbias"], g["dgate"], None, None


class Layer:
    """Weights in ``dtype``, the norm's in fp32; heads of 64 x 64, each with its own
    decay."""

    def __init__(self, width=256, heads=4, dtype=torch.bfloat16, seed=0, device="cuda"):
        self.width, self.heads, self.head = width, heads, 64
        gen = torch.Generator().manual_seed(seed)

        def w(*s):
            return (torch.randn(*s, generator=gen) / s[0] ** 0.5).to(device, dtype).requires_grad_()

        inner = heads * self.head
        self.w_qkvg, self.w_out = w(width, 4 * inner), w(inner, width)
        self.norm = [torch.ones(inner, device=device).requires_grad_(),
                     torch.zeros(inner, device=device).requires_grad_()]
        self.feature_norm = [torch.ones(width, device=device).requires_grad_(),
                             torch.zeros(width, device=device).requires_grad_()]
        self.log_decay = -torch.exp2(-1.0 - torch.arange(heads, device=device).float())

    def parameters(self):
        return [self.w_qkvg, self.w_out, *self.norm, *self.feature_norm]

    def project(self, x):
        """q, k, v: slices of one projection, taken by the kernels as they are."""
        B, T, _ = x.shape
        q, k, v, g = (x @ self.w_qkvg).view(B, T, 4, self.heads, self.head).unbind(2)
        return q * (1 / self.head), k, v, g.reshape(B * T, 1, -1).contiguous()

    def finish(self, o, gate):
        y = GroupNorm.apply(o.reshape(gate.shape), *self.norm, gate, self.heads, False)
        return y.view(*o.shape[:-2], -1) @ self.w_out

    def train_forward(self, x):
        """The layer, then a norm with SiLU over all tokens' features of a sample (which
        lets later tokens into earlier ones: for training on whole samples, not for
        generation, and not part of ``serve``)."""
        q, k, v, gate = self.project(x)
        y = self.finish(Attention.apply(q, k, v, self.log_decay), gate)
        return GroupNorm.apply(x + y, *self.feature_norm, None, 8, True)


def train(steps=30, batch=4, tokens=200, seed=0):
    """Fits a fixed random target; returns the losses."""
    layer = Layer(seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    x, target = (torch.randn(batch, tokens, layer.width, generator=gen).cuda().bfloat16()
                 for _ in range(2))
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        opt.zero_grad(set_to_none=True)
        loss = (layer.train_forward(x) - target).float().square().mean()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    return losses


@torch.no_grad()
def serve(lengths=(70, 1, 333), branches=3, steps=5, seed=0):
    """Returns [(inputs of a branch, its outputs of the extended tokens)] and the
    layer, so that a caller can compare them with a single pass."""
    layer = Layer(seed=seed)
    H, D = layer.heads, layer.head
    gen = torch.Generator().manual_seed(seed + 1)
    rows, pages = 2 * len(lengths) * (branches + 1), 4 * len(lengths) * (branches + 1)

    def ints(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def tokens(n):
        return torch.randn(n, layer.width, generator=gen).cuda().bfloat16()

    # the cache: one page per state, a table of the pages of each row
    pool = torch.empty(pages, H, D, D, device="cuda")
    table = torch.full((rows, 2), -1, dtype=torch.int32, device="cuda")
    counts, refs = ints(*[0] * rows), ints(*[0] * pages)

    # prompts: packed, one scan; each prompt's row starts with a page of zeros
    n = len(lengths)
    prompts = [tokens(t) for t in lengths]
    cu = ints(*[sum(lengths[:i]) for i in range(n + 1)])
    fresh, *_ = gdn.gdn_pages_fork(pool, table, counts, refs, ints(*[-1] * n), ints(*range(n)),
                                   table_out=table, counts_out=counts, refs_out=refs, check=True)
    q, k, v, _ = layer.project(torch.cat(prompts)[None])
    _, states = gdn.gdn_lin_fwd(q, k, v, layer.log_decay, None, cu, check=True)
    pool[fresh.long()] = states

    # branches: each starts from a copy of its prompt's state
    parents = [i for i in range(n) for _ in range(branches)]
    children = list(range(n, n + len(parents)))
    gdn.gdn_pages_fork(pool, table, counts, refs, ints(*parents), ints(*children),
                       table_out=table, counts_out=counts, refs_out=refs, check=True)
    seen = {c: [prompts[p]] for c, p in zip(children, parents)}
    outputs = {c: [] for c in children}

    def extend(alive):
        """One token for each row of ``alive``."""
        x = tokens(len(alive))
        current = table[alive].gather(1, (counts[alive].long() - 1)[:, None])[:, 0].contiguous()
        q, k, v, gate = layer.project(x[:, None])
        o, _ = gdn.gdn_lin_decode(q[:, 0].contiguous(), k[:, 0].contiguous(),
                                  v[:, 0].contiguous(), layer.log_decay, pool, current, check=True)
        y = layer.finish(o, gate)
        for i, c in enumerate(alive):
            seen[c].append(x[i:i + 1])
            outputs[c].append(y[i:i + 1])

    for _ in range(steps):
        extend(children)
    # the prompts and every second branch leave; the pool is made dense; the rest go on
    gone = list(range(n)) + children[::2]
    gdn.gdn_pages_free(table, counts, refs, ints(*gone), table_out=table, counts_out=counts,
                       refs_out=refs, check=True)
    live, table, refs = gdn.gdn_pages_compact(pool, table, counts, refs, check=True)
    alive = children[1::2]
    assert int(live) == len(alive) and int(table.max()) < len(alive)
    for _ in range(steps):
        extend(alive)
    return [(torch.cat(seen[c]), torch.cat(outputs[c])) for c in children], layer


@torch.no_grad()
def whole(layer, x):
    """The layer's outputs for one sequence in a single pass."""
    q, k, v, gate = layer.project(x[None])
    o, _ = gdn.gdn_lin_fwd(q, k, v, layer.log_decay)
    return layer.finish(o, gate)[0]


if __name__ == "__main__":
    losses = train()
    print(f"training: loss {losses[0]:.3f} -> {losses[-1]:.3f} in {len(losses)} steps")
    results, layer = serve()
    worst = 0.0
    for x, y in results:
        want = whole(layer, x)[-len(y):].float()
        worst = max(worst, float((y.float() - want).norm() / want.norm()))
    print(f"serving: {len(results)} branches, token by token against one pass: {worst:.1e}")
