"""A packed training batch of gdn_bwd at its real size, on the GPU: as the dense call on the same
rows, in memory that goes by the tokens."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 64), (torch.float32, 128)])
def test_packed_training_of_128_sequences(dtype, D):
    """bf16 with heads of 64: the same bits, but for dg, whose terms are sums of up to 16 partial
    ones by atomics, in any order: 15 x 2^-24 of their magnitudes.  Else gradients are sums of
    D / 32 slices by atomics: 2^-22 of their norm."""
    N, T, H = 128, 1024, 4
    gen = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    q, v, d_o = (r(N, T, H, D).to(dtype) for _ in range(3))
    k = torch.nn.functional.normalize(r(N, T, H, D), dim=-1).to(dtype)
    g, beta = -torch.rand(N, T, H, generator=gen, device="cuda"), torch.sigmoid(r(N, T, H)).to(dtype)
    h0, d_last = r(N, H, D, D), r(N, H, D, D)
    dense = G.gdn_bwd(q, k, v, g, beta, d_o, h0, None, d_last)
    cu = T * torch.arange(N + 1, dtype=torch.int32, device="cuda")
    flat = lambda t: t.view(1, N * T, *t.shape[2:])  # noqa: E731
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    packed = G.gdn_bwd(flat(q), flat(k), flat(v), flat(g), flat(beta), flat(d_o), h0, cu, d_last, check=True)
    results = sum(t.numel() * t.element_size() for t in packed.values())
    # states of every 64 or 8 tokens in 4 GiB, records and scratch of CTAs: no more than dense
    need = G.gdn_bwd_workspace_size(N, T, H, D, D)
    assert torch.cuda.max_memory_allocated() - held - results < 1.1 * need + (1 << 28) < 8 << 30
    for n, t in packed.items():
        a, b = t.reshape(dense[n].shape), dense[n]
        if D == 64 and n != "dg":
            assert torch.equal(a, b), n
        else:
            tol = 2.0 ** -20 if D == 64 else 2.0 ** -22
            assert float((a.double() - b.double()).norm()) <= tol * float(b.double().norm()), n


def test_ragged_sequences_with_empty_ones():
    """Chunks that end inside sequences, empty sequences (the first among them, before whose slot
    there is no record to read), one of a single token: as the sequences
    by themselves (bf16, heads of 64: bits, dg as above)."""
    lens = [0, 1, 64, 65, 0, 130, 7, 63, 200, 0]
    H, D = 3, 64
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    T, N = sum(lens), len(lens)
    b16 = torch.bfloat16
    q, v, d_o = (r(1, T, H, D).to(b16) for _ in range(3))
    k = torch.nn.functional.normalize(r(1, T, H, D), dim=-1).to(b16)
    g, beta = -torch.rand(1, T, H, generator=gen, device="cuda"), torch.sigmoid(r(1, T, H)).to(b16)
    h0, d_last = r(N, H, D, D), r(N, H, D, D)
    cu = [sum(lens[:n]) for n in range(N + 1)]
    got = G.gdn_bwd(q, k, v, g, beta, d_o, h0, torch.tensor(cu, dtype=torch.int32).cuda(), d_last, check=True)
    for n, (a, b) in enumerate(zip(cu, cu[1:])):
        if a == b:
            assert torch.equal(got["dh0"][n], d_last[n])
            continue
        one = G.gdn_bwd(*(t[:, a:b].clone() for t in (q, k, v, g, beta, d_o)), h0[n:n + 1], None,
                        d_last[n:n + 1])
        assert torch.equal(got["dh0"][n], one["dh0"][0])
        for m in ("dq", "dk", "dv", "dbeta"):
            assert torch.equal(got[m][:, a:b], one[m]), (n, m)
        off = (got["dg"][:, a:b].double() - one["dg"].double()).norm()
        assert float(off) <= 2.0 ** -20 * float(one["dg"].double().norm()), n
