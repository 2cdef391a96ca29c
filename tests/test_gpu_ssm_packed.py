"""Packed training batches of the scan at their real sizes, on the GPU: as the dense call on
the same rows, bit for bit, in memory that goes by the tokens."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu


def test_packed_training_of_128_sequences():
    N, T, D, S = 128, 1024, 2048, 16
    gen = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=gen, device="cuda").to(dtype)  # noqa: E731
    x, dt, gate, d_y = (r(N, T, D) for _ in range(4))
    b, c = r(N, T, 1, S), r(N, T, 1, S)
    A_log = r(D, S, dtype=torch.float32)
    how = dict(D_skip=r(D, dtype=torch.float32), dt_bias=r(D, dtype=torch.float32) - 3, dt_softplus=True)
    h0 = r(N, D, S, dtype=torch.float32)
    dense = G.gdn_ssm_bwd(x, dt, A_log, b, c, d_y, h0, gate=gate, **how)
    cu = T * torch.arange(N + 1, dtype=torch.int32, device="cuda")
    flat = lambda t: t.view(1, N * T, *t.shape[2:])  # noqa: E731
    torch.cuda.synchronize()
    held = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    packed = G.gdn_ssm_bwd(flat(x), flat(dt), A_log, flat(b), flat(c), flat(d_y), h0, cu,
                           gate=flat(gate), check=True, **how)
    results = sum(t.numel() * t.element_size() for t in packed.values())
    # kept states of every eighth token, partial sums of b and c for 16 CTAs of channels: some
    # 2.4 GiB at these sizes
    assert torch.cuda.max_memory_allocated() - held - results < 4 << 30
    for n, t in packed.items():
        assert torch.equal(t.reshape(dense[n].shape), dense[n]), n
