"""The selective scan, the short convolution and the q/k norm at their limits: rows and pages
whose offsets pass 32 bits, the most sequences, channels and heads, calls on several streams
at once.  The results are those of the same call on small dense tensors, bit for bit, unless a
test says otherwise."""
import pytest
import torch

from linear_attention_recurrence_gated_gb300 import gdn as G

pytestmark = pytest.mark.gpu
FAR = 2 ** 28   # elements from row to row: the tenth row lies beyond 2^31 of them


def rand(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def far(t, base, at):
    """t [1, T, ...] as a slice, from element `at`, of rows FAR elements apart."""
    n = t[0, 0].numel()
    v = base.as_strided((1, t.shape[1], n), (t.shape[1] * FAR, FAR, 1), at)
    v.copy_(t.reshape(1, -1, n))
    return v.as_strided(t.shape, (t.shape[1] * FAR, FAR) + t.stride()[2:], at)


def same(a, b):
    assert a.keys() == b.keys() if isinstance(a, dict) else len(a) == len(b)
    for n in (a if isinstance(a, dict) else range(len(a))):
        assert (a[n] is None and b[n] is None) or torch.equal(a[n], b[n]), n


def scan_inputs(T, D, S, seed=0, B=1):
    return dict(x=rand(seed, B, T, D), dt=rand(seed + 1, B, T, D), A_log=rand(seed + 2, D, S, dtype=torch.float32),
                b=rand(seed + 3, B, T, 1, S), c=rand(seed + 4, B, T, 1, S), gate=rand(seed + 5, B, T, D),
                d_y=rand(seed + 6, B, T, D), bias=rand(seed + 7, D, dtype=torch.float32) - 2)


def scan(i, **kw):
    return G.gdn_ssm_fwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], gate=i["gate"], dt_bias=i["bias"],
                         dt_softplus=True, **kw)


def scan_bwd(i, **kw):
    return G.gdn_ssm_bwd(i["x"], i["dt"], i["A_log"], i["b"], i["c"], i["d_y"], gate=i["gate"],
                         dt_bias=i["bias"], dt_softplus=True, **kw)


def test_rows_beyond_32_bits():
    T = 10
    base = torch.empty(T * FAR, dtype=torch.bfloat16, device="cuda")
    i = scan_inputs(T, 64, 16)
    j = dict(i)
    for k, n in enumerate(("x", "dt", "b", "c", "gate")):
        j[n] = far(i[n], base, 128 * k)
    same(scan(i), scan(j))
    same(scan_bwd(i), scan_bwd(j))
    w = rand(9, 64, 4, dtype=torch.float32)
    same(G.gdn_conv_fwd(i["x"], w), G.gdn_conv_fwd(j["x"], w))
    same(G.gdn_conv_bwd(i["x"], w, i["d_y"]), G.gdn_conv_bwd(j["x"], w, i["d_y"]))
    q, k = rand(10, 1, T, 4, 64), rand(11, 1, T, 2, 64)
    fq, fk = far(q, base, 0), far(k, base, 1024)
    freq = (10000.0 ** (-torch.arange(0, 64, 2) / 64)).cuda()
    same(G.gdn_qk_norm(q, k, inv_freq=freq), G.gdn_qk_norm(fq, fk, inv_freq=freq))
    dq, dk = rand(12, *q.shape), rand(13, *k.shape)
    same(G.gdn_qk_norm_bwd(q, k, dq, dk, inv_freq=freq), G.gdn_qk_norm_bwd(fq, fk, dq, dk, inv_freq=freq))


@pytest.mark.parametrize("D", [64, 40 * 1024])
def test_pages_beyond_32_bits(D):
    """(few sequences, and as many channels as take the form for large calls)"""
    P, S = 10, 16
    pages = torch.tensor([9, 0, -1, 8, 5], dtype=torch.int32).cuda()
    N = pages.numel()
    x, dt, b, c = rand(0, N, D), rand(1, N, D), rand(2, N, 1, S), rand(3, N, 1, S)
    A_log = rand(4, D, S, dtype=torch.float32)
    pool = rand(5, P, D, S, dtype=torch.float32)
    base = torch.empty(P * FAR, dtype=torch.float32, device="cuda")
    wide = base.as_strided((P, D, S), (FAR, S, 1))
    wide.copy_(pool)
    y, _ = G.gdn_ssm_step(x, dt, A_log, b, c, pool, pages, dt_softplus=True)
    far_y, _ = G.gdn_ssm_step(x, dt, A_log, b, c, wide, pages, dt_softplus=True)
    assert torch.equal(y, far_y) and torch.equal(pool, wide)
    w = rand(6, D, 4, dtype=torch.float32)
    pool = rand(7, P, 3, D)
    wide = base.view(torch.bfloat16).as_strided((P, 3, D), (FAR, D, 1))
    wide.copy_(pool)
    y, _ = G.gdn_conv_step(x, w, pool, pages=pages)
    far_y, _ = G.gdn_conv_step(x, w, wide, pages=pages)
    assert torch.equal(y, far_y) and torch.equal(pool, wide)


def test_most_sequences():
    """16384 sequences of one token, packed and as rows of a batch."""
    N, D, S = 16384, 24, 8
    cu = torch.arange(N + 1, dtype=torch.int32).cuda()
    i = scan_inputs(1, D, S, B=N)
    h0 = rand(20, N, D, S, dtype=torch.float32)
    j = {n: t if n in ("A_log", "bias") else t.reshape(1, N, *t.shape[2:]) for n, t in i.items()}
    a, b = scan(i, initial_state=h0), scan(j, initial_state=h0, cu_seqlens=cu, check=True)
    assert torch.equal(a[0].view(-1), b[0].view(-1)) and torch.equal(a[1], b[1])
    a = scan_bwd(i, initial_state=h0)
    b = scan_bwd(j, initial_state=h0, cu_seqlens=cu, check=True)
    for n in ("dx", "ddt", "db", "dc", "dgate", "dh0"):
        assert torch.equal(a[n].view(-1), b[n].view(-1)), n
    w, prev = rand(21, D, 4, dtype=torch.float32), rand(22, N, 3, D)
    a, b = G.gdn_conv_fwd(i["x"], w, None, prev), G.gdn_conv_fwd(j["x"], w, None, prev, cu, check=True)
    assert torch.equal(a[0].view(-1), b[0].view(-1)) and torch.equal(a[1], b[1])
    a = G.gdn_conv_bwd(i["x"], w, i["d_y"], None, prev)
    b = G.gdn_conv_bwd(j["x"], w, j["d_y"], None, prev, cu, check=True)
    for n in ("dx", "dx_prev"):
        assert torch.equal(a[n].view(-1), b[n].view(-1)), n


def test_most_channels():
    """2^20 channels: their last ones as by themselves."""
    D, S, n = 2 ** 20, 8, 264
    i = scan_inputs(3, D, S)
    j = {k: t if k in ("b", "c") else t[-n:] if t.dim() < 3 else t[..., -n:].contiguous() for k, t in i.items()}
    y, last = scan(i)
    small_y, small_last = scan(j)
    assert torch.equal(y[..., -n:], small_y) and torch.equal(last[:, -n:], small_last)
    w = rand(30, D, 4, dtype=torch.float32)
    y, _ = G.gdn_conv_fwd(i["x"], w)
    assert torch.equal(y[..., -n:], G.gdn_conv_fwd(j["x"], w[-n:])[0])
    g = G.gdn_conv_bwd(i["x"], w, i["d_y"])
    small = G.gdn_conv_bwd(j["x"], w[-n:], j["d_y"])
    assert torch.equal(g["dx"][..., -n:], small["dx"])


def test_most_heads():
    """4096 heads, 8 tokens of them together: as 64 tokens of 64 heads for each token."""
    T, D = 2440, 8
    q, k = rand(40, 1, T, 4096, D), rand(41, 1, T, 1, D)
    freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).cuda()
    pos = torch.arange(T, dtype=torch.int32).cuda()[None]
    w = rand(42, D, dtype=torch.float32)
    q1, k1 = G.gdn_qk_norm(q, k, w, w, pos, freq)
    q2, _ = G.gdn_qk_norm(q.view(1, T * 64, 64, D), k.repeat(1, 64, 1, 1), w, w,
                          pos.repeat_interleave(64, 1), freq)
    assert torch.equal(q1.view(-1), q2.view(-1))
    _, k3 = G.gdn_qk_norm(k, k, w, w, pos, freq)
    assert torch.equal(k1, k3)


def test_calls_at_once():
    """Backward passes of the scan on two streams, their states in tensor memory, beside linear
    attention's on a third, which uses it too: each as by itself."""
    cases = [scan_inputs(700, 1280, 16, seed=50), scan_inputs(900, 640, 32, seed=60)]
    alone = [scan_bwd(i) for i in cases]
    q, k, v = rand(70, 2, 1024, 8, 64), rand(71, 2, 1024, 8, 64), rand(72, 2, 1024, 8, 64)
    decay = -torch.rand(8, generator=torch.Generator().manual_seed(1)).cuda()
    attend = lambda s: G.gdn_lin_fwd(q, k, v, decay, stream=s)  # noqa: E731
    alone.append(attend(None))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for _ in range(6):
        got.append([scan_bwd(i, stream=s) for i, s in zip(cases, streams)] + [attend(streams[2])])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(alone, g):
            same(a, b) if not torch.is_tensor(a) else same([a], [b])
