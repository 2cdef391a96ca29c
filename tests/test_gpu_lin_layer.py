"""The example layer: linear attention, the gated norm and the state pages together,
in training and in serving."""
from __future__ import annotations

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "linear_attention_layer", os.path.join(ROOT, "examples", "linear_attention_layer.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_branches_equal_a_single_pass(example):
    """Token by token on forked, freed and compacted pages against one scan of the
    whole sequence.  Both round the attention's output and the norm's to bf16
    (2^-9 each) and the scan its weights and state too; the norm and the last
    product pass relative errors on: four roundings of 1.6e-3 root mean square on
    either side stay below 1e-2."""
    results, layer = example.serve()
    assert len(results) == 9 and {len(y) for _, y in results} == {5, 10}
    for x, y in results:
        want = example.whole(layer, x)[-len(y):].float()
        assert float((y.float() - want).norm() / want.norm()) <= 1e-2


def test_training_lowers_the_loss(example):
    losses = example.train(steps=25)
    assert losses[-1] < 0.8 * losses[0] and all(x == x for x in losses)


def test_gradients_of_the_whole_layer(example):
    """Against automatic differentiation of the same layer in plain 64-bit
    operations.  bf16 gradients pass some ten roundings of 1.6e-3 root mean square:
    2e-2."""
    layer = example.Layer(seed=3)
    x = torch.randn(2, 150, layer.width, generator=torch.Generator().manual_seed(4))
    x = x.cuda().bfloat16()
    way = torch.randn(x.shape, generator=torch.Generator().manual_seed(5)).cuda()
    (layer.train_forward(x).float() * way).sum().backward()

    w = [p.detach().double().requires_grad_() for p in layer.parameters()]
    xd = x.double()
    B, T, H, D = 2, 150, layer.heads, layer.head
    q, k, v, g = (xd @ w[0]).view(B, T, 4, H, D).unbind(2)
    age = torch.arange(T, device="cuda")
    age = (age[:, None] - age[None]).double()
    decay = torch.where(age >= 0, torch.exp(age * layer.log_decay.double()[:, None, None]), 0.0)
    scores = torch.einsum("bthd,bshd->bhts", q / D, k) * decay
    o = torch.einsum("bhts,bshd->bthd", scores, v)

    def norm(x, dims, weight, bias):
        m = x.mean(dims, keepdim=True)
        return (x - m) / (x.var(dims, unbiased=False, keepdim=True) + 1e-5).sqrt() * weight + bias

    silu = torch.nn.functional.silu
    y = norm(o, (3,), w[2].view(H, D), w[3].view(H, D)) * silu(g)
    y = y.reshape(B, T, -1) @ w[1] + xd
    u = norm(y.view(B, T, 8, -1), (1, 3), w[4].view(8, -1), w[5].view(8, -1))
    (silu(u).view(B, T, -1) * way.double()).sum().backward()
    for p, ref in zip(layer.parameters(), w):
        assert float((p.grad.double() - ref.grad).norm() / ref.grad.norm()) <= 2e-2
