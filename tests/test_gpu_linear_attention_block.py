"""The example block on the GPU: its gradients against plain torch operations in
fp64, its loss, and its serving path against whole sequences.

Bounds, RMS: bf16 rounds each of the block's stages (projections, scores,
attention's output, norm's output, output projection) by at most 2^-8 / sqrt(3)
of it, which stays below 2^-6 over the forward's and the backward's stages
together; a head's output may cancel against its terms before the norm scales
it up again, for which another factor of 2 is allowed: 2^-5."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
BOUND = 2.0 ** -5


@pytest.fixture(scope="module")
def example():
    from deltaproduct_householder_product_gb300 import build
    build.build()
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "linear_attention_block.py")
    spec = importlib.util.spec_from_file_location("linear_attention_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def plain_attend(q, k, v, log_decay):
    T = q.shape[1]
    t = torch.arange(T, device=q.device)
    age = (t[:, None] - t[None, :]).double()
    weight = torch.where(age >= 0, torch.exp(age[None] * log_decay.double()[:, None, None]), 0.0)
    return torch.einsum("bthd,bshd,hts,bshe->bthe", q, k, weight, v)


def plain_norm(x, weight, bias, heads):
    g = x.view(x.shape[0], heads, -1)
    d = g - g.mean(-1, keepdim=True)
    h = (d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt()).view(x.shape)
    return torch.nn.functional.silu(h * weight + bias)


def rms(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).square().mean().sqrt() / b.square().mean().sqrt())


@pytest.mark.parametrize("heads,head_dim,length", [(3, 64, 130), (2, 128, 257), (4, 32, 31)], ids=str)
def test_gradients(example, heads, head_dim, length):
    torch.manual_seed(heads)
    block = example.Block(128, heads, head_dim).cuda()
    exact = example.Block(128, heads, head_dim, dtype=torch.float64).cuda()
    exact.load_state_dict(block.state_dict())
    exact.log_decay = block.log_decay
    x = torch.randn(2, length, 128, device="cuda", dtype=torch.bfloat16, requires_grad=True)
    x64 = x.detach().double().requires_grad_()
    dy = torch.randn(2, length, 128, device="cuda", dtype=torch.bfloat16)
    y = block(x)
    y.backward(dy)
    want = exact(x64, plain_attend, plain_norm)
    want.backward(dy.double())
    assert rms(y, want) <= BOUND
    assert rms(x.grad, x64.grad) <= BOUND
    for (name, p), q in zip(block.named_parameters(), exact.parameters()):
        assert rms(p.grad, q.grad) <= BOUND, name


def test_trains_and_serves(example):
    losses, off = example.main(steps=30, batch=4, length=200)
    assert losses[-1] < losses[0]
    assert off <= BOUND
