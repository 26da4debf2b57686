"""The training example's block against automatic differentiation in 64 bits.

The same parameters (as the products read them, rounded to bf16), the same
routing and the same input. The block rounds every intermediate tensor to bf16
(off by 2^-9 rms or less of its size) and keeps three of them in 8 bits: a
value is off by up to half a step, the step at most 1/64 of its block's
largest value, which is about 3 standard deviations of 128 normal ones: an rms
error of 3/64/sqrt(12) = 1.4% of the standard deviation. A gradient meets at
most three of those (x, y or gate and up, the activation again) and about eight
roundings to bf16 in a chain: below 3% in the 2-norm, 5% is required.
"""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("train_block", os.path.join(ROOT, "examples", "train_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _plain(block, x):
    """The block's output in 64 bits, differentiable in its leaves."""
    leaves = {k: (v.bfloat16() if k in ("w1", "w2") else v).double().requires_grad_() for k, v in block.params.items()}
    x = x.double().requires_grad_()
    y = torch.nn.functional.layer_norm(x, (block.H,), leaves["norm_w"], leaves["norm_b"], 1e-5)
    idx = block.idx.long()
    weight = torch.softmax((y @ leaves["router"]).gather(1, idx), 1)
    out = torch.zeros_like(x)
    for e in range(block.E):
        token, k = (idx == e).nonzero(as_tuple=True)
        g, u = (y[token] @ leaves["w1"][e]).chunk(2, 1)
        z = (torch.nn.functional.silu(g) * u) @ leaves["w2"][e]
        out = out.index_add(0, token, weight[token, k].unsqueeze(1) * z)
    return x + out, x, leaves


def _rel(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("R,S,K,E,B,H,F", [(2, 96, 2, 8, 4, 128, 64), (4, 300, 3, 8, 2, 256, 128)])
def test_block_against_automatic_gradients(R, S, K, E, B, H, F):
    mod = _example()
    block = mod.Block(R, S, K, E, B, H, F, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    block.params["norm_w"].add_(0.2 * torch.randn(H, generator=g, device="cuda"))
    block.params["norm_b"].add_(0.2 * torch.randn(H, generator=g, device="cuda"))
    x = torch.randn(R * S, H, generator=g, device="cuda").bfloat16()
    dout = torch.randn(R * S, H, generator=g, device="cuda").bfloat16()
    out = block.forward(x)
    dx = block.backward(dout)
    assert int(block.plan.status.item()) == 0
    want, xl, leaves = _plain(block, x)
    want.backward(dout.double())
    assert _rel(out, want.detach()) < 0.05
    assert _rel(dx, xl.grad) < 0.05
    for name, leaf in leaves.items():
        assert _rel(block.grads[name], leaf.grad) < 0.05, name


def test_block_learns():
    mod = _example()
    block = mod.Block(2, 128, 2, 8, 4, 128, 64, seed=5)
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(256, 128, generator=g, device="cuda").bfloat16()
    target = x.float() + torch.tanh(x.float().roll(1, 1))
    losses = []
    for _ in range(10):
        diff = block.forward(x).float() - target
        block.backward((2 * diff / diff.numel()).bfloat16())
        block.step(rate=10.0)
        assert int(block.plan.status.item()) == 0
        losses.append(diff.square().mean().item())
    assert losses[-1] < 0.9 * losses[0], losses
