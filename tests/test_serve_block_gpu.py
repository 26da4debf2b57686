"""The serving example: the trained block's own forward pass and the captured step on the same tokens, the logits
against a product in 64 bits, places that come and go, and its gradient-free parts run together."""

import os
import sys

import pytest
import torch

import load_balancing_topk_gb300 as mep

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

from serve_block import GROUP, Server  # noqa: E402
from train_block import Block  # noqa: E402

pytestmark = pytest.mark.gpu


def make(places, bits, V=200, H=256, F=128):
    block = Block(R=2, S=places // 2, K=3, E=8, B=4, H=H, F=F, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    return block, Server(block, torch.randn(H, V, generator=g, device="cuda") * H ** -0.5, places, bits), g


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_a_step_is_the_trained_block():
    block, server, g = make(16, 16)
    x = torch.randn(16, 256, generator=g, device="cuda").bfloat16()
    h, logits = server.step(x, torch.arange(16, device="cuda"))
    want = block.forward(x)
    assert int(server.status) == 0 and int(block.plan.status) == 0
    # the block rounds gates, ups, activation, experts' outputs and their sum to bf16, the layer its result; both the new stream
    assert rel(h - x, want - x) < 6 * 2.0 ** -8
    z = torch.nn.functional.layer_norm(h.double(), (256,)).bfloat16()
    w = mep.mep_w4_load(server.head, 256, server.V, GROUP, dtype=torch.float32)
    # the norm's own rounding to bf16 may go the other way where fp32 and 64 bits differ
    assert rel(logits, z.double() @ w.double()) < 2.0 ** -8


@pytest.mark.parametrize("bits", [16, 4])
def test_places_come_and_go(bits):
    block, server, g = make(8, bits)
    x = torch.randn(8, 256, generator=g, device="cuda").bfloat16()
    alone = {}
    for t in range(8):
        h, logits = server.step(x[t:t + 1], torch.tensor([t], device="cuda"))
        alone[t] = (h[t].clone(), logits[t].clone())
        others = [s for s in range(t)]
        assert torch.equal(h[others], x[others])  # empty places pass through
    for places in ([0, 5, 7], [1, 2, 3, 4], list(range(8)), [6]):
        h, logits = server.step(x[places], torch.tensor(places, device="cuda"))
        for t in places:  # a token's result does not depend on who is beside it but for the order of its sums
            assert rel(h[t] - x[t], alone[t][0] - x[t]) < 2.0 ** -6 and rel(logits[t], alone[t][1]) < 2.0 ** -6
    assert int(server.status) == 0


def test_four_bits_stay_near_sixteen():
    """Quantisation noise: q within half a step, a step a seventh of the group's largest (about 0.37 of a normal weight's
    deviation): 0.11 of a weight in the root mean square, on either side of the gate and in the second product."""
    _, four, g = make(16, 4)
    _, sixteen, _ = make(16, 16)
    x = torch.randn(16, 256, generator=g, device="cuda").bfloat16()
    places = torch.arange(16, device="cuda")
    a, b = four.step(x, places)[0], sixteen.step(x, places)[0]
    assert 0.02 < rel(a - x, b - x) < 0.4
