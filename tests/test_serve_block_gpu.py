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


def test_tensors_that_are_mapped_must_be_the_devices_own():
    """Host memory, even pinned, behind a tensor map is refused by the library before anything is enqueued."""
    lib, T, K, N = mep.load_library(), 4, 64, 64
    dev = dict(dtype=torch.bfloat16, device="cuda")
    x, host = torch.zeros(T, K, **dev), torch.zeros(T, K, dtype=torch.bfloat16).pin_memory()
    w4, y = mep.mep_w4_save(torch.zeros(K, N, device="cuda")), torch.full((T, N), 3.0, **dev)
    ws = torch.empty(mep.w4_product_workspace_bytes(T, K, N), dtype=torch.uint8, device="cuda")
    bad = mep.STATUS_CODE["MEP_ERR_INVALID_ARG"]

    def product(x):
        return lib.mep_w4_product(x.data_ptr(), w4.data_ptr(), None, T, K, N, 128, ws.data_ptr(), ws.numel(), 0, y.data_ptr(), None)

    assert product(host) == bad and product(x) == 0
    idx, w = torch.zeros(T, 1, dtype=torch.int32, device="cuda"), torch.ones(T, 1, device="cuda")
    w1, w2, out = torch.zeros(2, K, 2 * N, **dev), torch.zeros(2, N, K, **dev), torch.empty(T, K, **dev)
    need = mep.expert_layer_workspace_bytes(T, 1, 2, K, N)
    room, host_room = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(need, dtype=torch.uint8).pin_memory()

    def layer(x, w1, ws):
        return lib.mep_expert_layer(x.data_ptr(), idx.data_ptr(), w.data_ptr(), w1.data_ptr(), w2.data_ptr(), 0, 128, None, T, 1, 2, K, N,
                                    ws.data_ptr(), ws.numel(), out.data_ptr(), None)

    assert layer(host, w1, room) == bad and layer(x, w1.cpu().pin_memory(), room) == bad and layer(x, w1, host_room) == bad
    assert layer(x, w1, room) == 0
    torch.cuda.synchronize()
