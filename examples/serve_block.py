"""The block of train_block.py answering: the next token of up to 64 sequences, the library alone, in one CUDA graph.

    python examples/serve_block.py [--places 16] [--steps 50] [--bits 4]

Layer norm -> router product and choice -> the whole expert layer in one call,
added to the residual stream -> layer norm -> a vocabulary's logits from a
matrix in 4 bits. The batch has a fixed number of places, some of them empty:
an empty place's logits are masked, so it has no expert, no expert's weights
are read for it, and its row passes through. The experts' weights are those of
the trained block in bf16, or in 4 bits with a scale for each 64 rows of a
column.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import load_balancing_topk_gb300 as mep  # noqa: E402
from train_block import Block  # noqa: E402

GROUP = 64


class Server:
    """A trained block for `places` sequences; head: fp32 [H, V], kept in 4 bits."""

    def __init__(self, block, head, places, bits=4):
        self.block, self.places, self.V = block, places, head.shape[1]
        E, H, F, dev = block.E, block.H, block.F, head.device
        self.kind = dict(F=F, group=GROUP) if bits == 4 else {}
        self.w1, self.w2 = block.home["w1"], block.home["w2"]
        if bits == 4:
            self.w1, self.w2 = mep.mep_w4_save(self.w1, GROUP, parts=2), mep.mep_w4_save(self.w2, GROUP)
        self.head = mep.mep_w4_save(head, GROUP)
        # what the captured step reads and writes, and its scratch
        self.x = torch.zeros(places, H, dtype=torch.bfloat16, device=dev)
        self.empty = torch.ones(places, 1, dtype=torch.bool, device=dev)
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.scratch = torch.empty(max(mep.expert_layer_workspace_bytes(places, block.K, E, H, F, bits == 4, GROUP),
                                       mep.w4_product_workspace_bytes(places, H, self.V, GROUP)),
                                   dtype=torch.uint8, device=dev)
        self.graph = None

    def _step(self):
        b, P = self.block, self.block.params
        y, _, _ = mep.mep_layer_norm(self.x, P["norm_w"], P["norm_b"])
        logits = (y.float() @ P["router"]).masked_fill_(self.empty, -float("inf"))
        idx, w = mep.mep_route(logits, b.K, skip_masked=True)
        h = self.x + mep.mep_expert_layer(y, idx, w, self.w1, self.w2, self.status, workspace=self.scratch, **self.kind)
        z, _, _ = mep.mep_layer_norm(h)
        return h, mep.mep_w4_product(z, self.head, self.V, GROUP, dtype=torch.float32, status=self.status, workspace=self.scratch)

    def step(self, x, sequences):
        """x bf16 [n, H] into the places `sequences` (n of them); (residual stream, logits) of all places."""
        self.empty.fill_(True)
        self.empty[sequences] = False
        self.x[sequences] = x
        if self.graph is None:
            self._step()  # first calls of kernels and libraries are not captured
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.out = self._step()
        self.graph.replay()
        return self.out


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--places", type=int, default=16)
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--bits", type=int, default=4, choices=[4, 16])
    a = ap.parse_args()
    block = Block(R=8, S=1, K=6, E=64, B=8, H=2048, F=1408)
    g = torch.Generator(device="cuda").manual_seed(1)
    head = torch.randn(2048, 32768, generator=g, device="cuda") * 2048 ** -0.5
    server = Server(block, head, a.places, a.bits)
    x = torch.randn(a.places, 2048, generator=g, device="cuda").bfloat16()
    places = torch.arange(0, a.places, device="cuda")
    server.step(x, places)
    torch.cuda.synchronize()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        h, logits = server.step(x, places)
        x = h[places]
    end.record()
    torch.cuda.synchronize()
    status = int(server.status.item())
    if status:
        raise SystemExit(mep.STATUS[status])
    print(f"{a.places} sequences, experts in {a.bits} bits: {begin.elapsed_time(end) / a.steps * 1e3:.0f} us a step, "
          f"next tokens {logits.argmax(1).tolist()[:8]}")


if __name__ == "__main__":
    main()
