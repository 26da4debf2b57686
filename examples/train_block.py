"""A pre-norm mixture-of-experts block, trained with the library alone.

    python examples/train_block.py [--steps 20] [--tokens 1024]

Forward: layer norm -> router -> plan -> dispatch -> two grouped products with
the gated activation between them -> combine, added to the residual stream.
Backward: the gradients of all of it; the experts' weight gradients land in the
home experts' and slots' fp32 tensors and mep_reduce_grad folds them together.

What the backward pass needs is kept in 8 bits: the norm's input and output per
token, and the first projection's output per buffer row. The norm's output is
kept before dispatch and permuted again, as bytes, when its weight gradient is
due, so a token is kept once and not K times. Only the experts' outputs stay in
bf16 (the routing weights' gradients are dot products with them).
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import load_balancing_topk_gb300 as mep  # noqa: E402


class Block:
    """R ranks' worth of one block: E experts of width F, K a token, B slots a rank."""

    def __init__(self, R, S, K, E, B, H, F, seed=0, device="cuda"):
        self.R, self.S, self.K, self.E, self.B, self.H, self.F = R, S, K, E, B, H, F
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return scale * torch.randn(*shape, generator=g, device=device)

        # fp32 parameters and their gradients
        self.params = {
            "norm_w": torch.ones(H, device=device),
            "norm_b": torch.zeros(H, device=device),
            "router": normal(H, E, scale=H ** -0.5),
            "w1": normal(E, H, 2 * F, scale=H ** -0.5),
            "w2": normal(E, F, H, scale=F ** -0.5),
        }
        self.grads = {k: torch.zeros_like(v) for k, v in self.params.items()}
        # slot tensors: weights as the products read them, gradients as mep_reduce_grad reads them
        bf16, f32 = torch.bfloat16, torch.float32
        self.slot = {k: torch.zeros(R, B, *v, dtype=bf16, device=device) for k, v in
                     {"w1": (H, 2 * F), "w2": (F, H), "w1t": (2 * F, H), "w2t": (H, F)}.items()}
        self.slot_grad = {k: torch.zeros(R, B, *v, dtype=f32, device=device) for k, v in
                          {"w1": (H, 2 * F), "w2": (F, H)}.items()}
        rows = R * S * K
        self.kept = {
            "x": torch.empty(R * S, mep.ckpt_row_bytes(H), dtype=torch.uint8, device=device),
            "y": torch.empty(R * S, mep.ckpt_row_bytes(H), dtype=torch.uint8, device=device),
            "gu": torch.empty(rows, 2, mep.ckpt_row_bytes(F), dtype=torch.uint8, device=device),
        }
        self.load_weights()

    def load_weights(self):
        """The bf16 forms of the weights that the products read: as they are, and transposed for the backward pass."""
        w1, w2 = self.params["w1"].bfloat16(), self.params["w2"].bfloat16()
        self.home = {"w1": w1, "w2": w2, "w1t": w1.transpose(1, 2).contiguous(), "w2t": w2.transpose(1, 2).contiguous()}

    def _product(self, x, name):
        p = self.plan
        mep.mep_prefetch(p.slot_expert, self.home[name], self.slot[name], p.status, self.E)
        return mep.mep_grouped_gemm(x, p.cu_seqlens, self.home[name], self.slot[name], p.status, self.R, self.S, self.K)

    def forward(self, x):
        """x bf16 [R*S, H] -> x + experts(norm(x))."""
        P = self.params
        y, self.mean, self.rstd = mep.mep_layer_norm(x, P["norm_w"], P["norm_b"], x_ckpt=self.kept["x"],
                                                     y_ckpt=self.kept["y"])
        top, idx = torch.topk(y.float() @ P["router"], self.K, dim=1)
        self.idx, self.weight = idx.to(torch.int32), torch.softmax(top, 1)
        self.plan = p = mep.mep_plan(self.idx, self.R, self.S, self.K, self.E, self.B)
        buf = mep.mep_dispatch(y, p.dst_pos, p.status, self.R, self.S, self.K)
        a = mep.mep_swiglu(self._product(buf, "w1"), ckpt=self.kept["gu"])
        self.z = self._product(a, "w2")
        return x + mep.mep_combine(self.z, self.weight, p.dst_pos, p.status, self.R, self.S, self.K)

    def backward(self, dout):
        """Gradient of x from dout bf16 [R*S, H]; the parameters' gradients go to self.grads."""
        p, R, S, K, E = self.plan, self.R, self.S, self.K, self.E
        G, P = self.grads, self.params
        dz, dweight = mep.mep_combine_backward(dout, self.z, self.weight, p.dst_pos, p.status, R, S, K)
        da = self._product(dz, "w2t")
        dgu, a = mep.mep_swiglu_backward(da, self.kept["gu"])
        mep.mep_grouped_wgrad(a, dz, p.cu_seqlens, G["w2"], self.slot_grad["w2"], p.status, R, S, K)
        dbuf = self._product(dgu, "w1t")
        rows = mep.mep_dispatch(self.kept["y"].view(torch.bfloat16), p.dst_pos, p.status, R, S, K)
        mep.mep_grouped_wgrad(rows.view(torch.uint8), dgu, p.cu_seqlens, G["w1"], self.slot_grad["w1"], p.status,
                              R, S, K)
        for name in ("w1", "w2"):
            mep.mep_reduce_grad(p.slot_expert, G[name], self.slot_grad[name], p.status, E)
        dy = mep.mep_dispatch_backward(dbuf, p.dst_pos, p.status, R, S, K).float()
        # the router: softmax over the chosen logits, then a dense product
        dtop = self.weight * (dweight - (self.weight * dweight).sum(1, keepdim=True))
        dlogits = torch.zeros(R * S, E, device=dy.device).scatter_(1, self.idx.long(), dtop)
        y = mep.mep_ckpt_load(self.kept["y"], self.H)
        G["router"].copy_(y.float().t() @ dlogits)
        dy += dlogits @ P["router"].t()
        dx, _, _ = mep.mep_layer_norm_backward(dy.bfloat16(), self.kept["x"], P["norm_w"], self.mean, self.rstd,
                                               dweight=G["norm_w"], dbias=G["norm_b"])
        return dout + dx

    def step(self, rate):
        for k, v in self.params.items():
            v.add_(self.grads[k], alpha=-rate)
        self.load_weights()

    def bytes_kept(self):
        return sum(t.numel() for t in self.kept.values()) + self.z.numel() * 2


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1024, help="tokens a rank")
    a = ap.parse_args()
    block = Block(R=4, S=a.tokens, K=4, E=16, B=4, H=512, F=256)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(4 * a.tokens, 512, generator=g, device="cuda").bfloat16()
    target = x.float() + torch.tanh(x.float().roll(1, 1))
    for i in range(a.steps):
        diff = block.forward(x).float() - target
        block.backward((2 * diff / diff.numel()).bfloat16())
        block.step(rate=40.0)
        status = int(block.plan.status.item())
        if status:
            raise SystemExit(f"step {i}: {mep.STATUS[status]}")
        print(f"step {i}: loss {diff.square().mean().item():.5f}")
    rows = block.R * block.S * block.K
    plain = 2 * (block.R * block.S * block.H + rows * block.H + rows * 3 * block.F + rows * block.H)
    print(f"kept for the backward pass: {block.bytes_kept() / 2**20:.1f} MiB (in bf16 {plain / 2**20:.1f})")


if __name__ == "__main__":
    main()
