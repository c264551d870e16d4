"""One sparse MoE layer on 8-bit weights, with a router of its own, as a program would run it.

Serving: the router is an ordinary linear layer; its logits go to `route_logits` (sigmoid scores, a
balance bias, expert groups), the choice to the dispatch, 8-bit experts and the combine.
Training the router: the gradient of the combine weights and of a balance loss goes back through
`route_logits_backward` and the linear layer, and the balance bias follows the experts' loads.

    python examples/int8_layer.py [--tokens 64] [--steps 20]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_moe_layer_route_gb300 as M  # noqa: E402


class Int8MoeLayer:
    """Weights are prepared once; buffers and workspaces are kept for a number of tokens."""

    def __init__(self, tokens, d=512, experts=32, top_k=4, d_ff=256, n_shared=1, n_groups=8,
                 topk_groups=4, seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(n, rows, cols):
            return (torch.randn(n, rows, cols, generator=g, device=device) / rows ** 0.5).bfloat16()

        self.W_router = (torch.randn(d, experts, generator=g, device=device) / d ** 0.5)
        self.bias = torch.zeros(experts, device=device)
        mats = [M.quantize_channels(w(n, *shape)) for n, shape in
                ((experts, (d, d_ff)), (experts, (d, d_ff)), (experts, (d_ff, d)),
                 (n_shared, (d, d_ff)), (n_shared, (d, d_ff)), (n_shared, (d_ff, d)))]
        self.weights = M.make_int8_weights(*mats)
        self.cfg = M.MoeConfig.make(tokens, d, experts, top_k, d_ff, n_shared=n_shared)
        self.gate = M.GateConfig.make(tokens, experts, top_k, score=M.SCORE_SIGMOID,
                                      n_groups=n_groups, topk_groups=topk_groups, group_top2=True,
                                      renormalize=True, scale=2.5)
        i32 = dict(dtype=torch.int32, device=device)
        self.idx = torch.empty(tokens, top_k, **i32)
        self.topk_w = torch.empty(tokens, top_k, device=device)
        self.scores = torch.empty(tokens, experts, device=device)
        self.counts, self.offsets = torch.empty(experts, **i32), torch.empty(experts + 1, **i32)
        self.perm_slot = torch.empty(tokens * top_k, **i32)
        self.slot_pos = torch.empty(tokens * top_k, **i32)
        self.y_slot = torch.empty(tokens * (top_k + n_shared), d, dtype=torch.float16,
                                  device=device)
        self.out = torch.empty(tokens, d, dtype=torch.bfloat16, device=device)
        self.d_logits = torch.empty(tokens, experts, device=device)
        self.ws = M.alloc_workspace(self.cfg, device)
        self.ws8 = M.alloc_int8_workspace(M.grouped_ffn_int8_workspace_size(self.cfg), device)

    def forward(self, x):
        """x [tokens, d] bf16 to [tokens, d] bf16; everything is enqueued on the current stream."""
        self.logits = x.float() @ self.W_router
        M.route_logits(self.gate, self.logits, self.bias, self.idx, self.topk_w, self.scores)
        M.permute(self.cfg, self.idx, self.counts, self.offsets, self.perm_slot, self.slot_pos,
                  self.ws)
        M.grouped_ffn_int8(self.cfg, x, self.perm_slot, self.offsets, self.topk_w, self.weights,
                           self.y_slot, self.ws8)
        M.combine(self.cfg, self.y_slot, self.slot_pos, self.out, self.ws)
        return self.out

    def router_gradient(self, x, d_out, balance=0.01):
        """Gradient of the router's weights for d_out [tokens, d], the gradient of the layer's output,
        and of `balance` times the sum over experts of (share of choices) x (mean score). The experts'
        outputs are held fixed. Then moves the balance bias by the loads."""
        T, k = self.idx.shape
        # out[t] = sum_j topk_w[t, j] y[t, j] and the slot rows hold topk_w * y
        slot = self.y_slot[:T * k].view(T, k, -1).float()
        d_w = (slot * d_out.float()[:, None, :]).sum(-1) / self.topk_w.clamp_min(1e-20)
        share = self.counts.float() / (T * k)
        d_scores = (balance / T * share).expand(T, -1).contiguous()
        M.route_logits_backward(self.gate, self.logits, self.idx, d_w, d_scores, self.d_logits)
        M.bias_update(self.counts, self.bias, 0.99, 0.01)
        return x.float().t() @ self.d_logits


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer = Int8MoeLayer(a.tokens)
    x = torch.randn(a.tokens, layer.cfg.d, device="cuda").bfloat16()
    target = torch.randn(a.tokens, layer.cfg.d, device="cuda")
    for step in range(a.steps):
        out = layer.forward(x)
        d_out = (out.float() - target) * (2.0 / out.numel())
        loss = (out.float() - target).square().mean()
        layer.W_router -= 50.0 * layer.router_gradient(x, d_out)
        if step % 5 == 0 or step == a.steps - 1:
            load = layer.counts.float()
            print(f"step {step:3d}  loss {loss.item():.6f}  most loaded expert "
                  f"{(load.max() / load.mean()).item():.2f} x the mean")
    faults = M.device_status(layer.ws) | M.device_status(layer.ws8)
    assert faults == 0, f"device fault bits {faults:#x}"


if __name__ == "__main__":
    main()
