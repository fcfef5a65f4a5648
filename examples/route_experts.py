"""Trains a mixture of experts with its router in block-scaled FP8, then serves
it from 4-bit weights.

    python examples/route_experts.py [--steps 40]

Forward: the router's logits give every token its experts and weights
(lp_moe_gate); the pairs are sorted by expert (lp_moe_sort) and the tokens'
rows go to their experts straight as FP8, along both axes (lp_moe_gather_quant);
two grouped products with a ReLU between them; the rows come back by their
weights (lp_moe_combine).  Backward: the gradient goes to the experts' rows times
their weights, as FP8 (lp_moe_gather_quant), and into the weights
(lp_moe_combine_bwd), whose gradient goes on to the logits (lp_moe_gate_bwd); the
rows' gradient is summed by token (lp_moe_combine without weights).  One AdamW
step over the experts and the router.  A token is served by the same calls on
MXFP4 copies of the weights (lp_grouped_fwd_w4) and rows in bf16 (lp_moe_gather).
The data is synthetic: targets from a random teacher.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import fp8_gemm_backward_amd as lp  # noqa: E402
from train_experts import ExpertLinear, adamw  # noqa: E402


class Router:
    """[E, K]: an fp32 master with 8-bit AdamW moments; its bf16 copy makes fp32 logits."""

    def __init__(self, E, K, gen):
        n = E * K
        self.master = torch.randn(E, K, generator=gen, device="cuda") * K ** -0.5
        self.copy = self.master.bfloat16()
        self.grad = torch.empty_like(self.copy)
        self.moments = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(-(-n // 128), device="cuda") for _ in range(2)]

    def forward(self, x):
        return x.float() @ self.copy.float().T

    def backward(self, x, grad_logits):
        self.grad.copy_(grad_logits.T @ x.float())
        return grad_logits @ self.copy.float()


class RoutedExperts:
    """x [T, width] -> [T, width] through topk of E experts a token."""

    def __init__(self, experts, topk, width, hidden, gen):
        self.experts, self.topk = experts, topk
        self.router = Router(experts, width, gen)
        self.up, self.down = ExpertLinear(experts, hidden, width, gen), ExpertLinear(experts, width, hidden, gen)

    def forward(self, x, mask=None):
        """(y, what the backward needs).  mask [T, E]: added to the logits; -inf bars a token from an expert."""
        s = {"x": x, "logits": self.router.forward(x)}
        if mask is not None:
            s["logits"] += mask
        s["weights"], s["chosen"] = lp.lp_moe_gate(s["logits"], self.topk)
        s["offsets"], s["rows"], s["order"] = lp.lp_moe_sort(s["chosen"], self.experts)
        x_cols, s["x_rows"] = lp.lp_moe_gather_quant(x, s["order"], s["offsets"], self.topk)
        s["h"] = lp.lp_grouped_fwd(x_cols, self.up.weight, s["offsets"])
        s["a"] = torch.relu(s["h"])
        s["y"] = self.down.forward(s["a"], s["offsets"])
        return lp.lp_moe_combine(s["y"], s["rows"], s["weights"]), s

    def backward(self, grad, s):
        """The gradient of x; the weights' go to the layers' grad."""
        off = s["offsets"]
        _, grad_weights = lp.lp_moe_combine_bwd(grad, s["y"], s["rows"], s["weights"], need_dy=False)
        y_cols, y_rows = lp.lp_moe_gather_quant(grad, s["order"], off, self.topk, weights=s["weights"])
        lp.lp_grouped_bwd(y_rows, lp.lp_r128_quant(s["a"], -2, off), None, off, need_dx=False, grad_w=self.down.grad)
        grad_a = lp.lp_grouped_bwd(y_cols, None, self.down.weight, off, need_dw=False)[0]
        h_cols, h_rows = lp.lp_r128_quant_dual(torch.where(s["h"] > 0, grad_a, 0), off)
        lp.lp_grouped_bwd(h_rows, s["x_rows"], None, off, need_dx=False, grad_w=self.up.grad)
        grad_rows = lp.lp_grouped_bwd(h_cols, None, self.up.weight, off, need_dw=False)[0]
        grad_logits = lp.lp_moe_gate_bwd(grad_weights, s["logits"], s["weights"], s["chosen"])
        return lp.lp_moe_combine(grad_rows, s["rows"]).float() + self.router.backward(s["x"], grad_logits)

    def layers(self):
        return [self.router, self.up, self.down]

    def requantize(self):
        self.up.requantize()
        self.down.requantize()


class Served:
    """A trained layer's MXFP4 copy."""

    def __init__(self, layer):
        self.router, self.topk, self.experts = layer.router.copy.float(), layer.topk, layer.experts
        self.up, self.down = (lp.lp_mx_quant(m.copy, -1, "mxfp4") for m in (layer.up, layer.down))

    def forward(self, x, mask=None):
        logits = x.float() @ self.router.T
        if mask is not None:
            logits += mask
        weights, chosen = lp.lp_moe_gate(logits, self.topk)
        offsets, rows, _ = lp.lp_moe_sort(chosen, self.experts)
        h = lp.lp_grouped_fwd_w4(lp.lp_moe_gather(x, rows), self.up, offsets)
        return lp.lp_moe_combine(lp.lp_grouped_fwd_w4(torch.relu(h), self.down, offsets), rows, weights)


def train(steps=40, experts=8, topk=2, tokens=1000, width=256, hidden=512, seed=0):
    """Returns the layer, the tokens and the loss before every step and after the last."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = RoutedExperts(experts, topk, width, hidden, gen)
    x = torch.randn(tokens, width, generator=gen, device="cuda").bfloat16()
    target = torch.tanh(x.float() @ torch.randn(width, width, generator=gen, device="cuda") * width ** -0.5)
    plan, losses = adamw(layer.layers(), 0.01), []
    for step in range(1, steps + 2):
        y, saved = layer.forward(x)
        diff = y.float() - target
        losses.append(diff.square().mean())
        if step > steps:
            break
        layer.backward((diff * (2.0 / diff.numel())).bfloat16(), saved)
        lp.lp_adamw(plan, lr=2e-3, step=step)
        layer.requantize()
    return layer, x, [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    steps = ap.parse_args().steps
    layer, x, losses = train(steps)
    for k in range(0, steps + 1, max(steps // 5, 1)):
        print(f"step {k:4d}  loss {losses[k]:.4f}", flush=True)
    y, alone = layer.forward(x)[0], Served(layer).forward(x[:1])
    print(f"token 0 served from 4 bits: differs from the batch in 8 by {float((alone[0] - y[0]).norm() / y[0].norm()):.2f} of it")


if __name__ == "__main__":
    main()
