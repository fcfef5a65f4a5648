"""Trains a two-layer mixture of experts in block-scaled FP8, then serves it
token by token.

    python examples/train_experts.py [--steps 60]

Per step and layer: the forward quantizes its own input
(lp_grouped_fwd_dyn); the saved input and the gradient are quantized along
the tokens, the gradient along its columns too (lp_r128_quant,
lp_r128_quant_dual); grad_X and grad_W are grouped products; one AdamW step
over both layers with 8-bit moments (lp_adamw) also writes the bf16 copies of
the new fp32 weights, from which lp_b128_quant makes the next step's FP8
weights.  Everything between these calls is elementwise.  The data is
synthetic: tokens with a given expert each, targets from a random teacher.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fp8_gemm_backward_amd as lp  # noqa: E402


class ExpertLinear:
    """G weights [N, K]: fp32 masters, 8-bit AdamW moments, FP8 working copies."""

    def __init__(self, G, N, K, gen):
        n = G * N * K
        self.master = torch.randn(G, N, K, generator=gen, device="cuda") * K ** -0.5
        self.copy = self.master.bfloat16()
        self.grad = torch.empty_like(self.copy)
        self.moments = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.zeros(-(-n // 128), device="cuda") for _ in range(2)]
        self.weight = lp.lp_b128_quant(self.copy)

    def forward(self, x, offsets):
        return lp.lp_grouped_fwd_dyn(x, self.weight, offsets)

    def backward(self, x, grad_out, offsets, need_dx=True):
        grad_cols, grad_rows = lp.lp_r128_quant_dual(grad_out, offsets)
        x_rows = lp.lp_r128_quant(x, -2, offsets)
        lp.lp_grouped_bwd(grad_rows, x_rows, None, offsets, need_dx=False, grad_w=self.grad)
        return lp.lp_grouped_bwd(grad_cols, None, self.weight, offsets, need_dw=False)[0] if need_dx else None

    def requantize(self):
        lp.lp_b128_quant(self.copy, self.weight.codes, self.weight.scales)


def adamw(layers, weight_decay):
    return lp.AdamWPlan([m.master for m in layers], [m.grad for m in layers], [m.moments[0] for m in layers],
                        [m.moments[1] for m in layers], exp_avg_scales=[m.scales[0] for m in layers],
                        exp_avg_sq_scales=[m.scales[1] for m in layers], copies=[m.copy for m in layers],
                        weight_decay=weight_decay)


def train(steps=60, experts=8, tokens=2000, width=512, hidden=1024, seed=0):
    """Returns the layers, the tokens with their offsets, and the loss before every step and after the last."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    up, down = ExpertLinear(experts, hidden, width, gen), ExpertLinear(experts, width, hidden, gen)
    share = torch.rand(experts, generator=gen, device="cuda").square()
    share[experts // 2] = 0                                  # an expert without tokens
    sizes = (share / share.sum() * tokens).floor().long()
    offsets = sizes.cumsum(0).to(torch.int32)
    rows = int(sizes.sum())
    x = torch.randn(rows, width, generator=gen, device="cuda").bfloat16()
    expert = torch.repeat_interleave(torch.arange(experts, device="cuda"), sizes)
    teacher = torch.randn(experts, width, generator=gen, device="cuda")
    target = torch.tanh(x.float()) * teacher[expert]
    plan, losses = adamw([up, down], 0.01), []
    for step in range(1, steps + 2):
        h = up.forward(x, offsets)
        a = torch.relu(h)
        diff = down.forward(a, offsets).float() - target
        losses.append(diff.square().mean())
        if step > steps:
            break
        grad = (diff * (2.0 / diff.numel())).bfloat16()
        grad_a = down.backward(a, grad, offsets)
        up.backward(x, torch.where(h > 0, grad_a, 0), offsets, need_dx=False)
        lp.lp_adamw(plan, lr=2e-3, step=step)
        up.requantize()
        down.requantize()
    return up, down, x, offsets, [float(v) for v in losses]


def serve(up, down, token, expert):
    """One token [1, width] through its expert: the weights are streamed once, the token is quantized inside."""
    def one(layer):
        return lp.QTensor("fp8_b128", layer.weight.codes[expert:expert + 1], layer.weight.scales[expert:expert + 1])
    return lp.lp_linear_fwd_dyn(torch.relu(lp.lp_linear_fwd_dyn(token, one(up))), one(down))


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    steps = ap.parse_args().steps
    up, down, x, offsets, losses = train(steps)
    for k in range(0, steps + 1, max(steps // 6, 1)):
        print(f"step {k:4d}  loss {losses[k]:.4f}", flush=True)
    y = down.forward(torch.relu(up.forward(x, offsets)), offsets)
    row = int(offsets[0]) - 1                                 # the first expert's last token
    alone = serve(up, down, x[row:row + 1], 0)
    print(f"token {row} served alone: differs from the batch by {float((alone - y[row]).abs().max()):.2e} "
          f"of {float(y[row].abs().max()):.2f}")


if __name__ == "__main__":
    main()
