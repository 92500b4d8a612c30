"""Training steps of a two-layer perceptron whose linear layers run on
block-scaled 8-bit floats, then a single token through the trained layers.

Each step quantises the fp32 master weights (128 x 128 blocks), runs both
layers through ``fp8_linear`` (the quantised inputs are the products' operands
and all that is kept for the backward pass), and gives the optimizer the
gradients that ``weight_grad_fp8`` computes from those checkpoints.

Usage: python examples/fp8_mlp_step.py [--steps 20] [--tokens 4096] [--width 1024] [--hidden 4096]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import gemm_collective_tiles_gb300 as gct


class Layer:
    """fp32 master weights (K, N), their codes and scales, and a bias."""

    def __init__(self, K, N, generator):
        self.weight = (torch.randn(K, N, generator=generator, device="cuda") / K ** 0.5).requires_grad_()
        self.bias = torch.zeros(N, dtype=torch.bfloat16, device="cuda", requires_grad=True)
        self.codes, self.scales = gct.empty_fp8(K, N, "tiles")

    def quantize(self):
        gct.quantize_fp8(self.weight.detach(), self.codes, self.scales, block="tiles")

    def __call__(self, x, workspace):
        return gct.fp8_linear(x, self.codes, self.scales, self.weight, self.bias, workspace=workspace)


def train(steps=20, tokens=4096, width=1024, hidden=4096, rate=None, seed=0):
    """Fit a random linear map; returns the losses and the layers."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    up, down = Layer(width, hidden, g), Layer(hidden, width, g)
    target = torch.randn(width, width, generator=g, device="cuda") / width ** 0.5
    workspace = gct.Workspace(256)  # grows to what the layers need
    optimizer = torch.optim.Adam([up.weight, up.bias, down.weight, down.bias], lr=rate or 0.75 / width)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda")
        want = x @ target
        for layer in (up, down):
            layer.quantize()
        y = down(torch.relu(up(x.bfloat16(), workspace)), workspace)
        loss = ((y.float() - want) ** 2).mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
        if gct.query_status(workspace)[0]:
            raise RuntimeError("a product gave up waiting on the device")
    return losses, (up, down)


def one_token(layers, x):
    """The decode form: one row through the quantised layers, without autograd."""
    workspace = None
    for i, layer in enumerate(layers):
        layer.quantize()
        codes, scales = gct.empty_fp8(1, x.shape[1])
        gct.quantize_fp8(x, codes, scales)
        y = torch.empty(1, layer.codes.shape[1], dtype=torch.bfloat16, device="cuda")
        workspace = gct.matmul_fp8(codes, scales, layer.codes, layer.scales, y, bias=layer.bias.detach(), workspace=workspace)
        x = torch.relu(y) if i == 0 else y
    return x


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, default in (("steps", 20), ("tokens", 4096), ("width", 1024), ("hidden", 4096)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    losses, layers = train(a.steps, a.tokens, a.width, a.hidden)
    print("loss:", " ".join("%.4f" % v for v in losses))
    y = one_token(layers, torch.randn(1, a.width, device="cuda").bfloat16())
    print("one token:", tuple(y.shape), "finite" if torch.isfinite(y).all() else "not finite")
