"""Train a small block of WTConv layers and a gated scan, then serve its scan pixel by pixel.

Two WTConv layers turn an image's planes into values and gates, the gated scan carries them over
all pixels in reading order, and the block learns the running mean of its input, which no local
filter can compute.  Every step runs on the library's kernels: the layers' forward and backward, the
scan's, the norm over all gradients and one AdamW update of every parameter, clipped by that norm on
the device.

    python examples/train_scan_block.py [--steps 60] [--state-bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from memory_bound_cnn_gb300 import (  # noqa: E402
    AdamW,
    WTConvFunction,
    gated_scan,
    wtconv_scan_forward,
    wtconv_scan_step,
)
from memory_bound_cnn_gb300.inputs import LayerShape, make_inputs  # noqa: E402

PARAMS = ("base_w", "base_bias", "base_scale", "wavelet_w", "wavelet_scale")


def train(steps=60, state_bits=8, B=8, C=16, side=32, lr=5e-3, seed=0, device="cuda"):
    """Losses of `steps` steps, and the block's scan inputs of the last one for serving."""
    shape = LayerShape(B, C, side, side, 2, 5, "bf16")
    layers = [{k: v.to(device).requires_grad_() for k, v in make_inputs(shape, seed + i).items() if k in PARAMS}
              for i in range(2)]
    gate_bias = torch.full((C,), 2.0, device=device, requires_grad=True)
    params = [layer[k] for layer in layers for k in PARAMS] + [gate_bias]
    for p in params:
        p.grad = torch.zeros_like(p)  # fixed buffers, which autograd adds to
    optimiser = AdamW([p.detach() for p in params], [p.grad for p in params], state_bits=state_bits, lr=lr)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    position = torch.arange(1, side * side + 1, device=device).view(side, side)
    losses = []
    for _ in range(steps):
        x = (torch.randn(B, C, side, side, generator=gen, device=device) +
             2 * torch.randn(B, C, 1, 1, generator=gen, device=device)).bfloat16()
        target = x.float().flatten(2).cumsum(2).view_as(x) / position
        for p in params:
            p.grad.zero_()
        value, gate = (WTConvFunction.apply(x, *[layer[k] for k in PARAMS]) for layer in layers)
        y, _ = gated_scan(value, gate, gate_bias)
        loss = (y.float() - target).square().mean()
        loss.backward()
        optimiser.step(clip=optimiser.grad_norm(max_norm=1.0))
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), (value.detach(), gate.detach(), gate_bias.detach())


def serve(value, gate, gate_bias, pixels):
    """The scan of the first pixels of every image, one call per pixel on a pool of states."""
    B, C = value.shape[:2]
    pool = torch.zeros(B, C, device=value.device)
    value, gate = (t.flatten(2).permute(2, 0, 1).contiguous() for t in (value, gate))
    return torch.stack([wtconv_scan_step(value[t], gate[t], gate_bias, pool) for t in range(pixels)], 2)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state-bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    losses, (value, gate, gate_bias) = train(a.steps, a.state_bits)
    print(f"loss: first {losses[0]:.4f}, last {losses[-1]:.4f}")
    pixels = 40
    served = serve(value, gate, gate_bias, pixels)
    whole, _, _ = wtconv_scan_forward(value, gate, gate_bias)
    print("served pixel by pixel, largest difference from the scan:",
          float((served.float() - whole.flatten(2)[:, :, :pixels].float()).abs().max()))


if __name__ == "__main__":
    main()
