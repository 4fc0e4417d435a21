"""Train a small block of WTConv layers and a gated scan, then serve its scan pixel by pixel.

Two WTConv layers turn an image's planes into values and gates, the gated scan carries them over
all pixels in reading order, and the block learns the running mean of its input, which no local
filter can compute.  Every step runs on the library's kernels: the layers' forward and backward, the
scan's, the norm over all gradients and one AdamW update of every parameter, clipped by that norm on
the device.

With ``--mixer selective`` the layers' planes join a residual stream of tokens instead, and a selective
scan takes the gated scan's place: the norm with the residual's addition, a short causal convolution, and a
scan whose steps and maps depend on the pixel.

    python examples/train_scan_block.py [--steps 60] [--state-bits 8] [--mixer gated]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from memory_bound_cnn_gb300 import (  # noqa: E402
    AdamW,
    WTConvFunction,
    causal_conv,
    gated_scan,
    rms_norm,
    selective_scan,
    wtconv_causal_step,
    wtconv_rms_forward,
    wtconv_scan_forward,
    wtconv_scan_step,
    wtconv_selective_step,
)
from memory_bound_cnn_gb300.inputs import LayerShape, make_inputs  # noqa: E402

PARAMS = ("base_w", "base_bias", "base_scale", "wavelet_w", "wavelet_scale")


def run_steps(forward, params, steps, state_bits, B, C, side, lr, seed, device):
    """Losses of `steps` steps of `forward`, which maps images to planes, and what it last returned beside them."""
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
        y, rest = forward(x)
        loss = (y.float() - target).square().mean()
        loss.backward()
        optimiser.step(clip=optimiser.grad_norm(max_norm=1.0))
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), rest


def make_layers(B, C, side, seed, device):
    shape = LayerShape(B, C, side, side, 2, 5, "bf16")
    return [{k: v.to(device).requires_grad_() for k, v in make_inputs(shape, seed + i).items() if k in PARAMS} for i in range(2)]


def train(steps=60, state_bits=8, B=8, C=16, side=32, lr=5e-3, seed=0, device="cuda"):
    """Losses of `steps` steps, and the block's scan inputs of the last one for serving."""
    layers = make_layers(B, C, side, seed, device)
    gate_bias = torch.full((C,), 2.0, device=device, requires_grad=True)
    params = [layer[k] for layer in layers for k in PARAMS] + [gate_bias]

    def forward(x):
        value, gate = (WTConvFunction.apply(x, *[layer[k] for k in PARAMS]) for layer in layers)
        y, _ = gated_scan(value, gate, gate_bias)
        return y, (value.detach(), gate.detach(), gate_bias.detach())

    return run_steps(forward, params, steps, state_bits, B, C, side, lr, seed, device)


def selective_params(C, N, seed, device):
    """Parameters of the selective mixer: decays of 1 to N a unit of step, steps of 0.01 to 0.1."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    step = 0.01 * 10 ** torch.rand(C, generator=gen, device=device)
    p = {"norm": torch.ones(C, device=device), "conv": torch.randn(C, 4, generator=gen, device=device) / 2,
         "conv_bias": torch.zeros(C, device=device), "maps": torch.randn(2 * N, C, generator=gen, device=device) / C ** 0.5,
         "A_log": torch.log(torch.arange(1, N + 1, device=device).float()).repeat(C, 1), "D": torch.ones(C, device=device),
         "dt_bias": torch.log(torch.expm1(step))}
    return {k: v.requires_grad_() for k, v in p.items()}


def selective_mixer(value, dt, residual, p):
    """Tokens (B, T, C): the stream after the layers' values are added to it, and the scan's output."""
    u, total = rms_norm(value, p["norm"], residual=residual)
    u, _ = causal_conv(u, p["conv"], p["conv_bias"], layout="tokens")
    maps = (u @ p["maps"].to(u.dtype).t()).unflatten(2, (2, 1, -1))
    y, _ = selective_scan(u, dt, -torch.exp(p["A_log"]), maps[:, :, 0], maps[:, :, 1], D=p["D"], dt_bias=p["dt_bias"], layout="tokens")
    return y, total


def train_selective(steps=60, state_bits=8, B=8, C=16, side=32, N=16, lr=5e-3, seed=0, device="cuda"):
    """As train(), with the selective mixer; returns its inputs and parameters for serving."""
    layers, p = make_layers(B, C, side, seed, device), selective_params(C, N, seed, device)
    params = [layer[k] for layer in layers for k in PARAMS] + list(p.values())

    def forward(x):
        value, dt = (WTConvFunction.apply(x, *[layer[k] for k in PARAMS]).flatten(2).transpose(1, 2).contiguous() for layer in layers)
        residual = x.flatten(2).transpose(1, 2).float().contiguous()
        y, total = selective_mixer(value, dt, residual, p)
        out = y.float() + total
        return out.transpose(1, 2).unflatten(2, (side, side)), (value.detach(), dt.detach(), residual, {k: v.detach() for k, v in p.items()})

    return run_steps(forward, params, steps, state_bits, B, C, side, lr, seed, device)


def serve_selective(value, dt, residual, p, pixels):
    """The mixer of the first pixels of every image, one pixel a call on pools of the convolution's and the scan's
    states: (B, pixels, C)."""
    B, _, C = value.shape
    A, weight = -torch.exp(p["A_log"]), p["maps"].to(value.dtype).t()
    conv_pool = torch.zeros(B, C, 3, dtype=value.dtype, device=value.device)
    pool = torch.zeros(B, C, A.shape[1], device=value.device)
    out = []
    for t in range(pixels):
        u, _, _ = wtconv_rms_forward(value[:, t], p["norm"], residual=residual[:, t])
        u = wtconv_causal_step(u, p["conv"], conv_pool, p["conv_bias"])
        maps = (u @ weight).unflatten(1, (2, 1, -1))
        out.append(wtconv_selective_step(u, dt[:, t], A, maps[:, 0], maps[:, 1], pool, D=p["D"], dt_bias=p["dt_bias"]))
    return torch.stack(out, 1)


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
    ap.add_argument("--mixer", default="gated", choices=("gated", "selective"))
    a = ap.parse_args()
    pixels = 40
    if a.mixer == "selective":
        losses, (value, dt, residual, p) = train_selective(a.steps, a.state_bits)
        print(f"loss: first {losses[0]:.4f}, last {losses[-1]:.4f}")
        served = serve_selective(value, dt, residual, p, pixels)
        with torch.no_grad():
            whole, _ = selective_mixer(value, dt, residual, p)
        print("served pixel by pixel, largest difference from the scan:", float((served.float() - whole[:, :pixels].float()).abs().max()))
        return
    losses, (value, gate, gate_bias) = train(a.steps, a.state_bits)
    print(f"loss: first {losses[0]:.4f}, last {losses[-1]:.4f}")
    served = serve(value, gate, gate_bias, pixels)
    whole, _, _ = wtconv_scan_forward(value, gate, gate_bias)
    print("served pixel by pixel, largest difference from the scan:",
          float((served.float() - whole.flatten(2)[:, :, :pixels].float()).abs().max()))


if __name__ == "__main__":
    main()
