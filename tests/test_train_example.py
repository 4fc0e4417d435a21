"""The example that trains and serves with the scan, AdamW and the gradient norm together."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("train_scan_block", os.path.join(ROOT, "examples", "train_scan_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.gpu
@pytest.mark.parametrize("state_bits", [32, 8])
def test_block_trains_and_serves(state_bits):
    e = example()
    losses, (value, gate, gate_bias) = e.train(steps=60, state_bits=state_bits)
    assert sum(losses[-5:]) < 0.5 * sum(losses[:5])
    served = e.serve(value, gate, gate_bias, 20).float()
    whole = e.wtconv_scan_forward(value, gate, gate_bias)[0].flatten(2)[:, :, :20].float()
    # both hold h in fp32 and round it once to bf16: a state near a rounding boundary may fall either way
    assert (served - whole).abs().max() <= 2.0 ** -8 * whole.abs().max()
    assert torch.isfinite(served).all()
