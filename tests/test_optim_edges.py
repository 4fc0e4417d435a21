"""Corners of AdamW and the gradient norm: streams, averages that are not finite, tensors that move."""
import pytest
import torch

from memory_bound_cnn_gb300 import optim as O


@pytest.mark.gpu
def test_given_stream_without_workspace():
    """The side stream is held up while the current one uses whatever memory it can get again: the norm's
    scratch, its result and new lists of values keep theirs."""
    g = torch.Generator(device="cuda").manual_seed(30)
    n = 2_000_000
    p, grad = torch.randn(n, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda")
    q = p.clone()
    opt, other = O.AdamW([p], [grad], state_bits=8), O.AdamW([q], [grad], state_bits=8)
    clip = opt.grad_norm(1.0)
    opt.step(clip=clip)
    m, v = opt.state_values()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    late = other.grad_norm(1.0, stream=side)
    for _ in range(8):
        torch.empty(other._norm_bytes, dtype=torch.uint8, device="cuda").fill_(0xff)
    other.step(clip=late, stream=side)
    late_m, late_v = other.state_values(stream=side)
    torch.cuda.synchronize()
    assert torch.equal(clip, late) and torch.equal(p, q) and torch.equal(m[0], late_m[0]) and torch.equal(v[0], late_v[0])
