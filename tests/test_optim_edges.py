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


@pytest.mark.gpu
def test_averages_that_are_not_finite():
    """A finite gradient whose square passes fp32 makes its 8-bit block's v infinite, and NaN where the
    code is 0.  The parameters under a NaN become NaN at the next step: no finite step of any size."""
    p, g = torch.ones(600, device="cuda"), torch.full((600,), 1e-3, device="cuda")
    opt = O.AdamW([p], [g], state_bits=8)
    opt.step()
    g[300] = 2e19
    opt.step()
    bad = torch.isnan(opt.state_values()[1][0])
    assert int(bad[256:512].sum()) == 255 and int(bad.sum()) == 255
    g.fill_(1e-3)
    opt.step()
    assert torch.isnan(p[bad]).all() and torch.isfinite(p[~bad]).all() and float(p[~bad].abs().max()) < 1.01


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_nan_second_average_alone(bits):
    """v NaN beside a finite m, as states may be adopted: p is NaN there and nowhere else."""
    p, g = torch.ones(256, device="cuda"), torch.full((256,), 1e-3, device="cuda")
    opt = O.AdamW([p], [g], state_bits=bits)
    if bits == 32:
        opt.states["v"][0][100] = float("nan")
    else:
        opt.states["v_max"][0][0] = float("nan")
    opt.step()
    bad = torch.isnan(p)
    assert bad[100] and int(bad.sum()) == (1 if bits == 32 else 256)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_autograd_sees_a_step(bits):
    """A graph that saved a parameter, its working copy or a state before they were updated is refused."""
    p = torch.ones(600, device="cuda", requires_grad=True)
    copy = torch.ones(600, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(600, device="cuda", requires_grad=True)
    opt = O.AdamW([p.detach()], [torch.ones(600, device="cuda")], state_bits=bits, copies=[copy])
    losses = [(p * p).sum(), (copy * w).sum()]
    opt.step(clip=opt.grad_norm(1.0))
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            loss.backward()
    (p * p).sum().backward()  # a graph over the new values is as good as ever
    assert torch.equal(p.grad, 2 * p.detach())
    with torch.inference_mode():
        q = torch.ones(4, device="cuda")
        O.AdamW([q], [torch.ones(4, device="cuda")], state_bits=bits).step()
        assert (q < 1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_that_move(bits):
    """Parameters, gradients and copies that are given other memory are followed there; where that does not
    fit, the step is refused and nothing changes."""
    n = 3000
    p, other = torch.ones(n, device="cuda"), torch.full((n,), 7.0, device="cuda")
    g, copy = torch.full((n,), 0.5, device="cuda"), torch.ones(n, device="cuda").half()
    opt = O.AdamW([p], [g], state_bits=bits, copies=[copy])
    old = [t.data for t in (p, g, copy)]
    opt.step(clip=opt.grad_norm())
    p.data, other.data = other.data, p.data  # as a program that swaps averaged weights in does
    g.data, copy.data = torch.full((n,), -0.25, device="cuda"), torch.zeros(n, device="cuda").half()
    before = [t.clone() for t in old]
    clip = opt.grad_norm()
    assert abs(float(clip[0]) - 0.25 * n ** 0.5) < 1e-4
    opt.step(clip=clip)
    for a, b in zip(old, before):  # the memory that they had is left alone
        assert torch.equal(a, b)
    assert torch.equal(copy, p.half()) and (p != 7).all() and (p > 6.9).all()
    kept = p.clone()
    for t, bad in ((p, torch.ones(n + 1, device="cuda")), (g, torch.ones(n, device="cuda").bfloat16()), (p, torch.ones(n)),
                   (p, torch.ones(2 * n, device="cuda")[::2])):
        good = t.data
        t.data = bad
        with pytest.raises(ValueError, match=r"params\[0\]|grads\[0\]"):
            opt.step()
        t.data = good
    assert torch.equal(p, kept) and opt.count == 2
    opt.step()
    assert opt.count == 3 and not torch.equal(p, kept)


@pytest.mark.gpu
def test_shared_parameters_refuse():
    """A parameter that is given twice, or that lies within another, would be updated by two warps at once."""
    flat, grads = torch.ones(1000, device="cuda"), [torch.ones(500, device="cuda"), torch.ones(500, device="cuda")]
    for second in (flat[:500], flat[499:999]):
        with pytest.raises(ValueError, match=r"params\[0\] and params\[1\] share memory"):
            O.AdamW([flat[:500], second], grads)
    O.AdamW([flat[500:], flat[:500]], grads).step()
    assert (flat < 1).all()
    empty = flat[:0]
    O.AdamW([flat, empty, empty], [torch.ones(1000, device="cuda"), empty.clone(), empty.clone()]).step()


@pytest.mark.gpu
def test_values_of_32_bit_states():
    """Given lists are written in 32 bits as in 8; one that is not given is the states themselves."""
    p, g = torch.ones(30, 20, device="cuda"), torch.ones(600, device="cuda")
    opt = O.AdamW([p], [g])
    opt.step()
    m, v = [torch.zeros(600, device="cuda")], [torch.zeros(600, device="cuda")]
    got = opt.state_values(m, v)
    assert got[0] is m and got[1] is v
    assert torch.equal(m[0], opt.states["m"][0].view(-1)) and torch.equal(v[0], opt.states["v"][0].view(-1))
    assert float(m[0][0]) == pytest.approx(0.1) and opt.state_values(m)[1] is opt.states["v"]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    opt.step(stream=side)
    opt.state_values(m, stream=side)
    side.synchronize()
    assert torch.equal(m[0], opt.states["m"][0].view(-1))
    for bad in ([], [g[:1]], [g.half()], [torch.zeros(600)], [torch.zeros(1200, device="cuda")[::2]]):
        for bits in (32, 8):
            with pytest.raises(ValueError, match="v_out"):
                O.AdamW([p], [g], state_bits=bits).state_values(v_out=bad)
