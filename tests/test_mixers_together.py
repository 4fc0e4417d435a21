"""The norm, the causal convolution and the selective scan in a row, as a block uses them: the example that trains and
serves with them, their gradients through one another, streams, graphs and very long tensors."""
import importlib.util
import os

import pytest
import torch

import memory_bound_cnn_gb300 as P

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
    losses, (value, dt, residual, p) = e.train_selective(steps=6, state_bits=state_bits, B=3, side=16)
    assert all(torch.isfinite(torch.tensor(losses)))
    served = e.serve_selective(value, dt, residual, p, 40).float()
    whole, _ = e.selective_mixer(value, dt, residual, p)
    whole = whole[:, :40].float()
    # Norm and convolution are the same operations in the same order or differ by fp32 units before a rounding to bf16 that may
    # then fall the other way: a unit of bf16 (2^-7) of u and of its maps, which reach y through u, B, C and d x: at
    # most 4 units of the largest value where many positions add up, and y's own rounding.
    assert (served - whole).abs().max() <= 5 * 2.0 ** -7 * whole.abs().max()


def plain_block(v, lengths=None):
    """The same in fp64 with elementary operations, position by position."""
    total = v["x"] + v["residual"]
    u = total / torch.sqrt(total.square().mean(-1, keepdim=True) + 1e-6) * v["norm"]
    padded = torch.cat([torch.zeros_like(u[:, :3]), u], 1)
    u = sum(v["conv"][:, k] * padded[:, k:k + u.shape[1]] for k in range(4)) + v["conv_bias"]
    u = u * torch.sigmoid(u)
    step = torch.nn.functional.softplus(v["dt"] + v["dt_bias"])
    maps = (u @ v["maps"].t()).unflatten(2, (2, -1))
    h, ys = 0, []
    for t in range(u.shape[1]):
        h = torch.exp(step[:, t, :, None] * v["A"]) * h + (step[:, t] * u[:, t])[..., None] * maps[:, t, 0, None]
        ys.append((h * maps[:, t, 1, None]).sum(-1) + v["D"] * u[:, t])
    z = v["z"]
    return torch.stack(ys, 1) * z * torch.sigmoid(z), total


def own_block(v, layout="tokens"):
    u, total = P.rms_norm(v["x"], v["norm"], residual=v["residual"])
    turn = (lambda t: t.transpose(1, 2).contiguous()) if layout == "planes" else (lambda t: t)
    u, _ = P.causal_conv(turn(u), v["conv"], v["conv_bias"], layout=layout)
    maps = (turn(u) @ v["maps"].t()).unflatten(2, (2, 1, -1))
    b, c = maps[:, :, 0], maps[:, :, 1]
    if layout == "planes":
        b, c = (t.permute(0, 2, 3, 1).contiguous() for t in (b, c))
    y, _ = P.selective_scan(u, turn(v["dt"]), v["A"], b, c, D=v["D"], z=turn(v["z"]), dt_bias=v["dt_bias"], layout=layout)
    return turn(y), total


def block_inputs(B=2, T=45, C=24, N=6, seed=0, dtype=torch.float64):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    v = {"x": n(B, T, C), "residual": n(B, T, C), "dt": n(B, T, C), "z": n(B, T, C), "norm": 1 + 0.2 * n(C), "conv": n(C, 4) / 2,
         "conv_bias": 0.1 * n(C), "maps": n(2 * N, C) / C ** 0.5, "A": -torch.exp(0.3 * n(C, N)), "D": n(C), "dt_bias": n(C) - 2}
    return {k: t.float().to(dtype).cuda() for k, t in v.items()}


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["tokens", "planes"])
def test_gradients_through_the_block(layout):
    """fp32 against autograd in fp64.  A value passes about 45 positions and 60 operations of 2^-24 each on its way, at
    worst in one direction, through factors of a few units: 1e-4 of the largest value of a gradient is allowed."""
    exact = {k: t.requires_grad_() for k, t in block_inputs().items()}
    own = {k: t.detach().float().requires_grad_() for k, t in exact.items()}
    g = torch.Generator(device="cuda").manual_seed(5)
    outs = plain_block(exact)
    gy, gt = (torch.randn(outs[0].shape, generator=g, device="cuda", dtype=torch.float64).float().double() for _ in range(2))
    torch.autograd.backward(outs, [gy, gt])
    got = own_block(own, layout)
    for a, b in zip(got, outs):
        assert (a.double() - b).abs().max() <= 1e-4 * b.abs().max()
    torch.autograd.backward(got, [gy.float(), gt.float()])
    for k in exact:
        assert (own[k].grad.double() - exact[k].grad).abs().max() <= 1e-4 * exact[k].grad.abs().max(), k


@pytest.mark.gpu
def test_two_graphs_and_eager_calls_in_turn():
    """Two captured graphs, each with memory of its own, and eager calls between their replays."""
    a, b, c = ({k: t.detach() for k, t in block_inputs(seed=s, T=200, dtype=torch.float32).items()} for s in (1, 2, 3))
    want = [own_block(v) for v in (a, b, c)]
    graphs, outs = [], []
    for v in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(own_block(v))
        graphs.append(graph)
    for _ in range(3):
        graphs[0].replay()
        eager = own_block(c)
        graphs[1].replay()
        graphs[0].replay()
    for got, w in ((outs[0], want[0]), (outs[1], want[1]), (eager, want[2])):
        assert all(torch.equal(x, y) for x, y in zip(got, w))


@pytest.mark.gpu
def test_streams_in_parallel():
    """The same calls on two streams at once, each with its own scratch."""
    inputs = [{k: t.detach() for k, t in block_inputs(seed=s, T=300, C=40, dtype=torch.float32).items()} for s in (1, 2)]
    want = [own_block(v) for v in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(own_block(inputs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, y) for r in got[i] for x, y in zip(r, want[i]))


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """Sequences that lie more than 2^32 bytes and 2^31 elements apart."""
    B, T, C, N = 2, 40, 24, 5
    gap = (1 << 31) + 64
    big = torch.empty(gap + T * C, dtype=torch.bfloat16, device="cuda")
    far = big.as_strided((B, T, C), (gap, C, 1))
    g = torch.Generator(device="cuda").manual_seed(3)
    near = torch.randn(B, T, C, generator=g, device="cuda").bfloat16()
    far.copy_(near)
    maps = torch.randn(B, T, 1, N, generator=g, device="cuda").bfloat16()
    A, w, norm = -torch.rand(C, N, generator=g, device="cuda"), torch.randn(C, 4, generator=g, device="cuda"), torch.ones(C, device="cuda")
    scan = lambda x: P.wtconv_selective_forward(x, near, A, maps, maps, z=x, layout="tokens")  # noqa: E731
    assert all(torch.equal(p, q) for p, q in zip(scan(far)[:2], scan(near)[:2]))
    conv = lambda x: P.wtconv_causal_forward(x, w, layout="tokens")  # noqa: E731
    assert all(torch.equal(p, q) for p, q in zip(conv(far), conv(near)))
    y = big.as_strided((B, T, C), (gap, C, 1))
    P.wtconv_selective_forward(near, near, A, maps, maps, layout="tokens", y=y)
    assert torch.equal(y, P.wtconv_selective_forward(near, near, A, maps, maps, layout="tokens")[0])
    rows = big.as_strided((2, T * C), (gap, 1))
    flat = near.reshape(2, -1)
    rows.copy_(flat)
    weight = norm.repeat(T)
    assert torch.equal(P.wtconv_rms_forward(rows, weight)[0], P.wtconv_rms_forward(flat, weight)[0])
