"""The gated scan (include/wtconv_scan.h) against its definition in fp64, and its refusals."""
import ctypes

import numpy as np
import pytest
import scan_reference as R
import torch

from memory_bound_cnn_gb300 import scan as S
from memory_bound_cnn_gb300 import wtconv as W

DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def make(B, T, C, layout, dtype, seed=0, lengths=None, h0=True, bias=(1.0, 6.0)):
    """Inputs on the GPU; positions past a length hold NaN."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    shape = (B, T, C) if layout == "tokens" else (B, C, T)

    def normal(*s):
        return torch.randn(*s, generator=g, device="cuda")

    d = {"x": normal(*shape).to(dtype), "gate": normal(*shape).to(dtype), "dy": normal(*shape).to(dtype),
         "gate_bias": torch.rand(C, generator=g, device="cuda") * (bias[1] - bias[0]) + bias[0],
         "h0": normal(B, C) if h0 else None, "dh_last": normal(B, C), "lengths": None}
    if lengths is not None:
        d["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        past = torch.arange(T, device="cuda")[None, :] >= d["lengths"][:, None]
        past = past[:, :, None] if layout == "tokens" else past[:, None, :]
        for k in ("x", "gate", "dy"):
            d[k].masked_fill_(past, float("nan"))
    return d


def reference(d, layout):
    x, gate, dy = (R.time_first(d[k], layout) for k in ("x", "gate", "dy"))
    x, gate, dy = (np.nan_to_num(v) if d["lengths"] is not None else v for v in (x, gate, dy))
    bias = d["gate_bias"].double().cpu().numpy()
    h0 = None if d["h0"] is None else d["h0"].double().cpu().numpy()
    n = None if d["lengths"] is None else d["lengths"].cpu().numpy()
    dh = None if d["dh_last"] is None else d["dh_last"].double().cpu().numpy()
    y, h_last, before = R.forward(x, gate, bias, h0, n)
    return {"y": y, "h_last": h_last, "before": before, **R.backward(x, gate, bias, dy, h0, dh, n)}


def run(d, layout, **kw):
    y, h_last, states = S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], d["h0"], d["lengths"], layout,
                                              keep_states=True)
    dx, dg, db, dh0 = S.wtconv_scan_backward(d["x"], d["gate"], d["gate_bias"], states, d["dy"], d["dh_last"],
                                             d["lengths"], layout, **kw)
    return {"y": y, "h_last": h_last, "states": states, "dx": dx, "d_gate": dg, "d_gate_bias": db, "d_h0": dh0}


def check(got, want, layout, dtype):
    for k in ("y", "dx", "d_gate"):
        R.assert_near(k, R.time_first(got[k], layout), want[k], dtype)
    for k in ("h_last", "d_h0"):
        R.assert_near(k, got[k].double().cpu().numpy(), want[k])
    R.assert_near("d_gate_bias", got["d_gate_bias"].double().cpu().numpy(), want["d_gate_bias"],
                  scale=want["abs"].max())
    states = R.time_first(got["states"], layout)
    R.assert_near("states", states, want["before"][::S.SCAN_KEEP])


# -------------------------------------------------------------------------- the definition (CPU)

def test_reference_gradients_match_differences():
    """Central differences of the fp64 forward: truncation ~ 1e-10, cancellation ~ 1e-16 / 1e-5."""
    rng = np.random.default_rng(3)
    T, B, C = 5, 3, 2
    v = {"x": rng.standard_normal((T, B, C)), "gate": rng.standard_normal((T, B, C)),
         "gate_bias": rng.standard_normal(C), "h0": rng.standard_normal((B, C))}
    dy, dh, n = rng.standard_normal((T, B, C)), rng.standard_normal((B, C)), np.array([5, 0, 3])
    live = (np.arange(T)[:, None] < n)[:, :, None]

    def loss(v):
        y, h, _ = R.forward(v["x"], v["gate"], v["gate_bias"], v["h0"], n)
        return np.sum(np.where(live, y * dy, 0.0)) + np.sum(h * dh)

    g = R.backward(v["x"], v["gate"], v["gate_bias"], dy, v["h0"], dh, n)
    for name, grad in (("x", "dx"), ("gate", "d_gate"), ("gate_bias", "d_gate_bias"), ("h0", "d_h0")):
        for i in np.ndindex(*v[name].shape):
            up, down = ({**v, name: v[name].copy()} for _ in range(2))
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - g[grad][i]) < 1e-8, (name, i)


# ---------------------------------------------------------------------------- refusals (CPU)

FAKE = ctypes.c_void_p(256)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p(258)


def _forward(B=2, T=16, C=8, layout=0, dtype=0, x=FAKE, x_st=(128, 16), gate=FAKE, bias=FAKE, h0=None, lengths=None,
             y=FAKE, y_st=(128, 16), h_last=None, states=None):
    return S._load().wtconv_scan_forward(B, T, C, layout, dtype, x, *x_st, gate, 128, 16, bias, h0, lengths, y, *y_st,
                                         h_last, states, None, 0, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), W.ERR_INVALID_ARG), (dict(T=0), W.ERR_INVALID_ARG), (dict(C=-1), W.ERR_INVALID_ARG),
    (dict(T=(1 << 30) + 1), W.ERR_INVALID_ARG), (dict(B=1 << 16, C=1 << 15), W.ERR_INVALID_ARG),
    (dict(layout=2), W.ERR_INVALID_ARG), (dict(dtype=3), W.ERR_UNSUPPORTED), (dict(x=None), W.ERR_INVALID_ARG),
    (dict(gate=None), W.ERR_INVALID_ARG), (dict(bias=None), W.ERR_INVALID_ARG), (dict(y=None), W.ERR_INVALID_ARG),
    (dict(x=ODD), W.ERR_INVALID_ARG), (dict(h0=ODD), W.ERR_INVALID_ARG), (dict(lengths=ODD), W.ERR_INVALID_ARG),
    (dict(states=ODD), W.ERR_INVALID_ARG), (dict(x_st=(-1, 16)), W.ERR_INVALID_ARG),
    (dict(x_st=(1 << 60, 16)), W.ERR_INVALID_ARG), (dict(y_st=(64, 16)), W.ERR_INVALID_ARG),
    (dict(y_st=(128, 15)), W.ERR_INVALID_ARG), (dict(y_st=(0, 16)), W.ERR_INVALID_ARG),
    (dict(y_st=(16, 16)), W.ERR_INVALID_ARG),
])
def test_forward_refuses(kw, status):
    assert _forward(**kw) == status


def test_backward_and_step_refuse():
    lib = S._load()
    act = (FAKE, 128, 16)

    def backward(states=FAKE, dx=act, db=FAKE, ws=FAKE, nbytes=1 << 20):
        return lib.wtconv_scan_backward(2, 16, 8, 0, 0, *act, *act, FAKE, states, None, *act, None, *dx, *act, db, None,
                                        ws, nbytes, None)

    assert backward(states=None) == W.ERR_INVALID_ARG
    assert backward(dx=(FAKE, 128, 8)) == W.ERR_INVALID_ARG
    assert backward(db=None) == W.ERR_INVALID_ARG
    assert backward(ws=ODD) == W.ERR_INVALID_ARG
    assert backward(nbytes=1) == W.ERR_WORKSPACE
    assert backward(ws=None) == W.ERR_WORKSPACE

    def step(B=4, C=8, dtype=1, pool=FAKE, n=4, slots=None, y_row=8):
        return lib.wtconv_scan_step(B, C, dtype, FAKE, 8, FAKE, 8, FAKE, pool, n, slots, FAKE, y_row, None)

    assert step(B=0) == W.ERR_INVALID_ARG
    assert step(pool=None) == W.ERR_INVALID_ARG
    assert step(n=3) == W.ERR_INVALID_ARG
    assert step(n=0, slots=FAKE) == W.ERR_INVALID_ARG
    assert step(slots=ODD) == W.ERR_INVALID_ARG
    assert step(y_row=7) == W.ERR_INVALID_ARG
    assert step(dtype=5) == W.ERR_UNSUPPORTED


def test_fault_injection_and_workspace_of_invalid_shapes(monkeypatch):
    assert S.wtconv_scan_workspace_size(S.OP_SCAN_BACKWARD, 0, 16, 8, 0, 0) == 0
    assert S.wtconv_scan_workspace_size(7, 2, 16, 8, 0, 0) == 0
    monkeypatch.setenv("WTCONV_INJECT_FAULT", "1")
    lib = S._load()
    assert lib.wtconv_scan_step(4, 8, 1, FAKE, 8, FAKE, 8, FAKE, FAKE, 4, None, FAKE, 8, None) == W.ERR_INJECTED
    act = (FAKE, 128, 16)
    assert lib.wtconv_scan_backward(2, 16, 8, 0, 0, *act, *act, FAKE, FAKE, None, *act, None, *act, *act, FAKE, None,
                                    FAKE, 1 << 20, None) == W.ERR_INJECTED


def test_binding_refuses():
    x = torch.zeros(2, 3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        S.wtconv_scan_forward(x, x, torch.zeros(3))
    with pytest.raises(ValueError, match="layout"):
        S.wtconv_scan_forward(x, x, torch.zeros(3), layout="rows")
    with pytest.raises(ValueError, match="CUDA"):
        S.wtconv_scan_step(x[0], x[0], torch.zeros(4), torch.zeros(3, 4))


# ------------------------------------------------------------------------------------ the kernels

SIZES = [(1, 1, 1), (2, 1, 8), (3, 2, 5), (1, 3, 64), (2, 31, 33), (2, 127, 16), (1, 128, 130), (2, 129, 3),
         (3, 255, 40), (1, 256, 64), (2, 257, 24), (2, 300, 77), (1, 1000, 96), (5, 784, 12), (1, 4097, 6), (2, 9001, 2)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype, layout):
    B, T, C = size
    d = make(B, T, C, layout, dtype, seed=T)
    check(run(d, layout), reference(d, layout), layout, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,C", [(37, 9), (400, 64), (2600, 20)])
def test_ragged_lengths(T, C, dtype, layout):
    """Empty, one-token, full, too long and negative lengths; NaN behind every end."""
    lengths = [0, 1, T, T + 5, -3, T // 2, 128 if T > 128 else 7, T - 1]
    d = make(len(lengths), T, C, layout, dtype, seed=5, lengths=lengths)
    got = run(d, layout)
    check(got, reference(d, layout), layout, dtype)
    assert torch.equal(got["h_last"][0], d["h0"][0]) and torch.equal(got["d_h0"][4], d["dh_last"][4])
    for k in ("y", "dx", "d_gate"):  # exact zeros behind the end
        assert (got[k][0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_optional_arguments(layout):
    d = make(2, 200, 24, layout, torch.float32, seed=8, h0=False)
    d["dh_last"] = None
    got = run(d, layout)
    check(got, reference(d, layout), layout, torch.float32)
    y, h_last, states = S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], layout=layout)
    assert states is None and torch.equal(y, got["y"]) and torch.equal(h_last, got["h_last"])


def embed(t, before, after, row_pad):
    """t's values in a larger NaN-filled buffer: padded rows, an odd start, other elements around."""
    B, R_, n = t.shape
    row = n + row_pad
    buf = torch.full((before + B * R_ * row + after,), float("nan"), dtype=t.dtype, device=t.device)
    view = buf.as_strided((B, R_, n), (R_ * row, row, 1), before)
    view.copy_(t)
    return buf, view


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("before,row_pad", [(0, 8), (1, 0), (3, 5), (8, 16)])
def test_strides_and_alignment(before, row_pad, dtype, layout):
    """Padded rows and odd starts, other ones for every tensor; nothing outside an output is written."""
    B, T, C = 3, 270, 40
    d = make(B, T, C, layout, dtype, seed=9)
    want = reference(d, layout)
    for i, k in enumerate(("x", "gate", "dy")):
        _, d[k] = embed(d[k], before + i * (before % 2), 4, row_pad)
    outs, bufs = {}, {}
    for k in ("y", "dx", "d_gate"):
        bufs[k], outs[k] = embed(torch.zeros_like(d["x"].contiguous()), before, 7, row_pad)
        bufs[k].fill_(-77.0)
    y, h_last, states = S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], d["h0"], None, layout, True, y=outs["y"])
    dx, dg, db, dh0 = S.wtconv_scan_backward(d["x"], d["gate"], d["gate_bias"], states, d["dy"], d["dh_last"], None,
                                             layout, dx=outs["dx"], d_gate=outs["d_gate"])
    got = {"y": y, "h_last": h_last, "states": states, "dx": dx, "d_gate": dg, "d_gate_bias": db, "d_h0": dh0}
    check(got, want, layout, dtype)
    for k in outs:
        inside = torch.zeros_like(bufs[k], dtype=torch.bool)
        inside.as_strided(outs[k].shape, outs[k].stride(), outs[k].storage_offset()).fill_(True)
        assert (bufs[k][~inside] == -77.0).all(), f"{k}: written outside its elements"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
def test_views_of_other_orders(dtype):
    """Halves of one projection; a time-first batch; one gate row repeated for every sequence."""
    B, T, C = 4, 150, 64
    d = make(B, T, C, "tokens", dtype, seed=10)
    want = reference(d, "tokens")
    both = torch.cat([d["x"], d["gate"]], 2)
    first = {**d, "x": both[:, :, :C], "gate": both[:, :, C:]}
    check(run(first, "tokens"), want, "tokens", dtype)
    turned = {**d, **{k: d[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "gate", "dy")}}
    check(run(turned, "tokens"), want, "tokens", dtype)
    shared = {**d, "gate": d["gate"][:1].expand(B, T, C)}
    check(run(shared, "tokens"), reference(shared, "tokens"), "tokens", dtype)


@pytest.mark.gpu
def test_image_planes_equal_flat_planes():
    d = make(2, 28 * 28, 12, "planes", torch.bfloat16, seed=11)
    flat = run(d, "planes")
    d4 = {**d, **{k: d[k].view(2, 12, 28, 28) for k in ("x", "gate", "dy")}}
    got = run(d4, "planes")
    for k in flat:
        assert torch.equal(got[k].reshape(flat[k].shape), flat[k]), k
    assert got["y"].shape == (2, 12, 28, 28)
    with pytest.raises(ValueError, match="contiguous"):
        S.wtconv_scan_forward(d4["x"].transpose(2, 3), d4["gate"], d["gate_bias"])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_offsets_past_32_bits(layout):
    """Sequences more than 2^31 elements apart, and rows more than 2^31 bytes apart."""
    B, T, C = 2, 130, 16
    d = make(B, T, C, layout, torch.bfloat16, seed=12)
    want = reference(d, layout)
    n_in = d["x"].shape[2]
    batch = (1 << 31) + 24
    store = torch.empty(batch + 16 * d["x"].shape[1] * n_in, dtype=torch.bfloat16, device="cuda")

    def far(t, start):
        view = store.as_strided(t.shape, (batch, n_in, 1), start)
        view.copy_(t)
        return view

    size = d["x"].shape[1] * n_in
    got = run({**d, "x": far(d["x"], 0), "gate": far(d["gate"], 2 * size), "dy": far(d["dy"], 4 * size)}, layout,
              dx=far(d["x"] * 0, 6 * size), d_gate=far(d["x"] * 0, 8 * size))
    check(got, want, layout, torch.bfloat16)
    del got, store


@pytest.mark.gpu
def test_gate_extremes():
    """Gates that hold, that reset and that lie beyond exp's range: a = 0 and a = 1 exactly."""
    z = torch.tensor([-200.0, -100.0, -88.8, -30.0, -1.0, 0.0, 1.0, 30.0, 88.8, 100.0, 200.0], device="cuda")
    T, C = 140, len(z)
    for layout in ("planes", "tokens"):
        d = make(2, T, C, layout, torch.float32, seed=13)
        d["gate_bias"] = z
        check(run(d, layout), reference(d, layout), layout, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_gradient_matches_differences_of_the_kernel(layout):
    """Along the gradient's own direction u: (L(v + e u) - L(v - e u)) / 2e = |grad|.  e |u| is small
    against the inputs: truncation (e^2) and fp32 rounding (1e-6 |L| / e) stay below 5e-3."""
    d = make(2, 300, 32, layout, torch.float32, seed=14)
    got = run(d, layout)

    def loss(v):
        y, h, _ = S.wtconv_scan_forward(v["x"], v["gate"], v["gate_bias"], v["h0"], None, layout)
        return float((y.double() * d["dy"].double()).sum() + (h.double() * d["dh_last"].double()).sum())

    for name, grad in (("x", "dx"), ("gate", "d_gate"), ("gate_bias", "d_gate_bias"), ("h0", "d_h0")):
        g = got[grad].double()
        size = float(g.norm())
        u = got[grad] / size
        e = 0.02 * float(d[name].double().norm())
        slope = (loss({**d, name: d[name] + e * u}) - loss({**d, name: d[name] - e * u})) / (2 * e)
        assert abs(slope - size) <= 5e-3 * size, (name, slope, size)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_autograd(layout):
    d = make(2, 200, 16, layout, torch.float32, seed=15, lengths=[200, 90])
    for k in ("x", "gate", "dy"):
        d[k] = torch.nan_to_num(d[k])
    want = reference(d, layout)
    x, bias, h0 = (d[k].clone().requires_grad_() for k in ("x", "gate_bias", "h0"))
    gate = d["gate"][:1].clone().requires_grad_()  # shared by the batch: its gradient is summed
    y, h = S.gated_scan(x, gate.expand_as(x), bias, h0, d["lengths"], layout)
    want = reference({**d, "gate": d["gate"][:1].expand_as(x)}, layout)
    torch.autograd.backward([y, h], [d["dy"], d["dh_last"]])
    R.assert_near("dx", R.time_first(x.grad, layout), want["dx"])
    R.assert_near("d_gate", R.time_first(gate.grad, layout), want["d_gate"].sum(1, keepdims=True))
    R.assert_near("d_gate_bias", bias.grad.double().cpu().numpy(), want["d_gate_bias"], scale=want["abs"].max())
    R.assert_near("d_h0", h0.grad.double().cpu().numpy(), want["d_h0"])
    y, h = S.gated_scan(x, gate.expand_as(x), bias, h0, d["lengths"], layout)  # a loss of h alone
    h.sum().backward()
    y, h = S.gated_scan(x, d["gate"], bias, None, None, layout)  # and of y alone
    y.sum().backward()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("B,C,n", [(1, 1, 1), (3, 7, 3), (8, 768, 20), (130, 33, 200), (2, 4100, 2)])
def test_step(B, C, n, dtype):
    """Single tokens on a pool: owned rows move, idle sequences and other rows do not."""
    g = torch.Generator(device="cuda")
    g.manual_seed(B * C)
    both = torch.randn(B, 2 * C + 1, generator=g, device="cuda").to(dtype)
    x, gate = both[:, :C], both[:, C:2 * C]
    bias = torch.rand(C, generator=g, device="cuda") * 4
    pool = torch.randn(n, C, generator=g, device="cuda")
    slots = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, n  # idle: outside the pool on either side
    before = pool.double().cpu().numpy()
    y = S.wtconv_scan_step(x, gate, bias, pool, slots)
    want, want_y = before.copy(), np.zeros((B, C))
    for b, s in enumerate(slots.tolist()):
        if 0 <= s < n:
            want_y[b], want[s], _ = R.forward(x[b].double().cpu().numpy()[None, None], gate[b].double().cpu().numpy()[None, None],
                                              bias.double().cpu().numpy(), before[s][None])
    R.assert_near("pool", pool.double().cpu().numpy(), want)
    R.assert_near("y", y.double().cpu().numpy(), want_y, dtype)
    if B > 2:
        assert (y[1] == 0).all() and (y[2] == 0).all()
        idle = sorted(set(range(n)) - set(slots.tolist()))
        assert np.array_equal(pool.double().cpu().numpy()[idle], before[idle])
    if n >= B:  # without slots: row b
        pool2 = torch.randn(n, C, generator=g, device="cuda")
        ref, _, _ = S.wtconv_scan_forward(x[:, None], gate[:, None], bias, pool2[:B].contiguous(), layout="tokens")
        assert torch.equal(S.wtconv_scan_step(x, gate, bias, pool2), ref[:, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_streams_graphs_and_repeats(layout):
    """Another stream, a captured graph and a second call give the first call's results bit for bit."""
    d = make(3, 1500, 48, layout, torch.bfloat16, seed=16, lengths=[1500, 700, 0])
    first = run(d, layout)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        other = run(d, layout)
    side.synchronize()
    for k in first:
        assert torch.equal(first[k], other[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(d, layout)
    for t in captured.values():
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    for k in first:
        assert torch.equal(first[k], captured[k]), k


@pytest.mark.gpu
def test_binding_refuses_on_the_gpu():
    d = make(2, 20, 8, "tokens", torch.float32)
    args = (d["x"], d["gate"], d["gate_bias"])
    with pytest.raises(ValueError, match="gate must match"):
        S.wtconv_scan_forward(d["x"], d["gate"].half(), d["gate_bias"], layout="tokens")
    with pytest.raises(ValueError, match="gate_bias"):
        S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"][:4], layout="tokens")
    with pytest.raises(ValueError, match="h0"):
        S.wtconv_scan_forward(*args, h0=d["h0"].half(), layout="tokens")
    with pytest.raises(ValueError, match="lengths"):
        S.wtconv_scan_forward(*args, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"), layout="tokens")
    with pytest.raises(ValueError, match="innermost"):
        S.wtconv_scan_forward(d["x"].transpose(1, 2), d["gate"].transpose(1, 2), d["gate_bias"])
    with pytest.raises(ValueError, match="empty"):
        S.wtconv_scan_forward(d["x"][:, :0], d["gate"][:, :0], d["gate_bias"], layout="tokens")
    with pytest.raises(W.WTConvError):  # rows of an output that overlap
        y = torch.empty(20 * 8 + 8, device="cuda").as_strided((2, 20, 8), (8, 8, 1))
        S.wtconv_scan_forward(*args, y=y, layout="tokens")
    with pytest.raises(ValueError, match="states"):
        S.wtconv_scan_backward(*args, None, d["dy"], layout="tokens")
    with pytest.raises(W.WTConvError) as e:
        S.wtconv_scan_backward(*args, torch.zeros(2, 1, 8, device="cuda"), d["dy"], layout="tokens",
                               workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == W.ERR_WORKSPACE
    with pytest.raises(W.WTConvError):  # more sequences than rows
        S.wtconv_scan_step(d["x"][0], d["gate"][0], d["gate_bias"], torch.zeros(4, 8, device="cuda"))


@pytest.mark.gpu
@pytest.mark.parametrize("B,C,T", [(2, 512, 1000), (3, 640, 4096), (16, 64, 777)])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
def test_shared_sequences(dtype, B, C, T):
    """Enough chains for clusters along time, too few to do without; no wait gives up."""
    lengths = [T, T // 3] + [T - 70 * b for b in range(2, B)]
    d = make(B, T, C, "tokens", dtype, seed=17, lengths=lengths)
    check(run(d, "tokens"), reference(d, "tokens"), "tokens", dtype)
    assert S.wtconv_scan_status() == W.OK


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_given_stream_and_workspace(layout):
    """An explicit stream and a caller's scratch of the size that is asked for, larger or misplaced."""
    d = make(2, 5000, 8, layout, torch.bfloat16, seed=18)
    want = run(d, layout)
    dims = (2, 5000, 8, {"planes": 0, "tokens": 1}[layout], 1)
    ws = [torch.empty(S.wtconv_scan_workspace_size(op, *dims) + 64, dtype=torch.uint8, device="cuda") for op in (0, 1)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, states = S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], d["h0"], None, layout, True, workspace=ws[0],
                                         stream=side)
    dx, dg, db, dh0 = S.wtconv_scan_backward(d["x"], d["gate"], d["gate_bias"], states, d["dy"], d["dh_last"], None, layout,
                                             workspace=ws[1], stream=side)
    side.synchronize()
    for k, t in (("y", y), ("h_last", h), ("states", states), ("dx", dx), ("d_gate", dg), ("d_gate_bias", db), ("d_h0", dh0)):
        assert torch.equal(t, want[k]), k
    with pytest.raises(ValueError, match="workspace"):
        S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], layout=layout, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    if ws[1].numel() > 64:
        with pytest.raises(W.WTConvError):
            S.wtconv_scan_backward(d["x"], d["gate"], d["gate_bias"], states, d["dy"], layout=layout, workspace=ws[1][8:])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("C", [4, 5, 12, 16, 17, 31, 67])
def test_few_channels_and_long_sequences(C, dtype, layout):
    """Narrow strips of tokens, segments of long rows, ragged ends in each of them."""
    T = 3000 + C
    d = make(3, T, C, layout, dtype, seed=C, lengths=[T, 1777, 63])
    check(run(d, layout), reference(d, layout), layout, dtype)
