"""The causal convolution (include/wtconv_ssm.h) against its definition in fp64, and its refusals."""
import ctypes

import numpy as np
import pytest
import ssm_reference as R
import torch
from test_selective import FAKE, ODD, act, embed

from memory_bound_cnn_gb300 import ssm as M
from memory_bound_cnn_gb300 import wtconv as W

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
LAYOUTS = ["planes", "tokens"]


def make(B, T, C, K, layout, dtype, seed=0, lengths=None, silu=True, absent=()):
    """Inputs on the GPU; positions past a length hold NaN."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    shape = (B, T, C) if layout == "tokens" else (B, C, T)
    d = {"x": normal(*shape).to(dtype), "dy": normal(*shape).to(dtype), "w": normal(C, K), "bias": normal(C),
         "state": normal(B, C, K - 1).to(dtype), "d_last": normal(B, C, K - 1).to(dtype), "silu": silu, "lengths": None}
    for k in absent:
        d[k] = None
    if lengths is not None:
        d["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        past = torch.arange(T, device="cuda")[None, :] >= d["lengths"][:, None]
        for k in ("x", "dy"):
            d[k].masked_fill_(past[:, :, None] if layout == "tokens" else past[:, None, :], float("nan"))
    return d


def time_first(t, layout):
    return t.movedim(1 if layout == "tokens" else -1, 0)


def reference(d, layout):
    def array(t):
        return None if t is None else np.nan_to_num(t.double().cpu().numpy())

    ref = {"silu": d["silu"], "lengths": None if d["lengths"] is None else d["lengths"].cpu().numpy()}
    ref.update({k: array(time_first(d[k], layout)) for k in ("x", "dy")})
    ref.update({k: array(d[k]) for k in ("w", "bias", "state", "d_last")})
    return R.causal(ref)


def run(d, layout, y=None, dx=None, **kw):
    more = {**{k: d[k] for k in ("bias", "state", "lengths", "silu")}, "layout": layout}
    y, last = M.wtconv_causal_forward(d["x"], d["w"], **more, y=y, stream=kw.get("stream"))
    g = M.wtconv_causal_backward(d["x"], d["w"], d["dy"], d_last=d["d_last"], **more, dx=dx, **kw)
    return {"y": y, "last": last, **dict(zip(("dx", "dw", "d_bias", "d_state"), g))}


def check(got, want, layout, dtype, absent=()):
    for k in ("y", "dx"):
        R.assert_within(k, time_first(got[k], layout), *want[k], dtype)
    for k, kind in (("dw", torch.float32), ("d_bias", torch.float32), ("d_state", dtype)):
        if got[k] is None:
            assert {"d_bias": "bias", "d_state": "state"}[k] in absent
        else:
            R.assert_within(k, got[k], *want[k], kind)
    assert np.array_equal(got["last"].double().cpu().numpy(), want["last"][0])  # copies


def test_reference_gradients_match_differences():
    """Central differences of the fp64 forward."""
    rng = np.random.default_rng(5)
    T, B, C, K = 6, 4, 2, 4
    n = rng.standard_normal
    d = {"x": n((T, B, C)), "dy": n((T, B, C)), "w": n((C, K)), "bias": n(C), "state": n((B, C, K - 1)), "d_last": n((B, C, K - 1)),
         "lengths": np.array([6, 0, 1, 4]), "silu": True}

    def loss(d):
        r = R.causal(d)
        return np.sum(r["y"][0] * d["dy"]) + np.sum(r["last"][0] * d["d_last"])

    g = R.causal(d)
    for name, grad in (("x", "dx"), ("w", "dw"), ("bias", "d_bias"), ("state", "d_state")):
        for i in np.ndindex(*d[name].shape):
            up, down = ({**d, name: d[name].copy()} for _ in range(2))
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - g[grad][0][i]) < 1e-8, (name, i)


# ---------------------------------------------------------------------------- refusals (CPU)

def shape(B=2, T=16, C=8, K=4, layout=0, dtype=0, silu=1):
    return M.CausalShape(B, T, C, K, layout, dtype, silu)


def _forward(s=None, x=None, w=FAKE, bias=FAKE, state=FAKE, lengths=None, y=None, last=None):
    ref = ctypes.byref
    return M._load().wtconv_causal_forward(ref(s or shape()), ref(x or act()), w, bias, state, lengths, ref(y or act()), last, None)


def _backward(s=None, x=None, dy=None, dx=None, d_last=FAKE, dw=FAKE, db=FAKE, d_state=FAKE, ws=FAKE, nbytes=1 << 30):
    ref = ctypes.byref
    return M._load().wtconv_causal_backward(ref(s or shape()), ref(x or act()), FAKE, FAKE, FAKE, None, ref(dy or act()), d_last,
                                            ref(dx or act()), dw, db, d_state, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), W.ERR_INVALID_ARG), (dict(T=0), W.ERR_INVALID_ARG), (dict(C=-2), W.ERR_INVALID_ARG), (dict(K=1), W.ERR_UNSUPPORTED),
    (dict(K=5), W.ERR_UNSUPPORTED), (dict(T=(1 << 30) + 1), W.ERR_INVALID_ARG), (dict(B=1 << 16, C=1 << 15), W.ERR_INVALID_ARG),
    (dict(layout=2), W.ERR_INVALID_ARG), (dict(silu=2), W.ERR_INVALID_ARG), (dict(dtype=3), W.ERR_UNSUPPORTED)])
def test_shapes_are_refused(kw, status):
    s = shape(**kw)
    assert _forward(s) == _backward(s) == status
    assert M._load().wtconv_causal_workspace_size(ctypes.byref(s)) == 0


def test_calls_refuse(monkeypatch):
    bad = W.ERR_INVALID_ARG
    for kw in (dict(x=act(None)), dict(x=act(ODD)), dict(x=act(FAKE, -1)), dict(w=None), dict(w=ODD), dict(bias=ODD), dict(lengths=ODD),
               dict(state=ODD), dict(last=ODD), dict(y=act(None)), dict(y=act(FAKE, 64, 16)), dict(y=act(FAKE, 128, 15))):
        assert _forward(**kw) == bad, kw
    for kw in (dict(x=act(None)), dict(dy=act(None)), dict(dx=act(FAKE, 128, 8)), dict(d_last=ODD), dict(dw=None), dict(dw=ODD),
               dict(db=ODD), dict(d_state=ODD), dict(ws=ODD)):
        assert _backward(**kw) == bad, kw
    assert _backward(ws=None) == _backward(nbytes=1) == W.ERR_WORKSPACE
    ref = ctypes.byref

    def step(s=None, x=None, pool=FAKE, n=2, slots=None, y=None):
        return M._load().wtconv_causal_step(ref(s or shape()), ref(x or act()), FAKE, FAKE, pool, n, slots, ref(y or act()), None)

    assert step(pool=None) == step(pool=ODD) == step(n=1) == step(n=0, slots=FAKE) == step(slots=ODD) == bad
    assert step(y=act(FAKE, 0, 7)) == step(x=act(FAKE, 0, -1)) == step(shape(C=0)) == bad
    assert step(shape(K=1)) == W.ERR_UNSUPPORTED
    x = torch.zeros(2, 6, 4)
    with pytest.raises(ValueError, match="CUDA"):
        M.wtconv_causal_forward(x, torch.zeros(6, 4))
    with pytest.raises(ValueError, match="CUDA"):
        M.wtconv_causal_step(x[0], torch.zeros(4, 4), torch.zeros(6, 4, 3))
    monkeypatch.setenv("WTCONV_INJECT_FAULT", "1")
    assert step() == _forward() == _backward() == W.ERR_INJECTED


# ------------------------------------------------------------------------------------ the kernels

SIZES = [(1, 1, 1), (2, 2, 8), (3, 3, 5), (2, 5, 40), (1, 63, 64), (2, 64, 33), (2, 65, 16), (1, 200, 260), (4, 257, 12), (1, 1030, 72),
         (2, 3000, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, K, dtype, layout):
    d = make(*size, K, layout, dtype, seed=K)
    check(run(d, layout), reference(d, layout), layout, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,C", [(2, 8), (37, 9), (400, 64)])
def test_ragged_lengths(T, C, dtype, layout):
    """Lengths shorter than the taps, empty, full, too long and negative; NaN behind every end."""
    lengths = [0, 1, T, T + 5, -3, 2, 3, T // 2, T - 1]
    d = make(len(lengths), T, C, 4, layout, dtype, seed=5, lengths=lengths)
    got = run(d, layout)
    check(got, reference(d, layout), layout, dtype)
    assert (got["y"][0] == 0).all() and (got["dx"][4] == 0).all()
    assert torch.equal(got["last"][0], d["state"][0]) and torch.equal(got["d_state"][4], d["d_last"][4])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("absent", [("bias",), ("state",), ("d_last",), ("bias", "state", "d_last")], ids=str)
def test_optional_arguments(absent, silu, layout):
    d = make(2, 70, 24, 4, layout, torch.float32, seed=8, silu=silu, absent=absent)
    check(run(d, layout), reference(d, layout), layout, torch.float32, absent)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("before,pad", [(0, 8), (1, 0), (3, 5)])
def test_strides_and_alignment(before, pad, dtype, layout):
    d = make(3, 72, 40, 4, layout, dtype, seed=9)
    want = reference(d, layout)
    outs, bufs = {}, {}
    for k in ("y", "dx"):
        bufs[k], outs[k] = embed(torch.zeros_like(d["x"]), before, 7, pad, 2)
        bufs[k].fill_(-77.0)
    for i, k in enumerate(("x", "dy")):
        _, d[k] = embed(d[k], before + i * (before % 2), 4, pad, 2)
    check(run(d, layout, **outs), want, layout, dtype)
    for k in outs:
        inside = torch.zeros_like(bufs[k], dtype=torch.bool)
        inside.as_strided(outs[k].shape, outs[k].stride(), outs[k].storage_offset()).fill_(True)
        assert (bufs[k][~inside] == -77.0).all(), f"{k}: written outside its elements"


@pytest.mark.gpu
def test_views_and_images():
    d = make(4, 100, 64, 4, "tokens", torch.bfloat16, seed=10)
    want = reference(d, "tokens")
    both = torch.cat([d["x"], d["dy"]], 2)
    check(run({**d, "x": both[:, :, :64], "dy": both[:, :, 64:]}, "tokens"), want, "tokens", torch.bfloat16)
    turned = {**d, **{k: d[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ("x", "dy")}}
    check(run(turned, "tokens"), want, "tokens", torch.bfloat16)
    p = make(2, 144, 20, 3, "planes", torch.float16, seed=3)
    flat = run(p, "planes")
    got = run({**p, **{k: p[k].unflatten(-1, (12, 12)) for k in ("x", "dy")}}, "planes")
    assert all(torch.equal(got[k].reshape(v.shape), v) for k, v in flat.items())
    again = run(p, "planes")
    assert all(torch.equal(again[k], v) for k, v in flat.items())


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("cut", [1, 2, 41])
def test_pieces_compose(cut, layout):
    """A sequence in two calls, the first's last state the second's beginning, and the gradients back through both."""
    d = make(2, 90, 12, 4, layout, torch.float32, seed=6)
    want = reference(d, layout)
    axis = 1 if layout == "tokens" else -1
    x0, x1 = d["x"].split([cut, 90 - cut], axis)
    dy0, dy1 = d["dy"].split([cut, 90 - cut], axis)
    more = {"bias": d["bias"], "layout": layout}
    y0, s0 = M.wtconv_causal_forward(x0, d["w"], state=d["state"], **more)
    y1, s1 = M.wtconv_causal_forward(x1, d["w"], state=s0, **more)
    dx1, dw1, db1, ds1 = M.wtconv_causal_backward(x1, d["w"], dy1, state=s0, d_last=d["d_last"], **more)
    dx0, dw0, db0, ds0 = M.wtconv_causal_backward(x0, d["w"], dy0, state=d["state"], d_last=ds1, **more)
    check({"y": torch.cat([y0, y1], axis), "last": s1, "dx": torch.cat([dx0, dx1], axis), "dw": dw0 + dw1, "d_bias": db0 + db1,
           "d_state": ds0}, want, layout, torch.float32)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("B,C,K", [(1, 1, 2), (3, 70, 4), (5, 300, 3)])
def test_steps_equal_the_convolution(B, C, K, dtype):
    T = 6
    d = make(B, T, C, K, "tokens", dtype, seed=7)
    want = reference(d, "tokens")
    pool = torch.full((2 * B + 1, C, K - 1), 5.0, device="cuda", dtype=dtype)
    slots = torch.arange(2 * B - 1, -1, -2, dtype=torch.int32, device="cuda")
    pool[slots.long()] = d["state"]
    ys = [M.wtconv_causal_step(d["x"][:, t], d["w"], pool, d["bias"], slots) for t in range(T)]
    R.assert_within("y", torch.stack(ys), *want["y"], dtype)
    assert np.array_equal(pool[slots.long()].double().cpu().numpy(), want["last"][0])
    assert (pool[[i for i in range(2 * B + 1) if i not in slots.tolist()]] == 5.0).all()
    # idle sequences, no slots, no bias, no silu
    before = pool.clone()
    idle = slots.clone()
    idle[0] = 2 * B + 1
    y = M.wtconv_causal_step(d["x"][:, 0], d["w"], pool, None, idle, silu=False)
    assert (y[0] == 0).all() and torch.equal(pool[slots[0].long()], before[slots[0].long()])
    state = d["state"].clone()
    plain = make(B, T, C, K, "tokens", dtype, seed=7, silu=False, absent=("bias",))
    R.assert_within("y", M.wtconv_causal_step(d["x"][:, 0], d["w"], state, silu=False), *(v[0] for v in reference(plain, "tokens")["y"]), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_autograd_stream_and_graph(layout):
    d = make(2, 60, 20, 4, layout, torch.float32, seed=11)
    want = run(d, layout)
    leaves = {k: d[n].clone().requires_grad_() for k, n in (("x", "x"), ("weight", "w"), ("bias", "bias"), ("state", "state"))}
    y, last = M.causal_conv(**leaves, layout=layout)
    torch.autograd.backward([y, last], [d["dy"], d["d_last"]])
    for k, g in (("x", "dx"), ("weight", "dw"), ("bias", "d_bias"), ("state", "d_state")):
        assert torch.equal(leaves[k].grad, want[g]), k
    _, last = M.causal_conv(**leaves, layout=layout)
    last.sum().backward()
    y, _ = M.causal_conv(**leaves, layout=layout)
    (g,) = torch.autograd.grad(y.sum(), leaves["x"], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = run(d, layout, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    other = make(2, 60, 20, 4, layout, torch.float32, seed=12)
    want = run(other, layout)
    with torch.cuda.graph(graph):
        got = run(d, layout)
    for k in ("x", "dy", "w", "bias", "state", "d_last"):
        d[k].copy_(other[k])
    graph.replay()
    assert all(torch.equal(got[k], want[k]) for k in want)
