"""The selective scan (include/wtconv_ssm.h) against its definition in fp64, and its refusals."""
import ctypes

import numpy as np
import pytest
import ssm_reference as R
import torch

from memory_bound_cnn_gb300 import scan as S
from memory_bound_cnn_gb300 import ssm as M
from memory_bound_cnn_gb300 import wtconv as W

DTYPES = [torch.float32, torch.bfloat16, torch.float16]
LAYOUTS = ["planes", "tokens"]
ACTIVATIONS = ("x", "dt", "z", "dy", "B", "C")


def make(B, T, C, N, layout, dtype, G=1, seed=0, lengths=None, softplus=True, absent=()):
    """Inputs on the GPU; positions past a length hold NaN."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    def shape(*inner):
        return (B, T, *inner) if layout == "tokens" else (B, *inner, T)

    d = {k: normal(*shape(C)).to(dtype) for k in ("x", "dt", "z", "dy")}
    d.update({k: normal(*shape(G, N)).to(dtype) for k in ("B", "C")})
    d["A"] = -(torch.arange(N, device="cuda") + 1) * torch.exp(0.2 * normal(C, N))
    step = 1e-3 * torch.exp(torch.rand(C, generator=gen, device="cuda") * 4.6)
    d["dt_bias"], d["D"], d["h0"], d["dh_last"] = torch.log(torch.expm1(step)), normal(C), normal(B, C, N), normal(B, C, N)
    if not softplus:
        d["dt"] = (d["dt"].abs().float() * (step if layout == "tokens" else step[:, None])).to(dtype)
        d["dt_bias"] = step
    d["lengths"], d["softplus"] = None, softplus
    for k in absent:
        d[k] = None
    if lengths is not None:
        d["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        past = torch.arange(T, device="cuda")[None, :] >= d["lengths"][:, None]
        for k in ACTIVATIONS:
            if d[k] is not None:
                view = [B] + [1] * (d[k].dim() - 1)
                view[1 if layout == "tokens" else -1] = T
                d[k].masked_fill_(past.view(view), float("nan"))
    return d


def time_first(t, layout):
    a = t.detach().double().cpu().numpy()
    return np.moveaxis(a, 1 if layout == "tokens" else -1, 0)


def reference(d, layout):
    ref = {"softplus": d["softplus"], "lengths": None if d["lengths"] is None else d["lengths"].cpu().numpy()}
    for name, k in (("x", "x"), ("dt", "dt"), ("z", "z"), ("dy", "dy"), ("Bm", "B"), ("Cm", "C")):
        ref[name] = None if d[k] is None else np.nan_to_num(time_first(d[k], layout))
    for k in ("A", "D", "dt_bias", "h0", "dh_last"):
        ref[k] = None if d[k] is None else d[k].double().cpu().numpy()
    return R.selective(ref)


def run(d, layout, stream=None, **out):
    inputs = [d[k] for k in ("x", "dt", "A", "B", "C")]
    more = {**{k: d[k] for k in ("D", "z", "dt_bias", "lengths", "softplus")}, "layout": layout, "stream": stream}
    y, h_last, states = M.wtconv_selective_forward(*inputs, h0=d["h0"], keep_states=True, y=out.pop("y", None), **more)
    names = ("dx", "d_dt", "dA", "dB", "dC", "dD", "dz", "d_dt_bias", "d_h0")
    grads = M.wtconv_selective_backward(*inputs, states, d["dy"], dh_last=d["dh_last"], **more, **out)
    return {"y": y, "h_last": h_last, **dict(zip(names, grads))}


def check(got, want, layout, dtype, absent=()):
    for k in ("y", "dx", "d_dt", "dB", "dC", "dz"):
        if got[k] is None:
            assert k == "dz" and "z" in absent
            continue
        value, bound = want[k]
        if dtype == torch.bfloat16 and k in want["cut"]:
            bound = bound + want["cut"][k]
        t = got[k].detach()
        t = t.movedim(1 if layout == "tokens" else -1, 0)
        R.assert_within(k, t, value, bound, dtype)
    for k in ("h_last", "dA", "d_h0", "dD", "d_dt_bias"):
        if got[k] is None:
            assert {"dD": "D", "d_dt_bias": "dt_bias"}[k] in absent
            continue
        R.assert_within(k, got[k], *want[k])


# -------------------------------------------------------------------------- the definition (CPU)

def test_reference_gradients_match_differences():
    """Central differences of the fp64 forward: truncation ~ 1e-9, cancellation ~ 1e-16 / 1e-5."""
    rng = np.random.default_rng(3)
    T, B, C, N, G = 5, 3, 4, 3, 2
    n = rng.standard_normal
    d = {"x": n((T, B, C)), "dt": n((T, B, C)), "z": n((T, B, C)), "Bm": n((T, B, G, N)), "Cm": n((T, B, G, N)), "A": -np.exp(n((C, N))),
         "D": n(C), "dt_bias": n(C), "h0": n((B, C, N)), "dy": n((T, B, C)), "dh_last": n((B, C, N)), "lengths": np.array([5, 0, 3]),
         "softplus": True}

    def loss(d):
        r = R.selective(d)
        return np.sum(r["y"][0] * d["dy"]) + np.sum(r["h_last"][0] * d["dh_last"])

    g = R.selective(d)
    for name, grad in (("x", "dx"), ("dt", "d_dt"), ("z", "dz"), ("Bm", "dB"), ("Cm", "dC"), ("A", "dA"), ("D", "dD"),
                       ("dt_bias", "d_dt_bias"), ("h0", "d_h0")):
        for i in np.ndindex(*d[name].shape):
            up, down = ({**d, name: d[name].copy()} for _ in range(2))
            up[name][i] += 1e-5
            down[name][i] -= 1e-5
            assert abs((loss(up) - loss(down)) / 2e-5 - g[grad][0][i]) < 1e-7, (name, i)


# ---------------------------------------------------------------------------- refusals (CPU)

FAKE, ODD = 256, 258  # aligned, never dereferenced: validation fails first


def shape(B=2, T=16, C=8, N=4, G=2, layout=0, dtype=0, softplus=1):
    return M.SelectiveShape(B, T, C, N, G, layout, dtype, softplus)


def inputs(**kw):
    act, maps = M.SsmTensor(FAKE, 128, 16), M.SsmTensor(FAKE, 128, 16)
    v = dict(x=act, dt=act, Bm=maps, Cm=maps, z=act, A=FAKE, D=FAKE, dt_bias=FAKE, h0=FAKE, lengths=None)
    return M.SelectiveInputs(**{**v, **kw})


def act(p=FAKE, batch=128, row=16):
    return M.SsmTensor(p, batch, row)


def _forward(s=None, y=None, h_last=None, states=None, ws=FAKE, nbytes=1 << 30, **kw):
    ref = ctypes.byref
    return M._load().wtconv_selective_forward(ref(s or shape()), ref(inputs(**kw)), ref(y or act()), h_last, states, ws, nbytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), W.ERR_INVALID_ARG), (dict(T=0), W.ERR_INVALID_ARG), (dict(C=-2), W.ERR_INVALID_ARG), (dict(N=0), W.ERR_INVALID_ARG),
    (dict(N=65), W.ERR_INVALID_ARG), (dict(G=0), W.ERR_INVALID_ARG), (dict(G=3), W.ERR_INVALID_ARG),
    (dict(T=(1 << 30) + 1), W.ERR_INVALID_ARG), (dict(B=1 << 16, C=1 << 15), W.ERR_INVALID_ARG),
    (dict(layout=2), W.ERR_INVALID_ARG), (dict(softplus=2), W.ERR_INVALID_ARG), (dict(dtype=3), W.ERR_UNSUPPORTED)])
def test_shapes_are_refused(kw, status):
    s = shape(**kw)
    assert _forward(s) == status
    assert M._load().wtconv_selective_workspace_size(1, ctypes.byref(s)) == 0
    act0 = act()
    ref = ctypes.byref
    grads = M.SelectiveGrads(act0, act0, act0, act0, act0, FAKE, FAKE, FAKE, FAKE)
    assert M._load().wtconv_selective_backward(ref(s), ref(inputs()), FAKE, ref(act0), None, ref(grads), FAKE, 1 << 40, None) == status


@pytest.mark.parametrize("kw", [
    dict(x=act(None)), dict(x=act(ODD)), dict(x=act(FAKE, -1)), dict(x=act(FAKE, 1 << 60)), dict(dt=act(None)), dict(Bm=act(None)),
    dict(Cm=act(ODD)), dict(z=act(ODD)), dict(A=None), dict(A=ODD), dict(D=ODD), dict(dt_bias=ODD), dict(h0=ODD), dict(lengths=ODD),
    dict(y=act(None)), dict(y=act(FAKE, 64, 16)), dict(y=act(FAKE, 128, 15)), dict(y=act(FAKE, 0, 16)), dict(h_last=ODD),
    dict(states=264)])
def test_forward_refuses(kw):
    assert _forward(**kw) == W.ERR_INVALID_ARG


def test_backward_and_step_refuse(monkeypatch):
    lib, ref, good = M._load(), ctypes.byref, act()

    def backward(states=FAKE, ws=FAKE, nbytes=1 << 30, dy=good, **kw):
        g = dict(dx=good, d_dt=good, dB=good, dC=good, dz=good, dA=FAKE, dD=FAKE, d_dt_bias=FAKE, d_h0=FAKE)
        return lib.wtconv_selective_backward(ref(shape()), ref(inputs()), states, ref(dy), None, ref(M.SelectiveGrads(**{**g, **kw})), ws,
                                             nbytes, None)

    assert backward(states=None) == backward(states=264) == W.ERR_INVALID_ARG
    for k in ("dx", "d_dt", "dB", "dC", "dz"):
        assert backward(**{k: act(None)}) == backward(**{k: act(FAKE, 128, 8)}) == W.ERR_INVALID_ARG
    for k in ("dA", "dD", "d_dt_bias", "d_h0"):
        assert backward(**{k: ODD}) == W.ERR_INVALID_ARG
    many = shape(B=1 << 16, T=1 << 30)  # a sum of 32 positions has a CTA of its own
    assert lib.wtconv_selective_workspace_size(S.OP_SCAN_BACKWARD, ref(many)) == 0
    g = M.SelectiveGrads(good, good, good, good, good, FAKE, FAKE, FAKE, FAKE)
    assert lib.wtconv_selective_backward(ref(many), ref(inputs()), FAKE, ref(good), None, ref(g), FAKE, 1 << 60, None) == W.ERR_INVALID_ARG
    assert backward(dA=None) == backward(dy=act(None)) == backward(ws=ODD) == W.ERR_INVALID_ARG
    assert backward(nbytes=1) == backward(ws=None) == W.ERR_WORKSPACE

    def step(s=None, pool=FAKE, n=2, slots=None, y=None, **kw):
        return lib.wtconv_selective_step(ref(s or shape()), ref(inputs(**kw)), pool, n, slots, ref(y or good), None)

    assert step(pool=None) == step(pool=ODD) == step(n=1) == step(n=0, slots=FAKE) == step(slots=ODD) == W.ERR_INVALID_ARG
    assert step(y=act(FAKE, 0, 7)) == step(x=act(FAKE, 0, -1)) == step(x=act(None)) == step(shape(B=0)) == W.ERR_INVALID_ARG
    assert step(shape(dtype=7)) == W.ERR_UNSUPPORTED
    monkeypatch.setenv("WTCONV_INJECT_FAULT", "1")
    assert step() == backward() == _forward() == W.ERR_INJECTED


def test_binding_refuses():
    x, m, A = torch.zeros(2, 6, 4), torch.zeros(2, 1, 3, 4), torch.zeros(6, 3)
    with pytest.raises(ValueError, match="CUDA"):
        M.wtconv_selective_forward(x, x, A, m, m)
    with pytest.raises(ValueError, match="layout"):
        M.wtconv_selective_forward(x, x, A, m, m, layout="rows")
    with pytest.raises(ValueError, match="CUDA"):
        M.wtconv_selective_step(x[0], x[0], A, m[0], m[0], torch.zeros(2, 6, 3))


# ------------------------------------------------------------------------------------ the kernels

SIZES = [(1, 1, 1, 1), (2, 1, 8, 16), (3, 2, 5, 3), (1, 15, 33, 16), (2, 16, 32, 8), (2, 17, 40, 13), (1, 31, 64, 16), (2, 32, 3, 64),
         (1, 33, 37, 33), (2, 100, 31, 20), (1, 128, 130, 4), (2, 257, 24, 16), (1, 600, 9, 64), (3, 300, 12, 9), (1, 2500, 6, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype, layout):
    B, T, C, N = size
    d = make(B, T, C, N, layout, dtype, seed=T)
    check(run(d, layout), reference(d, layout), layout, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
@pytest.mark.parametrize("B,T", [(1, 35), (2, 70)])
def test_one_channel(B, T, N, dtype, layout):
    """One channel with all the states of its lanes, whose rows of planes lie at any distance."""
    d = make(B, T, 1, N, layout, dtype, seed=N)
    check(run(d, layout), reference(d, layout), layout, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("C,G", [(6, 2), (70, 2), (96, 3), (4, 4)])
def test_groups(C, G, layout):
    d = make(2, 40, C, 5, layout, torch.bfloat16, G=G, seed=1)
    check(run(d, layout), reference(d, layout), layout, torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,C,N", [(37, 9, 16), (400, 40, 7), (2600, 5, 32)])
def test_ragged_lengths(T, C, N, dtype, layout):
    """Empty, one-token, full, too long and negative lengths; NaN behind every end."""
    lengths = [0, 1, T, T + 5, -3, T // 2, 128 if T > 128 else 7, T - 1]
    d = make(len(lengths), T, C, N, layout, dtype, seed=5, lengths=lengths)
    got = run(d, layout)
    check(got, reference(d, layout), layout, dtype)
    assert torch.equal(got["h_last"][0], d["h0"][0]) and torch.equal(got["d_h0"][4], d["dh_last"][4])
    for k in ("y", "dx", "d_dt", "dB", "dC", "dz"):  # exact zeros behind the end
        assert (got[k][0] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("absent", [("z",), ("D",), ("dt_bias",), ("h0", "dh_last"), ("z", "D", "dt_bias", "h0", "dh_last")], ids=str)
def test_optional_arguments(absent, softplus, layout):
    d = make(2, 150, 24, 6, layout, torch.float32, seed=8, softplus=softplus, absent=absent)
    check(run(d, layout), reference(d, layout), layout, torch.float32, absent)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_a_state_that_is_not_finite_stays_in_its_channel(layout):
    """An infinite state at the last position reaches what reads it, and nothing past the length or beside it."""
    d = make(2, 40, 33, 5, layout, torch.float32, seed=2, lengths=[20, 40])
    clean = run(d, layout)
    x = d["x"][0].T if layout == "planes" else d["x"][0]
    x[19, 3] = float("inf")
    got = run(d, layout)
    y, clean_y = (v["y"].transpose(1, 2) if layout == "planes" else v["y"] for v in (got, clean))
    assert not torch.isfinite(y[0, 19, 3]) and (y[0, 20:] == 0).all()
    y[0, 19, 3] = clean_y[0, 19, 3]
    assert torch.equal(y, clean_y)
    others = [c for c in range(33) if c != 3]
    assert torch.isfinite(got["dA"][others]).all() and torch.equal(got["d_h0"][1], clean["d_h0"][1])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_steps_of_zero_leave_the_state(layout):
    d = make(2, 300, 33, 7, layout, torch.float32, seed=2, softplus=False, absent=("dt_bias",))
    d["dt"].zero_()
    got = run(d, layout)
    assert torch.equal(got["h_last"], d["h0"]) and (got["dx"] != 0).any() and (got["dB"] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_an_infinite_input_reaches_no_gradient_before_its_two_positions(layout):
    d = make(2, 40, 33, 5, layout, torch.bfloat16, seed=2)
    clean = run(d, layout)
    (d["x"][0].T if layout == "planes" else d["x"][0])[20, 3] = float("inf")
    got = run(d, layout)
    for k in ("dB", "dC"):
        a, b = (time_first(v[k], layout) for v in (got, clean))
        assert np.array_equal(a[:20], b[:20]) and np.array_equal(a[:, 1], b[:, 1])
    assert not np.isfinite(time_first(got["dC"], layout)[20, 0]).all()


def embed(t, before, after, pad, rows_at):
    """t's values in a larger NaN-filled buffer: padded rows, an odd start, other elements around.  rows_at: the axes
    from there on lie in one row."""
    inner = int(np.prod(t.shape[rows_at:]))
    outer = t.shape[1:rows_at]
    row = inner + pad
    count = int(np.prod(outer)) if outer else 1
    buf = torch.full((before + t.shape[0] * count * row + after,), float("nan"), dtype=t.dtype, device=t.device)
    strides = [1] * t.dim()
    for i in range(t.dim() - 2, rows_at - 1, -1):
        strides[i] = strides[i + 1] * t.shape[i + 1]
    step = row
    for i in range(rows_at - 1, -1, -1):
        strides[i] = step
        step *= t.shape[i]
    view = buf.as_strided(t.shape, strides, before)
    view.copy_(t)
    return buf, view


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("before,pad", [(0, 8), (1, 0), (3, 5)])
def test_strides_and_alignment(before, pad, dtype, layout):
    """Padded rows and odd starts, other ones for every tensor; nothing outside an output is written."""
    B, T, C, N, G = 3, 70, 40, 6, 2
    d = make(B, T, C, N, layout, dtype, G=G, seed=9)
    want = reference(d, layout)
    rows_at = {k: (2 if layout == "tokens" else d[k].dim() - 1) for k in ACTIVATIONS}
    outs, bufs = {}, {}
    for k, like in (("y", "x"), ("dx", "x"), ("d_dt", "x"), ("dz", "x"), ("dB", "B"), ("dC", "B")):
        bufs[k], outs[k] = embed(torch.zeros_like(d[like].contiguous()), before, 7, pad, rows_at[like])
        bufs[k].fill_(-77.0)
    for i, k in enumerate(ACTIVATIONS):
        _, d[k] = embed(d[k], before + i * (before % 2), 4, pad, rows_at[k])
    check(run(d, layout, **outs), want, layout, dtype)
    for k in outs:
        inside = torch.zeros_like(bufs[k], dtype=torch.bool)
        inside.as_strided(outs[k].shape, outs[k].stride(), outs[k].storage_offset()).fill_(True)
        assert (bufs[k][~inside] == -77.0).all(), f"{k}: written outside its elements"


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
def test_views_of_other_orders(dtype):
    """Halves of one projection; a time-first batch; one B for every sequence."""
    B, T, C, N = 4, 50, 64, 16
    d = make(B, T, C, N, "tokens", dtype, seed=10)
    want = reference(d, "tokens")
    xz, bc = torch.cat([d["x"], d["z"]], 2), torch.cat([d["B"], d["C"]], 2)
    check(run({**d, "x": xz[:, :, :C], "z": xz[:, :, C:], "B": bc[:, :, :1], "C": bc[:, :, 1:]}, "tokens"), want, "tokens", dtype)
    turned = {**d, **{k: d[k].transpose(0, 1).contiguous().transpose(0, 1) for k in ACTIVATIONS}}
    check(run(turned, "tokens"), want, "tokens", dtype)
    shared = {**d, "B": d["B"][:1].expand(B, T, 1, N)}
    got = run({**shared}, "tokens", dB=torch.empty_like(d["B"]))
    check(got, reference(shared, "tokens"), "tokens", dtype)


@pytest.mark.gpu
def test_image_planes_equal_flat_planes():
    B, C, N, side = 2, 20, 8, 12
    d = make(B, side * side, C, N, "planes", torch.bfloat16, seed=3)
    flat = run(d, "planes")
    image = {**d, **{k: d[k].unflatten(-1, (side, side)) for k in ACTIVATIONS}}
    got = run(image, "planes")
    for k, v in flat.items():
        assert torch.equal(got[k].reshape(v.shape), v), k
    assert got["dx"].shape == image["x"].shape and got["dB"].shape == image["B"].shape


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_results_repeat(layout):
    d = make(2, 700, 70, 16, layout, torch.bfloat16, seed=4)
    a, b = run(d, layout), run(d, layout)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_pieces_compose(layout):
    """A sequence in two calls, the first's last state the second's beginning, and the gradients back through both."""
    d = make(2, 90, 12, 5, layout, torch.float32, seed=6)
    want = reference(d, layout)
    axis = 1 if layout == "tokens" else -1
    cut = lambda t, a, b: t.narrow(axis, a, b - a)  # noqa: E731
    parts = [{**d, **{k: cut(d[k], a, b) for k in ACTIVATIONS}} for a, b in ((0, 41), (41, 90))]
    names, more = ("x", "dt", "A", "B", "C"), ("D", "z", "dt_bias")
    kw = [{k: p[k] for k in more} for p in parts]
    y0, h0, s0 = M.wtconv_selective_forward(*[parts[0][k] for k in names], h0=d["h0"], layout=layout, keep_states=True, **kw[0])
    y1, h1, s1 = M.wtconv_selective_forward(*[parts[1][k] for k in names], h0=h0, layout=layout, keep_states=True, **kw[1])
    g1 = M.wtconv_selective_backward(*[parts[1][k] for k in names], s1, parts[1]["dy"], dh_last=d["dh_last"], layout=layout, **kw[1])
    g0 = M.wtconv_selective_backward(*[parts[0][k] for k in names], s0, parts[0]["dy"], dh_last=g1[-1], layout=layout, **kw[0])
    got = {"y": torch.cat([y0, y1], axis), "h_last": h1, "d_h0": g0[-1]}
    for k, i in (("dx", 0), ("d_dt", 1), ("dB", 3), ("dC", 4), ("dz", 6)):
        got[k] = torch.cat([g0[i], g1[i]], axis)
    for k, i in (("dA", 2), ("dD", 5), ("d_dt_bias", 7)):
        got[k] = g0[i] + g1[i]
    check(got, want, layout, torch.float32)


# ------------------------------------------------------------------------------------ one token

@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("B,C,N,G", [(1, 1, 1, 1), (3, 70, 16, 2), (5, 33, 13, 3), (2, 128, 64, 1), (9, 50, 8, 1), (4, 20, 30, 1)])
def test_steps_equal_the_scan(B, C, N, G, dtype):
    """Several steps on a pool; the other rows stay."""
    T = 6
    d = make(B, T, C, N, "tokens", dtype, G=G, seed=7)
    want = reference(d, "tokens")
    pool = torch.full((2 * B + 1, C, N), 5.0, device="cuda")
    slots = torch.arange(2 * B - 1, -1, -2, dtype=torch.int32, device="cuda")
    pool[slots.long()] = d["h0"]
    ys = [M.wtconv_selective_step(d["x"][:, t], d["dt"][:, t], d["A"], d["B"][:, t], d["C"][:, t], pool, d["D"], d["z"][:, t],
                                  d["dt_bias"], slots) for t in range(T)]
    R.assert_within("y", torch.stack(ys), *want["y"], dtype)
    R.assert_within("pool", pool[slots.long()], *want["h_last"])
    rest = [i for i in range(2 * B + 1) if i not in slots.tolist()]
    assert (pool[rest] == 5.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("N", [16, 5])
def test_step_without_options_and_with_idle_sequences(N):
    B, C = 5, 12
    d = make(B, 1, C, N, "tokens", torch.float32, seed=1, softplus=False, absent=("D", "z", "dt_bias"))
    args = [d["x"][:, 0], d["dt"][:, 0], d["A"], d["B"][:, 0], d["C"][:, 0]]
    want = reference(d, "tokens")
    pool = d["h0"].clone()
    y = M.wtconv_selective_step(*args, pool, softplus=False)
    R.assert_within("y", y[None], *want["y"])
    R.assert_within("pool", pool, *want["h_last"])
    pool2, slots = d["h0"].clone(), torch.tensor([0, -1, 2, B, 4], dtype=torch.int32, device="cuda")
    buf, given = embed(torch.zeros(B, C, device="cuda"), 3, 2, 5, 1)
    buf.fill_(-77.0)
    y2 = M.wtconv_selective_step(*args, pool2, slots=slots, softplus=False, y=given)
    busy, idle = [0, 2, 4], [1, 3]
    assert torch.equal(y2[busy], y[busy]) and (y2[idle] == 0).all()
    assert torch.equal(pool2[busy], pool[busy]) and torch.equal(pool2[idle], d["h0"][idle])
    assert int((buf == -77.0).sum()) == buf.numel() - B * C


# ----------------------------------------------------------------------------------- autograd

@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_autograd(layout):
    d = make(2, 60, 20, 6, layout, torch.float32, G=2, seed=11, lengths=[60, 33])
    for k in ACTIVATIONS:
        d[k] = torch.nan_to_num(d[k])
    names = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0")
    leaves = {k: d[k].clone().requires_grad_() for k in names}
    y, h_last = M.selective_scan(**leaves, lengths=d["lengths"], layout=layout)
    torch.autograd.backward([y, h_last], [d["dy"], d["dh_last"]])
    got = run(d, layout)
    for k, g in (("x", "dx"), ("dt", "d_dt"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"), ("dt_bias", "d_dt_bias"),
                 ("h0", "d_h0")):
        assert torch.equal(leaves[k].grad, got[g]), k
    # only one of the outputs, a broadcast gradient, inputs without gradients
    y, _ = M.selective_scan(leaves["x"], *[d[k] for k in names[1:]], lengths=d["lengths"], layout=layout)
    leaves["x"].grad = None
    y.sum().backward()
    ones = {**d, "dy": torch.ones_like(d["dy"]), "dh_last": None}
    assert torch.equal(leaves["x"].grad, run(ones, layout)["dx"])
    _, h = M.selective_scan(**leaves, lengths=d["lengths"], layout=layout)
    h.sum().backward()


@pytest.mark.gpu
def test_second_derivatives_are_refused():
    d = make(1, 8, 4, 3, "tokens", torch.float32)
    x = d["x"].clone().requires_grad_()
    y, _ = M.selective_scan(x, d["dt"], d["A"], d["B"], d["C"], layout="tokens")
    (g,) = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.sum().backward()


# ------------------------------------------------------------------- streams, graphs, workspaces

@pytest.mark.gpu
def test_stream_and_workspace():
    d = make(2, 500, 40, 16, "tokens", torch.bfloat16, seed=12)
    want = run(d, "tokens")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = run(d, "tokens", stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(got[k], want[k]) for k in want)
    size = M._load().wtconv_selective_workspace_size(S.OP_SCAN_BACKWARD, ctypes.byref(M.SelectiveShape(2, 500, 40, 16, 1, 1, 1, 1)))
    for n, fine in ((size, True), (size - 16, False)):
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        if fine:
            assert torch.equal(_backward(d, ws)[0], want["dx"])
        else:
            with pytest.raises(W.WTConvError):
                _backward(d, ws)


def _backward(d, workspace):
    inputs = [d[k] for k in ("x", "dt", "A", "B", "C")]
    more = {**{k: d[k] for k in ("D", "z", "dt_bias")}, "layout": "tokens"}
    _, _, states = M.wtconv_selective_forward(*inputs, h0=d["h0"], keep_states=True, **more)
    return M.wtconv_selective_backward(*inputs, states, d["dy"], dh_last=d["dh_last"], workspace=workspace, **more)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_graph(layout):
    """Forward and backward captured, replayed on other inputs."""
    d, other = (make(2, 300, 40, 16, layout, torch.bfloat16, seed=s) for s in (13, 14))
    run(d, layout)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(d, layout)
    want = run(other, layout)
    for k in ACTIVATIONS + ("A", "D", "dt_bias", "h0", "dh_last"):
        d[k].copy_(other[k])
    graph.replay()
    assert all(torch.equal(got[k], want[k]) for k in want)
