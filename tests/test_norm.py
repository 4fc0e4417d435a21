"""The root-mean-square norm (include/wtconv_norm.h) against its definition in fp64, and its refusals.

Bounds, with u = 2^-24 (half a unit of fp32): the sum of C squares adds at most 32 in a row in a thread, 5 levels in
a warp and 16 warps: 54 u; the root 4u; half of that and the products: y is off by at most 40 u |y| beside its rounding.
The backward's mean is off by 60 u of the mean of absolute values; dw sums rows one after the other in a CTA."""
import ctypes

import numpy as np
import pytest
import torch
from ssm_reference import U, assert_within

from memory_bound_cnn_gb300 import norm as M
from memory_bound_cnn_gb300 import wtconv as W

TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32)]
ids = lambda t: "-".join(str(v)[6:] for v in t) if isinstance(t, tuple) else str(t)  # noqa: E731
EPS = 1e-5


def make(rows, C, dtype, total_dtype, seed=0, residual=True):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    d = {"x": normal(rows, C).to(dtype), "weight": 1 + 0.3 * normal(C), "residual": None, "dy": normal(rows, C).to(dtype), "d_total": None}
    if residual:
        d["residual"], d["d_total"] = (3 * normal(rows, C)).to(total_dtype), normal(rows, C).to(total_dtype)
    return d


def total_of(d):
    return d["x"] if d["residual"] is None else (d["x"].float() + d["residual"].float()).to(d["residual"].dtype)


def reference(d, eps=EPS):
    t = total_of(d).double().cpu().numpy().reshape(-1, d["x"].shape[-1])
    w, dy = (d[k].double().cpu().numpy().reshape(-1, t.shape[1]) for k in ("weight", "dy"))
    rstd = 1 / np.sqrt((t * t).mean(1, keepdims=True) + eps)
    n = t * rstd
    y = n * w
    g = dy * w
    mean, mean_abs = (g * n).mean(1, keepdims=True), np.abs(g * n).mean(1, keepdims=True)
    d_t = rstd * (g - n * mean)
    err = rstd * (np.abs(g) * 45 * U + np.abs(n) * mean_abs * 150 * U)
    if d["d_total"] is not None:
        d_t = d_t + d["d_total"].double().cpu().numpy().reshape(t.shape)
        err = err + U * np.abs(d_t)
    terms = (len(t) + 80) * U
    return {"y": (y, 40 * U * np.abs(y)), "rstd": (rstd[:, 0], 32 * U * rstd[:, 0]), "dx": (d_t, err),
            "dw": ((dy * n).sum(0), (np.abs(dy * n) * terms).sum(0))}


def run(d, stream=None, **out):
    y, total, rstd = M.wtconv_rms_forward(d["x"], d["weight"], d["residual"], EPS, stream=stream, **out)
    dx, dr, dw = M.wtconv_rms_backward(d["dy"], total, d["weight"], rstd, d["d_total"], d["residual"] is not None, stream=stream)
    return {"y": y, "total": total, "rstd": rstd, "dx": dx, "d_residual": dr, "dw": dw}


def check(got, d, want):
    C = d["x"].shape[-1]
    assert torch.equal(got["total"], total_of(d))
    for k, dtype in (("y", d["x"].dtype), ("dx", d["x"].dtype)):
        assert_within(k, got[k].reshape(-1, C), *want[k], dtype)
    assert_within("rstd", got["rstd"].reshape(-1), *want["rstd"])
    assert_within("dw", got["dw"], *want["dw"])
    if d["residual"] is None:
        assert got["d_residual"] is None
    else:
        assert_within("d_residual", got["d_residual"].reshape(-1, C), *want["dx"], d["residual"].dtype)


# ---------------------------------------------------------------------------- the definition, refusals (CPU)

def test_reference_gradients_match_differences():
    rng = np.random.default_rng(2)
    d = {"x": torch.tensor(rng.standard_normal((3, 5))), "weight": torch.tensor(rng.standard_normal(5)), "residual": None,
         "dy": torch.tensor(rng.standard_normal((3, 5))), "d_total": torch.tensor(rng.standard_normal((3, 5)))}
    g = reference(d)
    for name, grad in (("x", "dx"), ("weight", "dw")):
        for i in np.ndindex(*d[name].shape):
            values = []
            for step in (1e-5, -1e-5):
                e = {**d, name: d[name].clone()}
                e[name][i] += step
                values.append(float((torch.tensor(reference(e)["y"][0]) * d["dy"]).sum() + (e["x"] * d["d_total"]).sum()))
            assert abs((values[0] - values[1]) / 2e-5 - g[grad][0][i]) < 1e-8, (name, i)


FAKE, ODD = 256, 258


def row(p=FAKE, stride=8):
    return M.RmsTensor(p, stride)


def shape(rows=4, C=8, dtype=0, total=0, eps=1e-6):
    return M.RmsShape(rows, C, dtype, total, eps)


def _forward(s=None, x=row(), residual=row(), w=FAKE, y=row(), total=row(), rstd=None):
    ref = ctypes.byref
    return M._load().wtconv_rms_forward(ref(s or shape()), ref(x), ref(residual), w, ref(y), ref(total), rstd, None)


def _e4m3(s=None, x=row(), residual=row(), w=FAKE, block=0, q=FAKE, scales=FAKE, total=row()):
    ref = ctypes.byref
    return M._load().wtconv_rms_forward_e4m3(ref(s or shape()), ref(x), ref(residual), w, block, q, scales, ref(total), None)


def _backward(s=None, dy=row(), total=row(), w=FAKE, rstd=FAKE, d_total=row(), dx=row(), dr=row(), dw=FAKE, ws=FAKE, nbytes=1 << 30):
    ref = ctypes.byref
    return M._load().wtconv_rms_backward(ref(s or shape()), ref(dy), ref(total), w, rstd, ref(d_total), ref(dx), ref(dr), dw, ws, nbytes,
                                         None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=0), W.ERR_INVALID_ARG), (dict(C=0), W.ERR_INVALID_ARG), (dict(C=16385), W.ERR_INVALID_ARG),
    (dict(rows=(1 << 30) + 1), W.ERR_INVALID_ARG), (dict(eps=-1.0), W.ERR_INVALID_ARG), (dict(eps=float("nan")), W.ERR_INVALID_ARG),
    (dict(eps=float("inf")), W.ERR_INVALID_ARG), (dict(dtype=3), W.ERR_UNSUPPORTED), (dict(dtype=1, total=2), W.ERR_UNSUPPORTED),
    (dict(dtype=0, total=1), W.ERR_UNSUPPORTED)])
def test_shapes_are_refused(kw, status):
    s = shape(**kw)
    assert _forward(s) == _e4m3(s) == _backward(s) == status
    assert M._load().wtconv_rms_workspace_size(ctypes.byref(s)) == 0


def test_calls_refuse(monkeypatch):
    bad, none = W.ERR_INVALID_ARG, row(None)
    for kw in (dict(x=none), dict(x=row(ODD)), dict(x=row(FAKE, -8)), dict(w=None), dict(w=ODD), dict(y=none), dict(y=row(FAKE, 7)),
               dict(total=none), dict(total=row(FAKE, 7)), dict(residual=row(ODD)), dict(rstd=ODD),
               dict(s=shape(dtype=1, total=0), residual=none)):
        assert _forward(**kw) == bad, kw
    for kw in (dict(q=None), dict(scales=None), dict(scales=ODD), dict(total=none), dict(x=none)):
        assert _e4m3(**kw) == bad, kw
    assert _e4m3(block=64) == W.ERR_UNSUPPORTED
    for kw in (dict(dy=none), dict(total=none), dict(w=None), dict(rstd=None), dict(d_total=row(ODD)), dict(dx=row(FAKE, 7)),
               dict(dr=row(FAKE, 7)), dict(dx=none, dr=none), dict(dw=ODD), dict(ws=ODD)):
        assert _backward(**kw) == bad, kw
    assert _backward(ws=None) == _backward(nbytes=1) == W.ERR_WORKSPACE
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        M.wtconv_rms_forward(x, torch.zeros(8))
    monkeypatch.setenv("WTCONV_INJECT_FAULT", "1")
    assert _forward() == _e4m3() == _backward() == _backward(dw=None, ws=None) == W.ERR_INJECTED


# ------------------------------------------------------------------------------------ the kernels

SIZES = [(1, 1), (3, 7), (5, 32), (2, 255), (9, 256), (4, 257), (6, 512), (3, 513), (7, 768), (2, 1024), (3, 1025), (2, 2048), (3, 2056),
         (2, 4096), (1, 4100), (2, 8192), (3, 8200), (2, 16384), (1, 16383), (3000, 40), (2500, 776)]


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, types):
    d = make(*size, *types, seed=size[1])
    check(run(d), d, reference(d))
    d = make(*size, *types, seed=size[1], residual=False)
    check(run(d), d, reference(d))


@pytest.mark.gpu
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_e4m3(size, types, block):
    """Each value is off by half a step of e4m3 at most: 2^-4 of itself, 2^-10 of the scale where codes are
    subnormal; the fp32 before it adds 44 u to either side."""
    d = make(*size, *types, seed=size[1])
    d["x"][0] = 0
    d["residual"][0] = 0
    q, scales, total = M.wtconv_rms_forward_e4m3(d["x"], d["weight"], d["residual"], EPS, block)
    assert torch.equal(total, total_of(d)) and q.dtype == torch.float8_e4m3fn
    y = reference(d)["y"][0]
    rows, C = y.shape
    per = block or C
    blocks = -(-C // per)
    most = np.abs(np.pad(y, ((0, 0), (0, blocks * per - C)))).reshape(rows, blocks, per).max(2)
    got_scales = scales.double().cpu().numpy()
    assert got_scales.shape == (rows, blocks)
    assert (np.abs(got_scales - most / 448) <= 44 * U * most / 448).all()
    wide = np.repeat(got_scales, per, 1)[:, :C]
    got = q.to(torch.float32).double().cpu().numpy() * wide
    assert (np.abs(got - y) <= np.abs(y) * (2.0 ** -4 + 100 * U) + wide * 2.0 ** -10).all()
    assert (got[0] == 0).all() and (got_scales[0] == 0).all()
    # the largest of a block is the largest code
    top = np.abs(np.pad(q.to(torch.float32).cpu().numpy(), ((0, 0), (0, blocks * per - C)))).reshape(rows, blocks, per).max(2)
    assert (top[1:] == 448).all()


@pytest.mark.gpu
@pytest.mark.parametrize("block", [0, 128])
@pytest.mark.parametrize("C", [96, 768, 1000, 5000])
@pytest.mark.parametrize("x_power,w_power,eps", [(-100, -20, 2.0 ** -20), (-60, -68, 0.0), (55, 80, 2.0 ** -20), (-60, 30, 0.0), (3, -112, 2.0 ** -20)], ids=str)
def test_e4m3_of_small_and_large_values(C, block, x_power, w_power, eps):
    """Rows and weights of any size have y of theirs: codes do not change with a power of two that all of a row share.
    Where all values are below 2^-110, scales and codes are 0."""
    d = make(4, C, torch.float32, torch.float32, seed=6, residual=False)
    x, w = d["x"] * 2.0 ** x_power, d["weight"] * 2.0 ** w_power
    q, scales, _ = M.wtconv_rms_forward_e4m3(x, w, None, eps, block)
    t, w = x.double().cpu().numpy(), w.double().cpu().numpy()
    y = t / np.sqrt((t * t).mean(1, keepdims=True) + eps) * w
    per = block or C
    most = np.abs(np.pad(y, ((0, 0), (0, -C % per)))).reshape(4, -1, per).max(2)
    got = scales.double().cpu().numpy()
    small = most < 2.0 ** -110
    assert (got[small] == 0).all() and (np.abs(got - most / 448) <= 44 * U * most / 448)[~small].all()
    plain = M.wtconv_rms_forward_e4m3(d["x"], d["weight"], None, 0.0, block)[0].float()
    keep = torch.from_numpy(np.repeat(~small, per, 1)[:, :C].copy()).cuda()
    assert torch.equal(q.float(), torch.where(keep, plain, torch.zeros_like(plain)))


@pytest.mark.gpu
@pytest.mark.parametrize("C", [96, 768, 1000, 5000])
def test_values_that_are_not_finite_stay_in_their_row(C):
    d = make(6, C, torch.float32, torch.float32, seed=3)
    clean = run(d)
    d["x"][1, 3], d["x"][2, C - 1], d["residual"][4, 0] = float("nan"), float("inf"), -float("inf")
    got, fine = run(d), [0, 3, 5]
    for k in ("y", "total", "rstd", "dx"):
        assert torch.equal(got[k][fine], clean[k][fine]), k
    assert torch.isnan(got["y"][1]).all() and torch.isnan(got["y"][2, C - 1])
    for block in (0, 128):
        q, scales, _ = M.wtconv_rms_forward_e4m3(d["x"], d["weight"], d["residual"], EPS, block)
        assert torch.isfinite(scales[fine]).all() and torch.isnan(scales[[1], [0]]).all()
        assert torch.isnan(scales[2]).any() and torch.isnan(scales[4, 0])
        assert torch.isnan(q.float()[1, :3]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES, ids=ids)
@pytest.mark.parametrize("before,pad", [(0, 8), (1, 0), (3, 5)])
def test_strides_and_alignment(before, pad, types):
    from test_selective import embed
    rows, C = 5, 264
    d = make(rows, C, *types, seed=4)
    want = reference(d)
    bufs = {}
    out = {}
    for k, dtype in (("y", types[0]), ("total", types[1])):
        bufs[k], out[k] = embed(torch.zeros(rows, C, dtype=dtype, device="cuda"), before, 7, pad, 1)
        bufs[k].fill_(-77.0)
    for i, k in enumerate(("x", "residual", "dy", "d_total")):
        _, d[k] = embed(d[k], before + i * (before % 2), 4, pad, 1)
    check(run(d, **out), d, want)
    for k in out:
        assert int((bufs[k] == -77.0).sum()) == bufs[k].numel() - rows * C, k
    # a weight at an odd address
    d["weight"] = torch.cat([d["weight"][:1], d["weight"]])[1:]
    check(run(d), d, want)


@pytest.mark.gpu
def test_shapes_of_rows():
    """Leading axes, halves of a projection, one row, a row for every position; what has no one distance is refused."""
    d = make(24, 64, torch.bfloat16, torch.float32, seed=5)
    flat = run(d)
    deep = {k: v if k == "weight" else v.view(2, 3, 4, 64) for k, v in d.items()}
    got = run(deep)
    assert got["rstd"].shape == (2, 3, 4) and all(torch.equal(got[k].reshape(flat[k].shape), flat[k]) for k in flat)
    both = torch.cat([d["x"], d["dy"]], 1).view(2, 12, 128)
    halves = {**d, "x": both[..., :64], "dy": both[..., 64:], "residual": d["residual"].view(2, 12, 64), "d_total": d["d_total"].view(2, 12, 64)}
    got = run(halves)
    assert all(torch.equal(got[k].reshape(flat[k].shape), flat[k]) for k in flat)
    one = {k: v if k == "weight" else v[0] for k, v in d.items()}
    assert run(one)["rstd"].shape == ()
    q, scales, _ = M.wtconv_rms_forward_e4m3(one["x"], d["weight"], one["residual"], EPS, 128)
    assert q.shape == (64,) and scales.shape == (1,)
    repeated = d["x"][:1].expand(24, 64)
    assert torch.equal(M.wtconv_rms_forward(repeated, d["weight"])[0], M.wtconv_rms_forward(repeated.contiguous(), d["weight"])[0])
    with pytest.raises(ValueError, match="one distance"):
        M.wtconv_rms_forward(d["x"].view(4, 6, 64).transpose(0, 1), d["weight"])
    with pytest.raises(ValueError, match="innermost"):
        M.wtconv_rms_forward(d["x"].t(), torch.ones(24, device="cuda"))
    with pytest.raises(ValueError, match="residual"):
        M.wtconv_rms_forward(d["x"], d["weight"], d["x"].half())
    with pytest.raises(ValueError, match="block"):
        M.wtconv_rms_forward_e4m3(d["x"], d["weight"], block=32)


@pytest.mark.gpu
@pytest.mark.parametrize("types", TYPES, ids=ids)
def test_autograd_stream_and_graph(types):
    d = make(40, 136, *types, seed=6)
    want = run(d)
    leaves = {k: d[k].clone().requires_grad_() for k in ("x", "weight", "residual")}
    y, total = M.rms_norm(**leaves, eps=EPS)
    torch.autograd.backward([y, total], [d["dy"], d["d_total"]])
    for k, g in (("x", "dx"), ("weight", "dw"), ("residual", "d_residual")):
        assert torch.equal(leaves[k].grad, want[g]), k
    y = M.rms_norm(leaves["x"], leaves["weight"], eps=EPS)
    (g,) = torch.autograd.grad(y.float().sum(), leaves["x"], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        g.float().sum().backward()
    _, total = M.rms_norm(**leaves, eps=EPS)
    leaves["residual"].grad = None
    total.float().sum().backward()
    assert (leaves["residual"].grad == 1).all()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = run(d, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert all(torch.equal(got[k], want[k]) for k in want)
    other = make(40, 136, *types, seed=7)
    want = run(other)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(d)
    for k in d:
        d[k].copy_(other[k])
    graph.replay()
    assert all(torch.equal(got[k], want[k]) for k in want)
