"""Corners of the selective scan and the causal convolution: sums over channels that cancel, parts of a sequence whose
decays leave the range of fp32, inputs that are not finite, calls without gradients."""
import ctypes

import numpy as np
import pytest
import ssm_reference as R
import test_causal
import torch
from test_selective import DTYPES, LAYOUTS, make, reference, run, time_first

from memory_bound_cnn_gb300 import scan as S
from memory_bound_cnn_gb300 import ssm as M


# ------------------------------------------------------------------------ sums over channels

@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("N", [5, 16, 32, 64])
def test_sums_over_channels_that_cancel(N, dtype, layout):
    """Channels in pairs whose products differ in sign and, by about 1/64, in size: dB and dC are as exact as sums in fp32
    of the products, and rounded once.  (The other tests' bounds for bf16 would allow products of 11 bits.)"""
    d = make(2, 50, 64, N, layout, dtype, seed=N)
    for k, factor in (("x", 1 + 1 / 64), ("dt", 1), ("z", 1), ("dy", -1)):
        channels = d[k] if layout == "tokens" else d[k].transpose(1, 2)
        channels[:, :, 1::2] = (channels[:, :, 0::2].float() * factor).to(dtype)
    for k in ("A", "dt_bias"):
        d[k][1::2] = d[k][0::2]
    d["h0"][:, 1::2], d["dh_last"][:, 1::2] = d["h0"][:, 0::2].clone(), -d["dh_last"][:, 0::2]
    got, want = run(d, layout), reference(d, layout)
    for k in ("dB", "dC"):
        R.assert_within(k, got[k].movedim(1 if layout == "tokens" else -1, 0), *want[k], dtype)


# ------------------------------------------------------------------------- parts of a sequence

def parted(dt, A, **of_positions):
    """A sequence of 256 positions of few channels, cut into parts, whose steps are dt (256,)."""
    T, C, N = 256, 6, 4
    size = M._load().wtconv_selective_workspace_size(S.OP_SCAN_FORWARD, ctypes.byref(M.SelectiveShape(1, T, C, N, 1, 1, 0, 0)))
    assert size > 0  # (in one part the forward needs no workspace)
    d = make(1, T, C, N, "tokens", torch.float32, seed=3, softplus=False, absent=("dt_bias",))
    d["dt"].copy_(dt[None, :, None].expand(1, T, C))
    d["A"] = torch.tensor(A, device="cuda").repeat(C, 1)
    for k, keep in of_positions.items():  # 0 at other positions
        d[k] *= keep[None, :, None]
    return d


def check_parted(d, layout):
    """All results against the definition, which knows no parts, in tokens and as planes; not those that fp32 cannot hold."""
    if layout == "planes":
        d = {**d, **{k: d[k].movedim(1, -1).contiguous() for k in ("x", "dt", "z", "dy", "B", "C")}}
    got, want = run(d, layout), reference(d, layout)
    for k, t in got.items():
        if t is not None and np.abs(want[k][0]).max() < torch.finfo(torch.float32).max:
            inner = k in ("y", "dx", "d_dt", "dB", "dC", "dz")
            R.assert_within(k, t.movedim(1 if layout == "tokens" else -1, 0) if inner else t, *want[k])
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
def test_growth_over_parts_that_hold_nothing(layout):
    """States grow by exp(128) in a part of 64 positions, but are 0 up to the last 8; so are the gradients behind the
    first 8."""
    at = torch.arange(256, device="cuda")
    d = parted(torch.full((256,), 2.0, device="cuda"), [1.0, 0.5, -1.0, 2.0], x=at >= 248, dy=at < 8)
    d["h0"] = d["dh_last"] = None
    got = check_parted(d, layout)
    assert (got["h_last"] != 0).all() and (got["dx"].movedim(1 if layout == "tokens" else -1, 0)[:8] != 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rate,size", [(1.0, 1e-30), (-1.0, 1e30)])
def test_a_part_whose_factor_leaves_the_range(rate, size, layout):
    """Over 48 positions of the second part the states change by exp(96) or exp(-96), which is no normal fp32 number; what
    they make of a state of 1e-30 or 1e30 is.  (Of 1e30, d_dt and dA are not: a state times its gradient times exp(-24), 4e49.)"""
    at = torch.arange(256, device="cuda")
    zone = (at >= 64) & (at < 112)
    d = parted(2.0 * zone, [rate, 0.5 * rate, 0.25 * rate, rate], x=~zone, dy=at < 64)
    d["h0"], d["dh_last"] = d["h0"] * size, d["dh_last"] * size
    check_parted(d, layout)


# --------------------------------------------------------------------- what is not finite

@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_an_infinite_last_input_reaches_the_last_tap_alone(K, dtype, layout):
    """The input at a sequence's last position meets the last tap only; positions past the length sum nothing."""
    T, C, lengths = 16, 5, [5, 16, 10, 7]
    d = test_causal.make(4, T, C, K, layout, dtype, seed=K, lengths=lengths, silu=False)
    x = d["x"] if layout == "tokens" else d["x"].transpose(1, 2)
    for b, n in enumerate(lengths):
        x[b, n - 1] = 0
    want = test_causal.reference(d, layout)  # (of the other taps: their sums do not have that input)
    for b, n in enumerate(lengths):
        x[b, n - 1] = float("inf")
    got = test_causal.run(d, layout)
    R.assert_within("dw", got["dw"][:, :-1], want["dw"][0][:, :-1], want["dw"][1][:, :-1])
    R.assert_within("d_bias", got["d_bias"], *want["d_bias"])
    assert not torch.isfinite(got["dw"][:, -1]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T", [40, 256])  # in one part, and in several
@pytest.mark.parametrize("N", [1, 5, 16])
def test_an_infinite_step_lets_nothing_flow_back(N, T, layout):
    """exp(d A) is 0 where d is infinite and A negative: before it the gradients are those of a sequence that ends there,
    for any number of states."""
    d = make(1, T, 6, N, layout, torch.float32, seed=4)
    ended = {**d, "lengths": torch.tensor([20], dtype=torch.int32, device="cuda"), "dh_last": None}
    want = reference(ended, layout)
    d["dt"] = d["dt"].clone()
    (d["dt"][0] if layout == "tokens" else d["dt"][0].T)[20] = float("inf")
    got = run(d, layout)
    for k in ("dx", "d_dt"):
        t = got[k].movedim(1 if layout == "tokens" else -1, 0)
        R.assert_within(k, t[:20], want[k][0][:20], want[k][1][:20])


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("N", [5, 16, 40])
@pytest.mark.parametrize("what,at", [("x", 21), ("C", 21), ("dh_last", 0), ("h0", 0)])
def test_what_is_not_finite_stays_where_the_formulas_have_it(what, at, N, layout):
    """Of one infinite input; dB and dC may be NaN for its four states and two positions, wherever either of them is not
    finite."""
    d = make(2, 50, 34, N, layout, torch.float32, G=2, seed=N)
    if what in ("h0", "dh_last"):
        d[what][1, 20, 3] = float("inf")
    else:
        row = d[what][1] if layout == "tokens" else d[what][1].movedim(-1, 0)
        row[at][(3,) if what == "x" else (0, 3)] = float("inf")
    got = run(d, layout)
    ref = {"softplus": True, "lengths": None}
    for name, k in (("x", "x"), ("dt", "dt"), ("z", "z"), ("dy", "dy"), ("Bm", "B"), ("Cm", "C")):
        ref[name] = time_first(d[k], layout)
    for k in ("A", "D", "dt_bias", "h0", "dh_last"):
        ref[k] = d[k].double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = {k: np.isfinite(v[0]) for k, v in R.selective(ref).items() if k != "cut"}
    both = want["dB"] & want["dC"]
    near = np.ones((50, 2, 2, -(-N // 4) * 4), bool)
    near[:, :, :, :N] = both
    near = near.reshape(25, 2, 2, 2, -1, 4).all((1, 5), keepdims=True)
    near = np.broadcast_to(near, (25, 2, 2, 2, near.shape[4], 4)).reshape(50, 2, 2, -1)[..., :N]
    for k, fine in want.items():
        inner = k in ("y", "dx", "d_dt", "dB", "dC", "dz")
        finite = np.isfinite(time_first(got[k], layout) if inner else got[k].cpu().numpy())
        assert not (finite & ~fine).any(), k
        assert finite[near if k in ("dB", "dC") else fine].all(), k


# ------------------------------------------------------------------------ without gradients

@pytest.mark.parametrize("operator", ["selective", "gated"])
def test_states_are_kept_for_a_backward_only(operator, monkeypatch):
    """Under no_grad, and where no input needs a gradient, the forward is not asked for what the backward reads."""
    kept = []

    def forward(*args, keep_states=False, **kw):
        kept.append(keep_states)
        x = args[0]
        return x.clone(), x.new_zeros(2), (x.new_zeros(1) if keep_states else None)

    monkeypatch.setattr(M, "wtconv_selective_forward", forward)
    monkeypatch.setattr(S, "wtconv_scan_forward", forward)
    x, w = torch.zeros(1, 2, 3), torch.zeros(2, requires_grad=True)

    def call(w):
        return M.selective_scan(x, x, w, x, x) if operator == "selective" else S.gated_scan(x, x, w)

    with torch.no_grad():
        y, _ = call(w)
    assert kept == [False] and not y.requires_grad
    with torch.inference_mode():
        call(w)
    call(w.detach())
    y, _ = call(w)
    assert kept == [False, False, False, True] and y.requires_grad
