"""Corners of the gated scan: very long rows, far rows, masked garbage, streams, second derivatives."""
import numpy as np
import pytest
import scan_reference as R
import torch
from test_scan import DTYPES, check, make, reference, run

from memory_bound_cnn_gb300 import scan as S
from memory_bound_cnn_gb300 import wtconv as W


@pytest.mark.gpu
@pytest.mark.parametrize("extra", [4100, 4097])  # rows at multiples of 16 bytes, and not
def test_short_lengths_of_very_long_rows(extra):
    """Byte counts of a row that is more than 2^31 bytes longer than its sequence: NaN fills the row
    from position 5 on, and none of it reaches a result."""
    T, n = (1 << 29) + extra, 5
    g = torch.Generator().manual_seed(extra)
    head = torch.randn(n, generator=g)
    x = torch.full((1, 1, T), float("nan"), device="cuda")  # x, gate and dy alike: the inputs may overlap
    x[0, 0, :n] = head.cuda()
    bias, h0, dh = torch.ones(1, device="cuda"), torch.full((1, 1), 0.5, device="cuda"), torch.full((1, 1), 2.0, device="cuda")
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    y, h_last, states = S.wtconv_scan_forward(x, x, bias, h0, lengths, keep_states=True)
    dx, dg, db, dh0 = S.wtconv_scan_backward(x, x, bias, states, x, dh, lengths)
    v = head.double().numpy()[:, None, None]
    want_y, want_h, _ = R.forward(v, v, np.ones(1), np.full((1, 1), 0.5))
    want = R.backward(v, v, np.ones(1), v, np.full((1, 1), 0.5), np.full((1, 1), 2.0))
    for name, got, ref in (("y", y, want_y), ("dx", dx, want["dx"]), ("d_gate", dg, want["d_gate"])):
        R.assert_near(name, got[:, :, :n].double().cpu().numpy().transpose(2, 0, 1), ref)
        assert float(got[0, 0, n:].abs().max()) == 0, name
    R.assert_near("h_last", h_last.double().cpu().numpy(), want_h)
    R.assert_near("d_h0", dh0.double().cpu().numpy(), want["d_h0"])
    R.assert_near("d_gate_bias", db.double().cpu().numpy(), want["d_gate_bias"], scale=want["abs"].max())


@pytest.mark.gpu
def test_a_wait_that_gives_up_is_reported_once():
    """A bounded wait that nothing completes raises the flag; the host reads it once, and scans whose
    sequences are shared by clusters go on as before."""
    d = make(2, 1000, 512, "tokens", torch.bfloat16, seed=27)
    before = run(d, "tokens")
    assert S.wtconv_scan_status() == W.OK
    S.wtconv_scan_selftest_wait_timeout()
    assert S.wtconv_scan_status() == W.ERR_DEVICE_TIMEOUT
    assert S.wtconv_scan_status() == W.OK
    after = run(d, "tokens")
    for k in before:
        assert torch.equal(before[k], after[k]), k
    assert S.wtconv_scan_status() == W.OK


def dirty(sizes):
    """Blocks of these many bytes of the current stream's pool, filled with NaN or large bytes and let go."""
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xff)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("size", [(2, 5000, 8), (1, 40000, 16), (4, 300, 64)], ids=str)
def test_given_stream_without_workspace(size, layout):
    """The side stream is held up, so that the call's work runs after the current stream has used whatever
    memory it could get again: the call's scratch, and inputs that the caller has let go of.  Then the current
    stream is held up with writes to blocks that it has let go of, which a new output must not be put in."""
    B, T, C = size
    d = make(B, T, C, layout, torch.bfloat16, seed=28)
    want = run(d, layout)
    order = {"planes": 0, "tokens": 1}[layout]
    scratch = [S.wtconv_scan_workspace_size(op, B, T, C, order, 1) for op in (0, 1)]
    sizes = [n for n in (*scratch, d["x"].nbytes, d["h0"].nbytes, want["states"].nbytes, 4 * C) if n > 0] * 4
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for round in range(2):
        given = {k: v if v is None else v.clone() for k, v in d.items()}
        side.wait_stream(torch.cuda.current_stream())
        if round == 0:
            with torch.cuda.stream(side):
                torch.cuda._sleep(100_000_000)
        else:
            torch.cuda._sleep(100_000_000)
            dirty(sizes)
        y, h, states = S.wtconv_scan_forward(given["x"], given["gate"], given["gate_bias"], given["h0"], None, layout, True,
                                             stream=side)
        if round == 0:
            dirty(sizes)
        dx, dg, db, dh0 = S.wtconv_scan_backward(given["x"], given["gate"], given["gate_bias"], states, given["dy"],
                                                 given["dh_last"], None, layout, stream=side)
        del given
        if round == 0:
            dirty(sizes)
        torch.cuda.synchronize()
        for k, t in (("y", y), ("h_last", h), ("states", states), ("dx", dx), ("d_gate", dg), ("d_gate_bias", db), ("d_h0", dh0)):
            assert torch.equal(t, want[k]), (round, k)


@pytest.mark.gpu
def test_given_stream_step():
    """As above for single tokens; and results that the current stream still reads when they are let go of
    are not overwritten by the side stream's next call."""
    g = torch.Generator(device="cuda").manual_seed(29)
    x, gate = torch.randn(2, 64, 4096, generator=g, device="cuda").bfloat16()
    bias, pool = torch.ones(4096, device="cuda"), torch.zeros(64, 4096, device="cuda")
    want = S.wtconv_scan_step(x, gate, bias, pool.clone())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    first = x.clone()
    side.wait_stream(torch.cuda.current_stream())
    y = S.wtconv_scan_step(first, gate, bias, pool.clone(), stream=side)
    del first
    dirty([x.nbytes, pool[0].nbytes * 64] * 4)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(100_000_000)
    late = y.clone()  # runs after the sleep
    del y
    S.wtconv_scan_step(-x, gate, bias, pool, stream=side)  # runs at once
    torch.cuda.synchronize()
    assert torch.equal(late, want)


def check_second_derivatives(x, gate, bias, h0, layout):
    """First derivatives taken with create_graph are the plain ones; their derivative by any input of
    the scan is refused, also where a loss has other parts and where dy depends on nothing."""
    given = [t.clone().requires_grad_() for t in (x, gate, bias, h0)]
    y, h = S.gated_scan(*given, None, layout)
    plain = torch.autograd.grad(y.sum() + h.sum(), given, retain_graph=True)
    kept = torch.autograd.grad(y.sum() + h.sum(), given, create_graph=True)
    for a, b in zip(plain, kept):
        assert torch.equal(a, b) and b.requires_grad
    for t, g in zip(given, kept):
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.square().sum() + t.square().sum()).backward(retain_graph=True)
    scale = torch.ones((), requires_grad=True, device=x.device)  # dy depends on an input, the scan's inputs on none
    y, _ = S.gated_scan(given[0], gate, bias, None, None, layout)
    (g,) = torch.autograd.grad((y * scale).sum(), given[0], create_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(g.sum(), scale)


def test_second_derivatives_refuse_without_a_gpu(monkeypatch):
    def forward(x, gate, gate_bias, h0=None, lengths=None, layout="planes", keep_states=False):
        return x * 2, x.sum(2), x.clone()

    def backward(x, gate, gate_bias, states, dy, dh_last=None, lengths=None, layout="planes"):
        return dy * 2, dy * 3, dy.sum((0, 2)), dy.sum(2)

    monkeypatch.setattr(S, "wtconv_scan_forward", forward)
    monkeypatch.setattr(S, "wtconv_scan_backward", backward)
    x = torch.ones(2, 3, 4)
    check_second_derivatives(x, x, torch.ones(3), torch.ones(2, 3), "planes")


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_second_derivatives_refuse(layout):
    d = make(2, 100, 8, layout, torch.float32, seed=21)
    check_second_derivatives(d["x"], d["gate"], d["gate_bias"], d["h0"], layout)


@pytest.mark.gpu
def test_state_may_move_on_before_the_backward():
    """A state that is carried from call to call in place: the backward needs only what the forward kept."""
    d = make(2, 100, 8, "tokens", torch.float32, seed=31)
    x, state = d["x"].clone().requires_grad_(), d["h0"].clone()
    y, h = S.gated_scan(x, d["gate"], d["gate_bias"], state, None, "tokens")
    state.copy_(h.detach())
    y.backward(d["dy"])
    want = reference({**d, "dh_last": None}, "tokens")
    R.assert_near("dx", R.time_first(x.grad, "tokens"), want["dx"])


GARBAGE = [float("inf"), float("-inf"), float("nan")]


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,C", [(37, 9), (400, 64), (2600, 20), (1000, 512)])
@pytest.mark.parametrize("bad", GARBAGE, ids=str)
def test_zeros_past_a_length(bad, T, C, dtype, layout):
    """y, dx and d_gate are exact zeros from a length on, whatever states and gradients come to it."""
    lengths = [T, T // 2 + 3, 0, 1, min(T, 63)]
    d = make(len(lengths), T, C, layout, dtype, seed=22, lengths=lengths)
    d["dh_last"][1], d["h0"][3], d["dh_last"][4] = bad, bad, bad
    got = run(d, layout)
    for k in ("y", "dx", "d_gate"):
        v = R.time_first(got[k], layout)
        for b, n in enumerate(lengths):
            assert (v[n:, b] == 0).all(), (k, b)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("T,C", [(37, 9), (400, 64), (2600, 20), (1000, 512)])
@pytest.mark.parametrize("bad", GARBAGE, ids=str)
def test_empty_sequences_give_no_gradient(bad, T, C, dtype, layout):
    """A sequence without positions has no part in d_gate_bias, whatever its state and dh_last hold; those
    come out as h_last and d_h0 as they are."""
    lengths = [T, 0, T // 2]
    d = make(3, T, C, layout, dtype, seed=23, lengths=lengths)
    want = reference(d, layout)
    d["h0"][1], d["dh_last"][1] = bad, bad
    got = run(d, layout)
    R.assert_near("d_gate_bias", got["d_gate_bias"].double().cpu().numpy(), want["d_gate_bias"], scale=want["abs"].max())
    for k, given in (("h_last", "h0"), ("d_h0", "dh_last")):
        assert torch.equal(torch.nan_to_num(got[k][1], 5.0), torch.nan_to_num(d[given][1], 5.0)), k


@pytest.mark.gpu
def test_autograd_sees_what_is_written():
    """A graph that saved the pool or an output's buffer before a call wrote it is refused."""
    d = make(2, 20, 8, "tokens", torch.float32, seed=25)
    w = torch.ones(8, device="cuda", requires_grad=True)
    pool, y, dx, dg = (torch.zeros(s, device="cuda") for s in ((4, 8), (2, 20, 8), (2, 20, 8), (2, 20, 8)))
    losses = [(t * w).sum() for t in (pool, y, dx, dg)]
    S.wtconv_scan_step(d["x"][:, 0], d["gate"][:, 0], d["gate_bias"], pool)
    _, _, states = S.wtconv_scan_forward(d["x"], d["gate"], d["gate_bias"], layout="tokens", keep_states=True, y=y)
    S.wtconv_scan_backward(d["x"], d["gate"], d["gate_bias"], states, d["dy"], layout="tokens", dx=dx, d_gate=dg)
    for loss in losses:
        with pytest.raises(RuntimeError, match="modified by an inplace"):
            loss.backward()


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
def test_gates_that_cancel(layout):
    """a and b = 1 - a to a few units of their own value where a large gate and a large bias nearly cancel.
    Over one position of dy = 1 and no dh: dx = b and d_h0 = a exactly.  Units of 2^-24: z is rounded
    (|z|), its product with log2 e too (|z|), which is itself off by 0.23; these move e by 2.23 |z|, the
    exponential by 4, and e's error reaches b times a and a times b.  1 + e, its reciprocal and e a round
    once each; one more is left for the terms of second order."""
    g = torch.Generator(device="cuda").manual_seed(24)
    B, C = 512, 256
    z = torch.rand(B, C, generator=g, device="cuda") * 30 - 10
    bias = torch.rand(C, generator=g, device="cuda") * 40 + 20
    shape = (B, 1, C) if layout == "tokens" else (B, C, 1)
    gate, one = (z - bias).view(shape), torch.ones(shape, device="cuda")
    _, _, states = S.wtconv_scan_forward(one, gate, bias, layout=layout, keep_states=True)
    dx, _, _, d_h0 = S.wtconv_scan_backward(one, gate, bias, states, one, layout=layout)
    z = gate.view(B, C).double() + bias.double()
    a, b = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    for name, got, want, rest in (("a", d_h0, a, b), ("b", dx.view(B, C), b, a)):
        units = (got.double() - want).abs() / want * 2.0 ** 24
        assert (units <= (2.23 * z.abs() + 4) * rest + 4).all(), (name, float(units.max()))


@pytest.mark.parametrize("layout,C", [(layout, (1 << 31) - k) for layout in (0, 1) for k in (1, 2, 31, 32, 33, 256)])
def test_workspace_of_the_most_channels(layout, C):
    """B*C < 2^31: numbers of strips next to that limit are not formed past it.  One float a channel of
    every strip is what the sums of d_gate_bias take."""
    for dtype, width in ((W.F32, 32), (W.BF16, 64)):
        want = 4 * C if layout == 0 else 4 * (-(-C // width) * width)
        got = S.wtconv_scan_workspace_size(S.OP_SCAN_BACKWARD, 1, 1, C, layout, dtype)
        assert got == -(-want // 256) * 256
        assert S.wtconv_scan_workspace_size(S.OP_SCAN_FORWARD, 1, 1, C, layout, dtype) == 0


@pytest.mark.gpu
def test_step_of_the_most_channels():
    """One sequence of 2^31 - 1 channels: the first and the last are updated like any other."""
    C = (1 << 31) - 1
    x = torch.ones(1, C, dtype=torch.bfloat16, device="cuda")
    bias, pool = torch.zeros(C, device="cuda"), torch.zeros(1, C, device="cuda")
    y = S.wtconv_scan_step(x, x, bias, pool)
    want = 1 / (1 + np.exp(1.0))
    for at in (slice(0, 300), slice(C - 300, C)):
        R.assert_near("pool", pool[0, at].double().cpu().numpy(), np.full(300, want))
        R.assert_near("y", y[0, at].double().cpu().numpy(), np.full(300, want), torch.bfloat16)
    assert float((pool - pool[0, 0]).abs().max()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("start", [0, 1, 3])
def test_repeated_rows(start, dtype, layout):
    """One row for every position of tokens, one plane for every channel: a row stride of 0, also where the
    row starts at an odd element.  What lies before the row is NaN.  Results are those of the same rows laid out."""
    B, T, C = 3, 200, 40
    d = make(B, T, C, layout, dtype, seed=32)
    laid_out = dict(d)
    for k in ("x", "gate", "dy"):
        n = d[k].shape[2]
        buf = torch.full((start + n,), float("nan"), dtype=dtype, device="cuda")
        buf[start:] = d[k][0, 0]
        d[k] = buf[start:].expand(d[k].shape)
        laid_out[k] = d[k].contiguous()
    want = run(laid_out, layout)
    for k, t in run(d, layout).items():
        assert torch.equal(t, want[k]) and torch.isfinite(t).all(), k


@pytest.mark.gpu
@pytest.mark.parametrize("layout", ["planes", "tokens"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=lambda t: str(t)[6:])
def test_rows_past_32_bits(dtype, layout):
    """Rows of one sequence further apart than 2^31 elements in all, at any alignment."""
    B, T, C = (1, 130, 24) if layout == "tokens" else (1, 700, 130)
    d = make(B, T, C, layout, dtype, seed=26)
    want = reference(d, layout)
    rows, inner = d["x"].shape[1:]
    for odd in (0, 1):
        row = (1 << 24) + 1024 + odd
        store = torch.empty(rows * row, dtype=dtype, device="cuda")

        def far(t, k):
            view = store.as_strided(t.shape, (rows * row, row, 1), k * 1024)
            view.copy_(t)
            return view

        got = run({**d, "x": far(d["x"], 0), "gate": far(d["gate"], 1), "dy": far(d["dy"], 2)}, layout,
                  dx=far(d["x"] * 0, 3), d_gate=far(d["x"] * 0, 4))
        check(got, want, layout, dtype)
        del got, store
