"""Corners of the gated scan: very long rows, far rows, masked garbage, streams, second derivatives."""
import numpy as np
import pytest
import scan_reference as R
import torch
from test_scan import make, run

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
