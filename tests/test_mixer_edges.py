"""Corners of the selective scan: sums over channels that cancel."""
import pytest
import ssm_reference as R
import torch
from test_selective import DTYPES, LAYOUTS, make, reference, run


# ------------------------------------------------------------------------ sums over channels

@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", DTYPES, ids=lambda t: str(t)[6:])
@pytest.mark.parametrize("N", [5, 16, 32, 64])
def test_sums_over_channels_that_cancel(N, dtype, layout):
    """Channels in pairs whose products differ in sign and, by about 1/64, in size: dB and dC are as exact as sums in fp32
    of the products, and rounded once."""
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
