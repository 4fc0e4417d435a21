"""The layer's binding on a stream of the caller's: its scratch, outputs and inputs keep their memory."""
import pytest
import torch
from parity import PARAMS, to_device

from memory_bound_cnn_gb300 import inputs as I
from memory_bound_cnn_gb300 import wtconv as W


def dirty(sizes):
    """Blocks of these many bytes of the current stream's pool, filled and let go."""
    for n in sizes:
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xff)


@pytest.mark.gpu
@pytest.mark.parametrize("hold", ["side", "current"])
@pytest.mark.parametrize("dims", [(4, 32, 56, 56, 2, 5), (2, 8, 256, 256, 3, 5)], ids=str)
def test_given_stream_without_workspace(dims, hold):
    """side: the current stream uses whatever memory it can get again before the call's work has run.
    current: it still has writes queued to blocks that it let go of, which no output may lie in."""
    shape = I.LayerShape(*dims, dtype="f32")
    d = to_device(I.make_inputs(shape, seed=23))

    def call(d, **kw):
        p = [d[n] for n in PARAMS]
        y = W.wtconv_forward(d["x"], *p, **kw)
        dx = W.wtconv_backward_input(d["dy"], *p, **kw)
        g1 = W.wtconv_backward_weights(d["x"], d["dy"], *p, **kw)
        both, g2 = W.wtconv_backward(d["x"], d["dy"], *p, **kw)
        return [y, dx, both, *g1.values(), *g2.values()]

    want = call(d)
    scratch = [W.wtconv_workspace_size(op, *dims, W.F32) for op in range(4)]
    sizes = sorted({n for n in (*scratch, *(t.nbytes for t in d.values())) if n > 0}) * 4
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    given = {k: v.clone() for k, v in d.items()}
    side.wait_stream(torch.cuda.current_stream())
    if hold == "side":
        with torch.cuda.stream(side):
            torch.cuda._sleep(100_000_000)
    else:
        torch.cuda._sleep(100_000_000)
        dirty(sizes)
    got = call(given, stream=side)
    del given
    if hold == "side":
        dirty(sizes)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_external_stream():
    d = to_device(I.make_inputs(I.LayerShape(2, 8, 28, 28, 2, 5, dtype="bf16"), seed=24))
    p = [d[n] for n in PARAMS]
    want = W.wtconv_forward(d["x"], *p)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = W.wtconv_forward(d["x"], *p, stream=torch.cuda.ExternalStream(side.cuda_stream))
    side.synchronize()
    assert torch.equal(got, want)
