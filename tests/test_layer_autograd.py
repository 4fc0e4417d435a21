"""The layer's autograd function: first derivatives only, and a refusal beyond them."""
import pytest
import torch
from parity import PARAMS, to_device

from memory_bound_cnn_gb300 import inputs as I
from memory_bound_cnn_gb300 import wtconv as W

SHAPE = I.LayerShape(2, 4, 16, 16, 2, 3, dtype="f32")


def check_second_derivatives(d, turned):
    """turned: x arrives as a transposed view, of which the function keeps a contiguous copy."""
    leaf = d["x"].transpose(2, 3).contiguous() if turned else d["x"].clone()
    leaf.requires_grad_()
    params = [d[n].clone().requires_grad_() for n in PARAMS]
    y = W.WTConvFunction.apply(leaf.transpose(2, 3) if turned else leaf, *params)
    leaves = [leaf, *params]
    plain = torch.autograd.grad(y, leaves, d["dy"], retain_graph=True)
    kept = torch.autograd.grad(y, leaves, d["dy"], create_graph=True)
    for a, b in zip(plain, kept):
        assert torch.equal(a, b) and b.requires_grad
    for t, g in zip(leaves, kept):
        with pytest.raises(RuntimeError, match="second derivative"):
            (g.square().sum() + t.square().sum()).backward(retain_graph=True)
    with pytest.raises(RuntimeError, match="second derivative"):
        torch.autograd.grad(kept[1].sum(), leaf)


@pytest.mark.parametrize("turned", [False, True])
def test_second_derivatives_refuse_without_a_gpu(turned, monkeypatch):
    def backward(x, dy, base_w, base_bias, base_scale, wavelet_w, wavelet_scale):
        return dy * 2, {"d_base_w": base_w * 3, "d_base_bias": base_bias * 3, "d_base_scale": base_scale * 3,
                        "d_wavelet_w": wavelet_w * 3, "d_wavelet_scale": wavelet_scale * 3}

    monkeypatch.setattr(W, "wtconv_forward", lambda x, *params: x * 2)
    monkeypatch.setattr(W, "wtconv_backward", backward)
    check_second_derivatives(I.make_inputs(SHAPE, seed=25), turned)


@pytest.mark.gpu
@pytest.mark.parametrize("turned", [False, True])
def test_second_derivatives_refuse(turned):
    check_second_derivatives(to_device(I.make_inputs(SHAPE, seed=25)), turned)
