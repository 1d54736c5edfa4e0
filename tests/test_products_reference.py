"""The 64-bit gradients that the kernels are held to, against central
differences of the 64-bit definitions."""
import pytest
import torch

import product_reference as ref


def differences(f, x, d, h=1e-6):
    """<d, f> as a function of each element of x, by central differences."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + h
        up = (f() * d).sum()
        flat[i] = v - h
        down = (f() * d).sum()
        flat[i] = v
        out[i] = (up - down) / (2 * h)
    return g


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu", "swiglu"])
def test_activation_gradients(act):
    torch.manual_seed(1)
    z = 2 * torch.randn(3, 8, dtype=torch.float64)
    dy = torch.randn(3, 4 if act == "swiglu" else 8, dtype=torch.float64)
    zero = torch.zeros_like(z)
    fwd = (lambda: ref.gated(z, zero)[0]) if act == "swiglu" else (lambda: ref.activation(z, zero, act)[0])
    want = differences(fwd, z, dy)
    got = ref.gated_back(z, dy, torch.zeros_like(dy))[0] if act == "swiglu" else ref.activation_back(z, dy, act)[0]
    # the differences are off by about h^2 and by rounding over h
    assert (got - want).abs().max() <= 1e-7


def test_layer_gradients():
    """Gradients of a product by rows and by weights, and of the combine."""
    torch.manual_seed(2)
    x, w, dy = (torch.randn(s, dtype=torch.float64) for s in ((5, 4), (3, 4), (5, 3)))
    f = lambda: ref.product(x, w)[0]  # noqa: E731
    assert (differences(f, x, dy) - ref.product(dy, w.T)[0]).abs().max() <= 1e-7
    assert (differences(f, w, dy) - ref.product(dy.T, x.T)[0]).abs().max() <= 1e-7
    y, tw, dout = (torch.randn(s, dtype=torch.float64) for s in ((6, 4), (3, 2), (3, 4)))
    dst = torch.tensor([[2, 0], [-1, 3], [5, 1]])
    live = (dst >= 0).double()
    g = lambda: ((tw * live)[..., None] * y[dst.clamp_min(0)]).sum(1)  # noqa: E731
    by_pair, dw, _ = ref.combine_back(dout, y, tw, dst)
    dyr = torch.zeros_like(y)
    for t in range(3):
        for j in range(2):
            if dst[t, j] >= 0:
                dyr[dst[t, j]] = by_pair[t, j]
    assert (differences(g, y, dout) - dyr).abs().max() <= 1e-7
    assert (differences(g, tw, dout) - dw).abs().max() <= 1e-7
