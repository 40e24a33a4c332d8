"""The 8-bit linear layer's gradients against the exact ones and against differences, with bounds that a missing, negated, halved or
transposed gradient breaks.

A gradient is a b + (a's error) b + a (b's error) + (a's error) (b's error). An operand's error is at most half a step of
its 8-bit type: 2^-4 (e4m3) or 2^-3 (e5m2) of the value, or half the smallest step at its group's scale, whichever is
more. With |.| the Frobenius and |.|_2 the spectral norm, |e b| <= |e| |b|_2, and along the gradient g itself
<e b, g> <= |e| |g b^T|. No independence or symmetry of the errors is used: rounding is not unbiased where a
distribution falls off across a step."""

import pytest
import torch

from test_gpu_quantised_training import example, layer  # noqa: F401  (example is a fixture)

pytestmark = pytest.mark.gpu


def most(v, step, least):
    """The norm of the largest errors; least: half the smallest step over the largest value."""
    return float(torch.maximum(v.abs() * step, v.abs().max() * least).norm())


E4M3 = (2.0 ** -4, 2.0 ** -10 / 448)
E5M2 = (2.0 ** -3, 2.0 ** -17 / 57344)


def spectral(v):
    return float(torch.linalg.matrix_norm(v, 2))


def along(g, a, fa, b, fb, u):
    """The most that errors add to <a b, g>."""
    ea, eb = most(a, *fa), most(b, *fb)
    return (1 + u) * (ea * float((g @ b.t()).norm()) + eb * float((a.t() @ g).norm()) + ea * eb * spectral(g)) + u * float(g.norm()) ** 2


@pytest.mark.parametrize("T,C,N", [(60, 200, 150), (256, 384, 300), (1030, 640, 384)])
def test_gradients(example, T, C, N):  # noqa: F811
    x, w, dy, y, dx, before, grad = layer(example, T, C, N, 7)
    x, w, dy, dx = x.detach().double().cpu(), w.double().cpu(), dy.double().cpu(), dx.double().cpu()
    dw = (grad.double() - before.double()).cpu()
    for got, a, fa, b, fb, u in ((dx, dy, E5M2, w, E4M3, 2.0 ** -8), (dw, dy.t(), E5M2, x, E4M3, 2.0 ** -20)):
        want, ea, eb = a @ b, most(a, *fa), most(b, *fb)
        size = float(want.norm())
        bound = (1 + u) * (ea * spectral(b) + spectral(a) * eb + ea * eb) + u * size
        assert bound < 0.75 * size
        assert float((got - want).norm()) <= bound
        bound = along(want, a, fa, b, fb, u)
        assert bound < 0.5 * size ** 2
        assert abs(float((got * want).sum()) - size ** 2) <= bound


@pytest.mark.parametrize("T,C,N", [(60, 200, 150), (256, 384, 300)])
def test_differences(example, T, C, N):  # noqa: F811
    """Of the loss in 64 bits along the layer's gradients (the loss is linear in x and in w, so differences are exact)."""
    x, w, dy, y, dx, before, grad = layer(example, T, C, N, 9)
    x, w, g = x.detach().double().cpu(), w.double().cpu(), dy.double().cpu()
    dx, dw = dx.double().cpu(), (grad.double() - before.double()).cpu()
    h = 1e-3
    for got, a, fa, b, fb, u, loss in ((dx, g, E5M2, w, E4M3, 2.0 ** -8, lambda v, h: ((x + h * v) @ w.t() * g).sum()),
                                       (dw, g.t(), E5M2, x, E4M3, 2.0 ** -20, lambda v, h: (x @ (w + h * v).t() * g).sum())):
        d = float(loss(got, h) - loss(got, -h)) / (2 * h)
        size, bound = float(got.square().sum()), along(got, a, fa, b, fb, u)
        assert size > 0 and bound < 0.5 * size
        assert abs(d - size) <= bound + 1e-9 * size


def test_no_second_derivative(example):  # noqa: F811
    """The backward is made of calls that autograd does not see: asked to differentiate it, it says so."""
    x = torch.randn(64, 128, device="cuda").bfloat16().requires_grad_()
    w, grad = torch.randn(96, 128, device="cuda"), torch.zeros(96, 128, device="cuda")
    y = example.Fp8Linear.apply(x, w, grad)
    dx, = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="differentiate twice"):
        dx.float().sum().backward()
