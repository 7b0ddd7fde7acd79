"""The gradients' formulas against differences of the forward's, and the 8-bit format's own
definition, in 64 bits on the CPU."""
import math

import pytest
import torch

import train_reference as R


def case(n, H, I, seed):
    g = torch.Generator().manual_seed(seed)

    def randn(*shape, std=1.0):
        return torch.randn(*shape, generator=g, dtype=torch.float64) * std

    return randn(n, H), randn(2 * I, H, std=H ** -0.5), randn(H, I, std=I ** -0.5), randn(n, H)


@pytest.mark.parametrize("n,H,I", [(1, 64, 64), (5, 64, 128), (9, 192, 64)])
def test_gradients_against_differences(n, H, I):
    x, w13, w2, dy = case(n, H, I, n + H + I)
    h, _, _ = R.forward(x, w13, w2)
    _, _, dx, dw13, dw2 = R.backward(dy, x, w13, w2, h)
    g = torch.Generator().manual_seed(7)
    step = 1e-5
    for which, grad in ((0, dx), (1, dw13), (2, dw2)):
        args = [x, w13, w2]
        v = torch.randn(args[which].shape, generator=g, dtype=torch.float64)
        up, down = list(args), list(args)
        up[which] = args[which] + step * v
        down[which] = args[which] - step * v
        num = float(((R.forward(*up)[2] - R.forward(*down)[2]) * dy).sum()) / (2 * step)
        got = float((grad * v).sum())
        # central differences: step^2 times third derivatives, here below 1e3 of the terms, and
        # the sums' own 1e-16 over the step
        scale = float((grad * v).abs().sum())
        assert abs(num - got) <= 1e-6 * scale, (which, num, got)


def test_gradients_against_autograd():
    x, w13, w2, dy = (t.requires_grad_() for t in case(4, 64, 192, 5))
    h = x @ w13.T
    g, u = h.chunk(2, 1)
    y = (torch.nn.functional.silu(g) * u) @ w2.T
    want = torch.autograd.grad((y * dy).sum(), (x, w13, w2))
    with torch.no_grad():
        got = R.backward(dy, x, w13, w2, R.forward(x, w13, w2)[0])[2:]
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-11, atol=1e-13)


def test_e4m3_values():
    v = R.e4m3_values()
    assert v[126] == 448.0 and math.isnan(v[127]) and v[1] == 2.0 ** -9 and v[8] == 2.0 ** -6
    assert bool((v[1:127] > v[:126]).all())
    codes = torch.arange(256, dtype=torch.uint8)
    assert torch.equal(torch.nan_to_num(codes.view(torch.float8_e4m3fn).double(), nan=999.0),
                       torch.nan_to_num(v, nan=999.0))


def test_nearest_codes_are_the_types_conversion():
    g = torch.Generator().manual_seed(1)
    v = torch.randn(64, 96, generator=g) * torch.exp(4 * torch.randn(64, 96, generator=g))
    e = R.scale_exponents(v)
    q = (v.double().unflatten(-1, (-1, 32)) / R.power(e)[..., None]).flatten(-2)
    assert float(q.abs().max()) <= 448.0
    assert torch.equal(R.nearest_codes(v, e), q.float().to(torch.float8_e4m3fn).double())
    # the least such scale: half of it would not do
    most = v.double().unflatten(-1, (-1, 32)).abs().amax(-1)
    assert bool((most > 448.0 * R.power(e - 1)).all())
