"""The linear layer (GPU) element by element, at the ends of its arguments'
range, against float64."""
import math

import pytest

from .gpuhelp import say
from .test_gpu_linear import act64, rel

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def gelu_grid(t, dtype):
    """t x 64 values from -9 to 9 and the 64 x 64 identity: the products are
    exact, so the activation's argument is known to the last bit."""
    import torch
    x = torch.linspace(-9.0, 9.0, 64 * t, device="cuda").view(t, 64).to(dtype)
    return x, torch.eye(64, device="cuda").to(dtype)


def gelu_bound(z):
    """Relative error of 0.5 z erfc(-z / sqrt 2) in float32: the argument
    carries 1.5 roundings, which erfc(u) multiplies by 2 u^2 + 1 = z^2 + 1 at
    most; erfc itself 16 units of its last place; two roundings of products.
    The slope's other term, z exp(-z^2 / 2) / sqrt(2 pi), carries less."""
    return U32 * (1.5 * z * z + 40.0)


# rows, matrix cores for few tokens, tiles
@pytest.mark.parametrize("t", [4, 40, 130])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gelu_element_by_element(gpu_lib, t, dtype):
    import torch
    say(f"gelu {t} {dtype}")
    dt = getattr(torch, dtype)
    out = 2.0 ** -8 if dtype == "bfloat16" else 0.0   # one rounding of the output
    x, w = gelu_grid(t, dt)
    y, z = torch.empty_like(x), torch.empty_like(x)
    gpu_lib.linear_forward(x, w, y, act="gelu", preact=z)
    assert torch.equal(z, x)
    zz = x.double()
    want = act64(zz, "gelu")
    assert torch.all((y.double() - want).abs() <= (out + gelu_bound(zz)) * want.abs())


@pytest.mark.parametrize("t", [4, 40, 130])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gelu_slope_element_by_element(gpu_lib, t, dtype):
    """dx of dy = 1 through the identity is act'(z); with bfloat16 and few
    tokens it passes through two planes (2^-16), with more through one."""
    import torch
    say(f"gelu slope {t} {dtype}")
    dt = getattr(torch, dtype)
    out = 2.0 ** -8 + 2.0 ** -16 if dtype == "bfloat16" else 0.0
    x, w = gelu_grid(t, dt)
    dx = torch.empty_like(x)
    gpu_lib.linear_backward(torch.ones_like(x), weight=w, dx=dx, act="gelu", preact=x)
    z = x.double()
    phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
    rest = z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    slack = (gelu_bound(z) + U32) * (phi + rest.abs())
    assert torch.all((dx.double() - (phi + rest)).abs() <= out * (phi + rest).abs() + slack)
