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


#: float32 numbers at the top of the range: from FLT_MAX down across the
#: midpoint (about 3.396e38) from which rounding to bfloat16 gives infinity.
TOP = (3.4028234663852886e38, -3.4e38, 3.3962e38, -3.39615e38, 3.39e38, 1e38, -2e37, 1.0)


@pytest.mark.parametrize("t", [4, 40, 130])
def test_float32_values_near_the_largest(gpu_lib, t):
    """x (forward) and dy (backward) with entries up to FLT_MAX against small
    weights: every output is finite in float32 and has float32's accuracy."""
    import torch
    say(f"linear top {t}")
    g = torch.Generator(device="cuda").manual_seed(t)
    big = torch.tensor(TOP, device="cuda").repeat(t * 8).view(t, 64)
    w = torch.randn(64, 64, generator=g, device="cuda") * 1e-3
    y = torch.empty_like(big)
    gpu_lib.linear_forward(big, w, y)
    assert rel(y, big.double() @ w.double().T) <= 2.0 ** -19
    x = torch.randn(t, 64, generator=g, device="cuda") * 1e-4
    dx, dw = torch.empty_like(big), torch.empty_like(w)
    gpu_lib.linear_backward(big, x, w, dx=dx, dw=dw)
    assert rel(dx, big.double() @ w.double()) <= 2.0 ** -19
    assert rel(dw, big.double().T @ x.double()) <= 2.0 ** -19


def test_few_tokens_gradient_near_the_largest(gpu_lib):
    """bfloat16, at most 64 tokens, an activation: dz = dy act'(z) is held in
    two planes and may lie above the largest bfloat16 number in float32."""
    import torch
    t = 40
    z = torch.linspace(1.2, 1.3, t * 64, device="cuda").view(t, 64).bfloat16()
    zz = z.double()
    s = torch.sigmoid(zz)
    slope = s * (1 + zz * (1 - s))
    dy = torch.full_like(z, 3.3895313892515355e38)     # the largest
    dz = dy.double() * slope
    over = (dz > 3.3962e38) & (dz < 3.4028e38)
    assert over.any()
    dy = torch.where(over, dy, torch.zeros_like(dy))
    dz = dy.double() * slope
    w, dx = (torch.eye(64, device="cuda") * 2.0 ** -10).bfloat16(), torch.empty_like(z)
    gpu_lib.linear_backward(dy, weight=w, dx=dx, act="silu", preact=z)
    assert rel(dx, dz * 2.0 ** -10) <= 2.0 ** -8 + 2.0 ** -16


@pytest.mark.parametrize("t", [4, 40, 130])
def test_float32_values_near_zero(gpu_lib, t):
    """Entries below 2^-110: the planes end at 2^-133, so an entry is taken to
    within half of that (and the products with 1 are exact)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(t, 64, generator=g, device="cuda") * 2.0 ** -118
    w, y = torch.eye(64, device="cuda"), torch.empty_like(x)
    gpu_lib.linear_forward(x, w, y)
    assert float((y.double() - x.double()).abs().max()) <= 2.0 ** -134


def test_columns_of_one_buffer(gpu_lib):
    """y, z and the residual beside x in one buffer, dx beside dy: the bits of
    separate tensors, and the columns between them untouched."""
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        for t in (3, 40, 140):
            g = torch.Generator(device="cuda").manual_seed(t)
            buf = torch.randn(t, 200, generator=g, device="cuda").to(dtype)
            w = (torch.randn(32, 64, generator=g, device="cuda") * 0.1).to(dtype)
            x, y, z, r = buf[:, :64], buf[:, 64:96], buf[:, 96:128], buf[:, 129:161]
            x0, r0, gap = x.clone(), r.clone(), (buf[:, 128].clone(), buf[:, 161:].clone())
            want, zwant = torch.empty(t, 32, dtype=dtype, device="cuda"), torch.empty(t, 32, dtype=dtype, device="cuda")
            gpu_lib.linear_forward(x0, w, want, act="silu", residual=r0, preact=zwant)
            gpu_lib.linear_forward(x, w, y, act="silu", residual=r, preact=z)
            assert torch.equal(y, want) and torch.equal(z, zwant)
            assert torch.equal(x, x0) and torch.equal(r, r0)
            assert torch.equal(buf[:, 128], gap[0]) and torch.equal(buf[:, 161:], gap[1])
            dxw = torch.empty(t, 64, dtype=dtype, device="cuda")
            gpu_lib.linear_backward(r0, weight=w, dx=dxw)
            gpu_lib.linear_backward(r, weight=w, dx=x)
            assert torch.equal(x, dxw) and torch.equal(r, r0) and torch.equal(y, want)


def test_orthogonalize_beside_its_input(gpu_lib):
    import torch
    for m, n in ((3, 40), (70, 40), (300, 200)):
        g = torch.Generator(device="cuda").manual_seed(m)
        buf = torch.randn(m, 2 * n, generator=g, device="cuda")
        g0, want = buf[:, :n].clone(), torch.empty(m, n, device="cuda")
        gpu_lib.orthogonalize(g0, want)
        gpu_lib.orthogonalize(buf[:, :n], buf[:, n:])
        assert torch.equal(buf[:, n:], want) and torch.equal(buf[:, :n], g0)


@pytest.mark.parametrize("act", ["relu", "relu2", "gelu", "silu"])
def test_nan_preactivation_shows_in_the_gradients(gpu_lib, act):
    """A NaN pre-activation (a non-finite operand) makes its row of dx, its
    rows of dw and its entry of db NaN, and nothing else."""
    import torch
    for dtype in (torch.float32, torch.bfloat16):
        for t in (4, 40, 130):
            g = torch.Generator(device="cuda").manual_seed(t)
            x, w = torch.randn(t, 80, generator=g, device="cuda").to(dtype), torch.randn(48, 80, generator=g, device="cuda").to(dtype)
            dy, z = (torch.randn(t, 48, generator=g, device="cuda").to(dtype) for _ in range(2))
            z[2, 7] = float("nan")
            dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(48, device="cuda")
            gpu_lib.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, act=act, preact=z)
            for v, at in ((dx, 2), (dw, 7), (db.view(48, 1), 7)):
                assert torch.isnan(v[at]).all()
                assert torch.isfinite(v).all(1).sum() == v.shape[0] - 1
