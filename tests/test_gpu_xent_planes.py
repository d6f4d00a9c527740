"""Precision of dz in the cross entropy's bfloat16 gradients of few tokens (GPU):
two planes, 16 bits, up to 64 tokens however the rows lie, because a gradient
adds too few of its roundings for them to average out.

The inputs make dz's rounding visible behind the outputs' own: tokens come in
pairs of one x and one target whose dloss differ by -(1 + 2^-10), rows of W in
pairs of opposite sign with logits near zero, so that an output is the small
rest (2^-10, and the logits' size) of terms that nearly cancel and its own
rounding, relative to that rest, is far below the terms' 2^-8.

Bounds, element by element in float64: dz in two planes is off by at most 2^-16
of its value, its logit and exponential as in the other sizes' tests (the module
imported here says why), an output by the terms times that, by its sum's
roundings in float32 and by half a step of its own, 2^-8."""
import math

import pytest

from .gpuhelp import say
from .test_gpu_xent import IGNORE, rand, reference, z_error

pytestmark = pytest.mark.gpu


def paired(t, k, n, pad, seed=1):
    import torch
    bf = torch.bfloat16
    x, w = rand((t, k), seed, bf, pad), rand((n, k), seed + 1, bf, pad, 0.02 * k ** -0.5)
    x[1::2] = x[:t - 1:2][:t // 2]
    w[1::2] = -w[:n - 1:2][:n // 2]
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    y = torch.randint(0, n, (t,), generator=g, device="cuda")
    if t > 6:
        y[4] = y[2] = IGNORE
    y[1::2] = y[:t - 1:2][:t // 2]
    dloss = torch.rand(t, generator=g, device="cuda") / t + 0.1 / t
    dloss[1::2] = -(1 + 2.0 ** -10) * dloss[:t - 1:2][:t // 2]
    return x, w, y, dloss


@pytest.mark.parametrize("t", [2, 32, 33, 40, 47, 48, 49, 63, 64])
@pytest.mark.parametrize("k,pad", [(64, 0), (72, 8), (65, 0), (128, 3)])
def test_two_planes(gpu_lib, t, k, pad):
    import torch
    for n in (40, 131, 1000, 20001):
        say(f"cross entropy planes {t} {k} {n} {pad}")
        x, w, y, dloss = paired(t, k, n, pad)
        lse = torch.empty(t, device="cuda")
        gpu_lib.cross_entropy_forward(x, w, y, lse=lse)
        dx, dw = torch.full_like(x, float("nan")), torch.full_like(w, float("nan"))
        gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dx=dx, dw=dw)
        dz, size = reference(x, w, y, 0.0, 0.0, lse, dloss.abs())
        sign = dloss.double().sign()[:, None]
        dz = dz * sign
        err = dz.abs() * 2.0 ** -16 + size * (z_error(x, w) + 2.0 ** -21 + 2.0 ** -22)
        for got, a, lost, b, length in ((dx, dz, err, w.double(), n),
                                        (dw, dz.t().contiguous(), err.t().contiguous(), x.double(), t)):
            want, terms, worst = torch.mm(a, b), torch.mm(a.abs(), b.abs()), torch.mm(lost, b.abs())
            tol = 2.0 ** -8 * want.abs() + 1.01 * worst + terms * 2.0 ** -24 * (math.sqrt(6 * length / 32) + 8) + 1e-38
            d = (got.double() - want).abs()
            assert bool((d <= tol).all()), float((d / tol).max())
