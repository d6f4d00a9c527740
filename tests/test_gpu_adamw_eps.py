"""The AdamW step (GPU) where v lies near and below float32's smallest normal
number and eps is far below sqrt(v): the formula's step is about lr there, and a
root that takes such a v for zero would make it m / eps.

Tolerances.  An operation rounds by 2^-24 of its result or, below the normal
numbers, by half the distance of subnormal ones, 2^-150.  v: v b2, g g, (g g) c2
(and, from 8-bit states, s s), whose sum is exact where it is subnormal, and the
roundings of b2 and c2: 6 2^-24 v + 4 2^-150.  m: m b1 and g c1 with their
constants, and the sum: 4 2^-24 of the terms + 2 2^-150.  The step is monotonic in
m and v, so it lies between its values at the ends of those intervals, but for
the quotient's own roundings, below 2^-20 of it; X takes its own twice."""
import pytest

from .gpuhelp import say
from .test_gpu_adamw import spread, state8, tensor, unit

pytestmark = pytest.mark.gpu

LR, B1, B2 = 1e-2, 0.9, 0.95
U, SUB = 2.0 ** -24, 2.0 ** -150


def ends(G, m, v, step, eps):
    """Largest and smallest step of X in float64."""
    import torch
    g = G.double()
    m1, v1 = B1 * m + (1 - B1) * g, B2 * v + (1 - B2) * g * g
    em, ev = 4 * U * (B1 * m.abs() + (1 - B1) * g.abs()) + 2 * SUB, 6 * U * v1 + 4 * SUB
    us = []
    for a in (m1 - em, m1 + em):
        for b in ((v1 - ev).clamp(min=0), v1 + ev):
            us.append(LR / (1 - B1 ** step) * a / ((b / (1 - B2 ** step)).sqrt() + eps))
    us = torch.stack(us)
    slack = us.abs().amax(0) * 2.0 ** -20
    return us.amin(0) - slack, us.amax(0) + slack


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("eps", [1e-16, 1e-24, 1.2e-38])
@pytest.mark.parametrize("scale", [1e-16, 1e-18, 1e-19, 1e-20, 3e-22, 1e-30])
def test_steps(gpu_lib, bits, gdt, eps, scale):
    import torch
    say(f"adamw eps {eps} gradients {scale} {gdt} {bits}")
    n = 5003
    X, G = torch.zeros(n, device="cuda"), tensor(n, 1, getattr(torch, gdt), scale)
    st = (tensor(n, 2).zero_(), tensor(n, 3).zero_()) if bits == 32 else state8(n, 2, zero=True)
    for step in (1, 2, 3):
        x0, old = X.clone(), [t.clone() for t in st]
        gpu_lib.adamw_step_batched([(X, G) + tuple(st)], LR, step, betas=(B1, B2), eps=eps, seed=step)
        m, v = old[0].double(), old[1].double()
        if bits == 8:
            s, nb = old[2].view(torch.uint8), -(-n // 64)
            m, v = m * spread(unit(s[:nb]), n), (v * spread(unit(s[nb:]), n)).square()
        lo, hi = ends(G, m, v, step, eps)
        got = x0.double() - X.double()
        err = 4 * U * (x0.double().abs() + X.double().abs())
        ok = (got >= lo - err) & (got <= hi + err)
        assert bool(ok.all()), (int((~ok).sum()), got[~ok][:4], lo[~ok][:4], hi[~ok][:4])


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_is_lr(gpu_lib, bits):
    """m / (1 - b1) = g and v / (1 - b2) = g^2 after the first step, so X moves by
    lr whatever the gradient's magnitude is: within 2^-8 as long as v keeps eight
    bits (0.05 g^2 >= 2^-141)."""
    import torch
    G = torch.tensor([1e-18, -1e-19, 3e-20, -1e-20], device="cuda").repeat(32)
    X = torch.zeros(128, device="cuda")
    st = (torch.zeros_like(X), torch.zeros_like(X)) if bits == 32 else gpu_lib.adamw_state8(X)
    gpu_lib.adamw_step_batched([(X, G) + tuple(st)], LR, 1, betas=(B1, B2), eps=1e-25)
    assert bool(((X + LR * G.sign()).abs() <= LR * 2.0 ** -8).all()), X[:4]
