"""Training steps of a linear layer under an output head (GPU), the operators
together: linear forward, cross entropy forward and backward, linear backward,
Muon for the layer's matrix, AdamW for its bias (float32 states) and for the
head (8-bit states).

Gradients against the float64 formulas of the whole chain.  Each rounding to
bfloat16 (h, dz, dh, the outputs) is off by at most half a step, 2^-8 of the
value, and moves what follows by its product with the magnitudes there; the
float32 sums, their inputs' order aside, add at most 2^-18 of the terms'
magnitudes (reductions of at most 500)."""
import math

import pytest

from .gpuhelp import say

pytestmark = pytest.mark.gpu

T, K, H, N = 300, 96, 200, 500
IGNORE, SMOOTHING, Z_LOSS = -100, 0.1, 1e-3
HALF, SUMS = 2.0 ** -8, 2.0 ** -18


class Model:
    def __init__(self, lib):
        import torch
        gen = torch.Generator(device="cuda").manual_seed(5)
        self.lib = lib
        self.w = torch.randn(H, K, generator=gen, device="cuda") * K ** -0.5
        self.b = torch.randn(H, generator=gen, device="cuda") * 0.1
        self.head = torch.randn(N, H, generator=gen, device="cuda") * H ** -0.5
        self.x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
        self.y = torch.randint(0, N, (T,), generator=gen, device="cuda")
        self.y[::7] = IGNORE
        self.dloss = (self.y != IGNORE).float() / int((self.y != IGNORE).sum())
        self.momentum = torch.zeros_like(self.w)
        self.db, self.dw, self.dhead = (torch.empty_like(self.b), torch.empty(H, K, dtype=torch.bfloat16, device="cuda"),
                                        torch.empty(N, H, dtype=torch.bfloat16, device="cuda"))
        self.state_b = (torch.zeros_like(self.b), torch.zeros_like(self.b))
        self.state_head = lib.adamw_state8(self.head)
        self.plan_b = lib.AdamWPlan([(self.b, self.db) + self.state_b])
        self.plan_head = lib.AdamWPlan([(self.head, self.dhead) + self.state_head], weight_decay=0.1)
        self.wb, self.hb = torch.empty_like(self.dw), torch.empty_like(self.dhead)
        self.h, self.dh = (torch.empty(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.loss, self.lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")

    def gradients(self):
        lib, head = self.lib, dict(label_smoothing=SMOOTHING, z_loss=Z_LOSS, ignore_index=IGNORE)
        self.wb.copy_(self.w)
        self.hb.copy_(self.head)
        lib.linear_forward(self.x, self.wb, self.h, bias=self.b)
        lib.cross_entropy_forward(self.h, self.hb, self.y, self.loss, lse=self.lse, **head)
        lib.cross_entropy_backward(self.dloss, self.h, self.hb, self.y, self.lse, dx=self.dh, dw=self.dhead, **head)
        lib.linear_backward(self.dh, self.x, dw=self.dw, db=self.db)

    def update(self, step, scale=None):
        self.plan_b.step(1e-2, step, grad_scale=scale)
        self.plan_head.step(1e-2, step, grad_scale=scale)

    def matrix_update(self):
        ws = self.lib.muon_step(self.w, self.dw, self.momentum, lr=0.02, momentum=0.9, math="f16")
        self.lib.check_status(ws, 1)

    def state(self):
        import torch
        return [t.view(torch.uint8) if t.element_size() == 1 else t
                for t in (self.w, self.b, self.head, self.momentum) + self.state_b + self.state_head]


def check_gradients(m):
    import torch
    def mm(a, b):
        return torch.mm(a, b.contiguous())
    x, w, b, head = m.x.double(), m.wb.double(), m.b.double(), m.hb.double()
    h = mm(x, w.t()) + b
    eh = h.abs() * HALF + SUMS * (mm(x.abs(), w.abs().t()) + b.abs())
    z = mm(h, head.t())
    ez = mm(eh, head.abs().t()) * (1 + HALF) + SUMS * mm(h.abs(), head.abs().t())
    lse = torch.logsumexp(z, 1)
    worst = ez.max(1).values
    keep = m.y != IGNORE
    at = m.y.clamp(min=0)[:, None]
    loss = torch.where(keep, lse - (1 - SMOOTHING) * z.gather(1, at)[:, 0] - SMOOTHING * z.mean(1) + Z_LOSS * lse ** 2, 0.0)
    assert bool(((m.lse.double() - lse).abs() <= worst + SUMS * (1 + lse.abs())).all())
    assert bool(((m.loss.double() - loss).abs() <= 2 * worst + SUMS * (1 + loss.abs() + lse.abs()) +
                 Z_LOSS * (2 * lse.abs() + worst) * worst).all())
    d = m.dloss.double()[:, None]
    slope = 1 + 2 * Z_LOSS * lse[:, None]
    p = torch.exp(z - lse[:, None])
    dz = d * (slope * p - SMOOTHING / N)
    dz.scatter_add_(1, at, -(1 - SMOOTHING) * d)
    # exp's argument is off by an element's and by lse's error, the slope by lse's
    move = ez + worst[:, None]
    edz = d * (p * (slope * torch.expm1(move + SUMS) + 2 * Z_LOSS * worst[:, None] * torch.exp(move))) + \
        HALF * 1.1 * dz.abs() + SUMS * d * (slope * p + SMOOTHING / N)
    edz.scatter_add_(1, at, SUMS * d)

    def near(name, got, want, error, terms):
        tol = error + SUMS * terms + (HALF * (want.abs() + error) if got.dtype == torch.bfloat16 else 0.0) + 1e-30
        diff = (got.double() - want).abs()
        assert bool((diff <= tol).all()), (name, float((diff / tol).max()))
        return tol
    dh, dhead = mm(dz, head), mm(dz.t(), h)
    edh = near("dh", m.dh, dh, mm(edz, head.abs()), mm(dz.abs(), head.abs()))
    near("dhead", m.dhead, dhead, mm(edz.t(), h.abs() + eh) + mm(dz.abs().t(), eh), mm(dz.abs().t(), h.abs()))
    near("dw", m.dw, mm(dh.t(), x), mm(edh.t(), x.abs()), mm(dh.abs().t(), x.abs()))
    near("db", m.db, dh.sum(0), edh.sum(0), dh.abs().sum(0))


def check_update(x0, g, m0, v0, x, step, decay):
    """m0, v0: float64 moments before the step."""
    g = g.double()
    m, v = 0.9 * m0 + 0.1 * g, 0.999 * v0 + 0.001 * g * g
    move = 1e-2 / (1 - 0.9 ** step) * m / (v.sqrt() / math.sqrt(1 - 0.999 ** step) + 1e-8)
    want = x0 * (1 - 1e-2 * decay) - move
    # a few float32 roundings of each term; m's terms may cancel
    size = 1e-2 / (1 - 0.9 ** step) * (0.9 * m0.abs() + 0.1 * g.abs()) / (v.sqrt() / math.sqrt(1 - 0.999 ** step) + 1e-8)
    assert bool(((x.double() - want).abs() <= 2.0 ** -22 * (want.abs() + x0.abs()) + 2.0 ** -20 * size).all())
    return m, v


def test_training_steps(gpu_lib):
    import torch
    say("training steps of a layer and a head")
    m = Model(gpu_lib)
    mb, vb = (t.double() for t in m.state_b)
    for step in range(1, 5):
        m.gradients()
        check_gradients(m)
        b0, h0 = m.b.double().clone(), m.head.double().clone()
        scales = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), m.state_head[2].view(torch.uint8).int() - 127)
        def moment(codes, s):
            return (codes.double().reshape(-1) * s.repeat_interleave(64)[:codes.numel()]).reshape(codes.shape)
        half = scales.numel() // 2
        mh, vh = moment(m.state_head[0], scales[:half]), moment(m.state_head[1], scales[half:]) ** 2
        m.update(step)
        mb, vb = check_update(b0, m.db, mb, vb, m.b, step, 0.0)
        # float32 states of the steps before carry their own roundings
        mb, vb = (t.double() for t in m.state_b)
        check_update(h0, m.dhead, mh, vh, m.head, step, 0.1)
        before = m.w.clone()
        m.matrix_update()
        assert not torch.equal(m.w, before) and bool(torch.isfinite(m.w).all())
    # the same steps on a side stream: the same bits
    other, side = Model(gpu_lib), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for step in range(1, 5):
            other.gradients()
            other.update(step)
            other.matrix_update()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b in zip(m.state(), other.state()):
        assert torch.equal(a, b)


def test_training_step_captured(gpu_lib):
    """Gradients and AdamW of one step as a graph, replayed from changing states
    with eager work between: the eager call's bits each time."""
    import torch
    say("captured training step")
    m, scale = Model(gpu_lib), torch.ones(1, device="cuda")
    m.gradients()
    m.update(3, scale)
    start = [t.clone() for t in m.state()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.gradients()
        m.update(3, scale)
    for replay in range(4):
        scale.fill_(float("inf") if replay == 2 else 1.0 / (1 + replay))
        for t, s in zip(m.state(), start):
            t.copy_(s)
        m.w.mul_(1.0 - 0.1 * replay)
        at = [t.clone() for t in m.state()]
        graph.replay()
        got = [t.clone() for t in m.state()] + [m.loss.clone(), m.dw.clone()]
        torch.cuda.synchronize()
        for t, s in zip(m.state(), at):
            t.copy_(s)
        m.gradients()
        m.update(3, scale)
        for a, b in zip(got, m.state() + [m.loss, m.dw]):
            assert torch.equal(a, b), replay
        if replay == 2:   # a scale that is not finite leaves parameters and states
            for a, b in zip(m.state(), at):
                assert torch.equal(a, b)
