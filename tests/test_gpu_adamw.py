"""The AdamW step (GPU) against its formulas in float64, element by element.

float32 states: m, v carry at most four roundings of 2^-24 each of the terms'
magnitudes; X carries two of its own size and, in the step, the roundings of
m, v and the quotient (below 2^-20 of the step).  8-bit states: a code is what
the rounding rule gives for some value within the float32 computation's error
of the exact one; the rule is monotonic, so the code lies between the rule's
results at the ends of that interval."""
import math

import pytest

from .gpuhelp import say

pytestmark = pytest.mark.gpu

LR, B1, B2, EPS = 1e-2, 0.9, 0.95, 1e-8
U = 2.0 ** -24


def gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def tensor(n, seed, dtype=None, scale=1.0, shift=0):
    """n seeded normal values `shift` elements into an allocation, NaN around."""
    import torch
    dtype = dtype or torch.float32
    big = torch.full((n + shift + 9,), float("nan"), dtype=dtype, device="cuda")
    big[shift:shift + n] = (torch.randn(n, generator=gen(seed), device="cuda") * scale).to(dtype)
    return big[shift:shift + n]


def state8(n, seed, shift=0, zero=False):
    import torch
    nb = -(-n // 64)
    out = []
    for k in range(2):
        big = torch.full((n + shift + 9,), 0x7f, dtype=torch.uint8, device="cuda")
        v = torch.randn(n, generator=gen(seed + k), device="cuda") * 60
        v = (v if k == 0 else v.abs() + 1).clamp(-250, 250)
        big[shift:shift + n] = 0 if zero else v.to(torch.float8_e4m3fn).view(torch.uint8)
        out.append(big[shift:shift + n].view(torch.float8_e4m3fn))
    s = torch.randint(100, 118, (2 * nb,), generator=gen(seed + 2), device="cuda").to(torch.uint8)
    if zero:
        s.zero_()
    return out[0], out[1], s.view(torch.float8_e8m0fnu)


def unit(b):
    import torch
    return torch.exp2(b.double() - 127.0)


def spread(s, n):
    """Scales of n elements' blocks."""
    return s.repeat_interleave(64)[:n]


def rule(a, u, least):
    """floor(a / ulp + u) ulp in float64."""
    import torch
    e = (torch.frexp(a)[1] - 1).clamp(min=-6)
    ulp = torch.exp2(e.double() - 3)
    q = torch.floor(a / ulp + u)
    if least:
        q = q.clamp(min=1)
    return torch.where(a > 0, q * ulp, 0.0)


def dither(n, seed):
    import torch
    mask = 0xffffffff
    h = ((torch.arange(n, device="cuda") + 0x632be5ab * seed) & mask) * 0x9e3779b1 & mask
    h = (h ^ (h >> 15)) * 0x85ebca77 & mask
    h = h ^ (h >> 13)
    return (h & 0xffff).double() / 65536, (h >> 16).double() / 65536


def check_codes(code, byte, x, err, u, least):
    """code, byte: the state after the step; x (float64, >= 0 in magnitude of
    sign x) within err."""
    import torch
    n = x.numel()
    nb = -(-n // 64)
    pad = torch.zeros(nb * 64, dtype=torch.float64, device="cuda")
    pad[:n] = x.abs()
    top = pad.view(nb, 64).amax(1)
    def of(t):
        e = torch.frexp(t)[1].double() - 1 + 127
        return torch.where(t >= 2.0 ** -126, e - 7, 0.0).clamp(min=1)
    b = byte.double()
    assert bool(((b >= of(top * (1 - 2.0 ** -20))) & (b <= of(top * (1 + 2.0 ** -20)))).all())
    inv = 1.0 / spread(unit(b), n)
    a, d = x.abs() * inv, err * inv + 2.0 ** -18 * (x.abs() * inv).clamp(min=2.0 ** -6)
    lo, hi = rule((a - d).clamp(min=0), u, least), rule(a + d, u, least)
    got = code.double().abs()
    ok = (got >= lo) & (got <= hi)
    assert bool(ok.all()), (a[~ok][:5], got[~ok][:5], lo[~ok][:5], hi[~ok][:5])
    sure = (x.abs() > err) & (got > 0)
    assert bool((torch.sign(code.double())[sure] == torch.sign(x)[sure]).all())


def expect(X, G, m, v, lr, step, b1, b2, eps, wd, c):
    g = G.double() * c
    m1 = b1 * m + (1 - b1) * g
    v1 = b2 * v + (1 - b2) * g * g
    em = 4 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    ev = 6 * U * v1
    u = lr * (m1 / (1 - b1 ** step)) / ((v1 / (1 - b2 ** step)).sqrt() + eps)
    eu = u.abs() * 2.0 ** -20 + lr * (em / (1 - b1 ** step)) / ((v1 / (1 - b2 ** step)).sqrt() + eps)
    x = (1 - lr * wd) * X.double() - u
    ex = 4 * U * (X.double().abs() + u.abs()) + eu + 1e-37
    return x, ex, m1, em + 1e-44, v1, ev + 1e-44


def within(got, want, err):
    d = (got.double() - want).abs()
    assert bool((d <= err).all()), float((d / err.clamp(min=1e-300)).max())


def run(lib, sizes, gdt, bits, steps=2, shift=0, wd=0.1, c=None, seed=3, b1=B1, b2=B2, zero=False, scale=1e-3):
    import torch
    gdt = getattr(torch, gdt)
    entries, olds = [], []
    for k, n in enumerate(sizes):
        X = tensor(n, 10 * k, None, 0.02, shift)
        G = tensor(n, 10 * k + 1, gdt, scale, shift)
        if bits == 32:
            M, V = tensor(n, 10 * k + 2, None, 1e-3, shift), tensor(n, 10 * k + 3, None, 1e-3, shift).square_()
            if zero:
                M.zero_(), V.zero_()
            entries.append((X, G, M, V))
        else:
            entries.append((X, G) + state8(n, 10 * k + 2, shift, zero))
    decays = [wd * (k % 2) for k in range(len(sizes))]
    cs = 1.0 if c is None else float(c)
    for step in range(1, steps + 1):
        olds = [[t.clone() for t in e] for e in entries]
        lib.adamw_step_batched(entries, LR, step, betas=(b1, b2), eps=EPS, weight_decay=decays, grad_scale=c, seed=seed + step)
        for e, old, w in zip(entries, olds, decays):
            n = e[0].numel()
            if n == 0:
                continue
            assert torch.equal(e[1], old[1])
            X, G = old[0], old[1]
            if bits == 32:
                x, ex, m, em, v, ev = expect(X, G, old[2].double(), old[3].double(), LR, step, b1, b2, EPS, w, cs)
                within(e[2], m, em)
                within(e[3], v, ev)
            else:
                nb = -(-n // 64)
                s0, s1 = old[4].view(torch.uint8), e[4].view(torch.uint8)
                m0 = old[2].double() * spread(unit(s0[:nb]), n)
                r0 = old[3].double() * spread(unit(s0[nb:]), n)
                x, ex, m, em, v, ev = expect(X, G, m0, r0 * r0, LR, step, b1, b2, EPS, w, cs)
                um, uv = dither(n, seed + step)
                check_codes(e[2], s1[:nb], m, em, um, 0)
                check_codes(e[3], s1[nb:], v.sqrt(), 4 * U * v.sqrt() + 1e-30, uv, 1)
            within(e[0], x, ex)
    return entries


SIZES = [1, 2, 3, 4, 5, 63, 64, 65, 255, 1000, 1023, 1024, 1025, 4095, 4097, 100003]


@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_sizes(gpu_lib, gdt, bits):
    for n in SIZES:
        say(f"adamw {n} {gdt} {bits}")
        run(gpu_lib, [n], gdt, bits)


@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [1, 2, 3, 4, 8])
def test_lists_and_alignment(gpu_lib, gdt, bits, shift):
    """Several launches' worth of tensors, empty ones among them, at every
    alignment; what lies around them is NaN."""
    say(f"adamw list {gdt} {bits} shift {shift}")
    run(gpu_lib, [0, 77, 1, 0, 4096, 513], gdt, bits, shift=shift)
    run(gpu_lib, [(37 * k) % 300 for k in range(131)], gdt, bits, steps=1, shift=shift)


@pytest.mark.parametrize("bits", [32, 8])
def test_large_launches(gpu_lib, bits):
    """Several workgroups per tensor; past 256 MiB the accesses go past the
    caches, in other pieces."""
    say(f"adamw large {bits}")
    run(gpu_lib, [1 << 20, 70001, 64, 1 << 18], "bfloat16", bits)
    run(gpu_lib, [3000017], "float32", bits, shift=1, steps=1)
    run(gpu_lib, [9000001, 77, 12000003, 1025], "bfloat16", bits, steps=1)
    run(gpu_lib, [20000001, 2], "float32", bits, shift=2, steps=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_arguments(gpu_lib, bits):
    import torch
    c = torch.tensor([0.37], device="cuda")
    run(gpu_lib, [500, 2049], "bfloat16", bits, c=c)
    run(gpu_lib, [500, 2049], "float32", bits, b1=0.0, b2=0.0)
    run(gpu_lib, [500], "float32", bits, b1=0.99999, b2=0.9999999, zero=True, steps=3)
    run(gpu_lib, [500, 64], "float32", bits, zero=True, steps=3)
    run(gpu_lib, [500, 64], "float32", bits, scale=0.0, steps=2)
    run(gpu_lib, [700], "float32", bits, seed=(1 << 32) - 2)
    e = run(gpu_lib, [300], "float32", bits, zero=True, scale=0.0, steps=2)[0]
    assert not bool(e[2].float().any()) and not bool(e[3].float().any())


def test_state8_begins_at_zero(gpu_lib):
    import torch
    X = torch.randn(7, 33, device="cuda")
    M, V, S = gpu_lib.adamw_state8(X)
    assert M.shape == X.shape and S.numel() == 8
    G = torch.randn(7, 33, device="cuda")
    before = X.clone()
    gpu_lib.adamw_step(X, G, M, V, 0.1, 1, S=S)
    # the first step moves every element by lr in its gradient's direction
    assert torch.allclose(before - X, 0.1 * G.sign(), rtol=1e-4, atol=1e-6)


@pytest.mark.parametrize("bits", [32, 8])
def test_scale_that_is_not_finite_skips_the_step(gpu_lib, bits):
    import torch
    for value in (math.inf, -math.inf, math.nan):
        X, G = tensor(5000, 1), tensor(5000, 2)
        st = state8(5000, 3) if bits == 8 else (tensor(5000, 3), tensor(5000, 4).abs())
        old = [t.clone() for t in (X, *st)]
        gpu_lib.adamw_step_batched([(X, G) + tuple(st)], LR, 5, grad_scale=torch.tensor([value], device="cuda"))
        for a, b in zip((X, *st), old):
            assert torch.equal(a.view(torch.uint8) if a.dtype not in (torch.float32,) else a,
                               b.view(torch.uint8) if b.dtype not in (torch.float32,) else b)


def test_not_finite_elements(gpu_lib):
    """float32: the element alone; 8 bits: the block from the next step on."""
    import torch
    for bits in (32, 8):
        n = 64 * 40 + 5
        X, G = tensor(n, 1), tensor(n, 2, None, 1e-3)
        G[100], G[700], G[n - 1] = math.nan, math.inf, -math.inf
        st = (tensor(n, 3, None, 1e-3), tensor(n, 4, None, 1e-3).square_()) if bits == 32 else state8(n, 5)
        gpu_lib.adamw_step_batched([(X, G) + tuple(st)], LR, 1)
        bad = torch.zeros(n, dtype=torch.bool, device="cuda")
        bad[[100, 700, n - 1]] = True
        assert torch.equal(~torch.isfinite(X), bad)
        G.zero_()
        if bits == 8:
            for b in (1, 10, 40):
                bad[64 * b:64 * (b + 1)] = True
        gpu_lib.adamw_step_batched([(X, G) + tuple(st)], LR, 2)
        assert torch.equal(~torch.isfinite(X), bad)


def test_ends_of_the_range(gpu_lib):
    """Gradients whose squares are near float32's ends."""
    import torch
    for scale in (1e-18, 1e-12, 1e10, 1e18):
        for bits in (32, 8):
            say(f"adamw range {scale} {bits}")
            run(gpu_lib, [1000], "float32", bits, zero=True, scale=scale, steps=2)


def test_8bit_states_have_the_right_mean(gpu_lib):
    """With one constant gradient in many elements, m and sqrt(v) follow their
    float64 recursions in the mean though a step changes v by far less than
    half a code: after T steps the mean over N elements is off by less than
    five standard errors (each rounding is below an eighth of the value, and
    the decays leave at most 1 / (1 - beta) of them: a spread below 0.125
    sqrt(1 / (1 - beta^2)) of a value) plus sqrt(v)'s own bias, the mean of a
    root against the root of a mean: half its relative variance."""
    import torch
    n, T, b1, b2 = 1 << 16, 300, 0.9, 0.999
    X, G = torch.zeros(n, device="cuda"), torch.full((n,), 1e-3, device="cuda")
    M, V, S = gpu_lib.adamw_state8(X)
    plan = gpu_lib.AdamWPlan([(X, G, M, V, S)])
    for t in range(1, T + 1):
        plan.step(0.0, t, betas=(b1, b2))
    nb = n // 64
    s = S.view(torch.uint8)
    m = M.double() * spread(unit(s[:nb]), n)
    v = (V.double() * spread(unit(s[nb:]), n)).square()
    wm, wv = 1e-3 * (1 - b1 ** T), 1e-6 * (1 - b2 ** T)
    sm = 0.125 * (1 / (1 - b1 * b1)) ** 0.5
    assert abs(float(m.mean()) / wm - 1) <= 5 * sm / n ** 0.5
    # a step's rounding of sqrt(v) has a variance of at most (1/16)^2 of it,
    # (1/8)^2 / 4, and v's mean rises by that variance per step
    rise = sum(b2 ** (T - t) * (1 / 16) ** 2 * (1 - b2 ** t) for t in range(1, T + 1)) / (1 - b2 ** T)
    assert -0.02 <= float(v.mean()) / wv - 1 <= rise + 0.02


def test_same_bits_streams_and_graphs(gpu_lib):
    import torch
    def make():
        return [(tensor(n, n), tensor(n, n + 1, torch.bfloat16, 1e-3)) + state8(n, n + 2) for n in (5000, 70, 200001)]
    a, b, c = make(), make(), make()
    scale = torch.tensor([0.5], device="cuda")
    pa = gpu_lib.AdamWPlan(a, weight_decay=[0.1, 0.0, 0.2])
    for t in (1, 2, 3):
        pa.step(LR, t, grad_scale=scale, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for t in (1, 2, 3):
        gpu_lib.adamw_step_batched(b, LR, t, weight_decay=[0.1, 0.0, 0.2], grad_scale=scale, seed=9, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    pc = gpu_lib.AdamWPlan(c, weight_decay=[0.1, 0.0, 0.2])
    with torch.cuda.graph(graph):
        for t in (1, 2, 3):
            pc.step(LR, t, grad_scale=scale, seed=9)
    graph.replay()
    torch.cuda.synchronize()
    for x, y, z in zip(a, b, c):
        for p, q, r in zip(x, y, z):
            if p.dtype.itemsize == 1:
                p, q, r = (t.view(torch.uint8) for t in (p, q, r))
            assert torch.equal(p, q) and torch.equal(p, r)
    # the scale is read when the graph runs
    scale.fill_(math.nan)
    keep = [t.clone() for t in c[0][:1]]
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(keep[0], c[0][0])


def test_offsets_past_32_bits(gpu_lib):
    """More than 2^31 bytes of float32 before the checked elements, and an
    index past 2^31 elements of 8-bit states."""
    import torch
    n = (1 << 31) + 4099
    X = torch.zeros(n, device="cuda")
    G = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    M, V, S = gpu_lib.adamw_state8(X)
    tail = n - 3001
    G[tail:] = tensor(3001, 7, torch.bfloat16, 1e-3)
    G[:100] = 1.0
    gpu_lib.adamw_step_batched([(X, G, M, V, S)], LR, 1, eps=EPS)
    g = G[tail:].double()      # the first step: m / (1 - b1) = g, v / (1 - b2) = g^2
    assert torch.allclose(X[tail:].double(), -LR * g / (g.abs() + EPS), rtol=1e-3, atol=1e-6)
    assert bool((X[:100] < 0).all()) and not bool(X[100:tail].any())
    assert bool((V[tail:].float() > 0).eq(G[tail:] != 0).all()) and not bool(V[100:tail].view(torch.uint8).any())


def test_binding_refuses(gpu_lib):
    import torch
    X, G = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    M, V, S = gpu_lib.adamw_state8(X)
    f = torch.zeros(64, device="cuda")
    for bad in ([(X, G, f, f[:32])], [(X, G, f, f.clone()), (X, G, M, V, S)], [(X, G, M, V, S[:1])],
                [(X[::2], G[:32], f[:32], f[:32])], [(X, G, f, f.cpu())], [(X, G, f, f)], [(X, X, f, f.clone())]):
        with pytest.raises((ValueError, gpu_lib.DionError)):
            gpu_lib.adamw_step_batched(bad, LR, 1)
    for bad in ([(X, G.half(), f, f)], [(X, G, M, f, S)], [(X, G, f.half(), f)], [(X.half(), G, f, f)],
                [(X, G, M, V, S.view(torch.uint8))]):
        with pytest.raises(TypeError):
            gpu_lib.adamw_step_batched(bad, LR, 1)
    for kw in (dict(grad_scale=f), dict(grad_scale=torch.ones(1)), dict(grad_scale=torch.ones(1, device="cuda").half())):
        with pytest.raises(ValueError):
            gpu_lib.adamw_step(X, G, f, f.clone(), LR, 1, **kw)
    for kw in (dict(lr=math.nan, step=1), dict(lr=LR, step=0), dict(lr=LR, step=1, betas=(1.0, 0.9)), dict(lr=LR, step=1, eps=0.0)):
        with pytest.raises(gpu_lib.DionError):
            gpu_lib.adamw_step(X, G, f, f.clone(), **kw)
