"""Newton-Schulz orthogonalization and the Muon step (GPU) against the same
formulas in float64.

Tolerances (relative Frobenius error), from the arithmetic:

* math="f32": every factor carries 22 bits or more and every sum is float32.
  Five quintic iterations multiply the relative size of an early rounding by
  the ratio of the polynomial's slopes, at most a few tens (small p, where
  the errors of few singular values do not average, is the worst), so 32 *
  2^-22 = 7.6e-6 in a float32 output, plus bfloat16's 2^-9 in a bfloat16 one.
* math="f16": factors of 11 bits: 32 * 2^-12 / sqrt(12) = 2.3e-3 of
  independent roundings, doubled for spectra that are not flat; plus 2^-9
  in a bfloat16 output.
"""
import numpy as np
import pytest

from .gpuhelp import say

pytestmark = pytest.mark.gpu

Q = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
TOL32, TOL16, TOL_BF = 32 * 2.0 ** -22, 4.6e-3, 2.0 ** -9


def f32(x):
    return float(np.float32(x))


def ns64(G, coeffs):
    """Definition in float64 (any order of the sides)."""
    import torch
    norm = torch.linalg.vector_norm(G)
    X = G / norm if float(norm) > 0 else G.clone()
    for a, b, c in coeffs:
        a, b, c = f32(a), f32(b), f32(c)
        if G.shape[0] <= G.shape[1]:
            A = X @ X.T
            X = a * X + b * (A @ X) + c * (A @ (A @ X))
        else:
            A = X.T @ X
            X = a * X + b * (X @ A) + c * ((X @ A) @ A)
    return X


def rel(x, y):
    import torch
    n = float(torch.linalg.vector_norm(y))
    d = float(torch.linalg.vector_norm(x.double() - y))
    return d / n if n else d


def draw(m, n, seed, dtype, kind="normal"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(m, n, generator=g, device="cuda")
    if kind == "planted":
        k = min(8, m, n)
        a = torch.randn(m, k, generator=g, device="cuda") / m ** 0.5
        b = torch.randn(k, n, generator=g, device="cuda") / n ** 0.5
        z = z * 1e-3 + (a / torch.arange(1, k + 1, device="cuda")) @ b
    return z.to(dtype)


SHAPES = [(1, 1), (1, 7), (7, 1), (3, 2), (2, 300), (5, 732), (63, 65), (64, 64), (65, 63),
          (128, 256), (256, 128), (129, 257), (130, 1000), (385, 129), (600, 520), (1031, 773)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
def test_float32_accuracy(gpu_lib, m, n, gdt):
    import torch
    say(f"ns f32 {m}x{n} {gdt}")
    G = draw(m, n, 100 + m + n, getattr(torch, gdt))
    O = torch.full((m, n), float("nan"), device="cuda")
    ws = gpu_lib.orthogonalize(G, O, Q, 5, "f32")
    gpu_lib.check_status(ws, 1)
    assert rel(O, ns64(G.double(), [Q] * 5)) <= TOL32
    Ob = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gpu_lib.orthogonalize(G, Ob, Q, 5, "f32")
    assert torch.equal(Ob, O.bfloat16())   # one rounding of the same values


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("kind", ["normal", "planted"])
def test_float16_products(gpu_lib, m, n, kind):
    import torch
    say(f"ns f16 {m}x{n} {kind}")
    G = draw(m, n, 200 + m + n, torch.bfloat16, kind)
    O = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    ws = gpu_lib.orthogonalize(G, O, Q, 5, "f16")
    gpu_lib.check_status(ws, 1)
    assert rel(O, ns64(G.double(), [Q] * 5)) <= TOL16 + TOL_BF


def test_cubic_converges_to_the_polar_factor(gpu_lib):
    import torch
    for m, n in ((96, 200), (200, 96)):
        g = torch.Generator(device="cuda").manual_seed(m)
        u = torch.linalg.qr(torch.randn(m, 96, generator=g, device="cuda", dtype=torch.float64))[0]
        v = torch.linalg.qr(torch.randn(n, 96, generator=g, device="cuda", dtype=torch.float64))[0]
        s = torch.linspace(0.5, 1.0, 96, device="cuda", dtype=torch.float64)
        G = ((u * s) @ v.T).float()
        O = torch.empty(m, n, device="cuda")
        gpu_lib.orthogonalize(G, O, CUBIC, 16, "f32")
        assert rel(O, u @ v.T) <= 1e-5       # converged: O is the polar factor


def test_coefficients_per_iteration(gpu_lib):
    import torch
    cs = [(3.0, -3.2, 1.2), (2.0, -1.5, 0.5), CUBIC]
    G = draw(190, 140, 5, torch.float32)
    O = torch.empty_like(G)
    gpu_lib.orthogonalize(G, O, cs, 3, "f32")
    assert rel(O, ns64(G.double(), cs)) <= TOL32
    gpu_lib.orthogonalize(G, O, Q, 1, "f32")
    assert rel(O, ns64(G.double(), [Q])) <= TOL32


@pytest.mark.parametrize("scale", [1e-30, 1e-12, 1e12, 1e30])
def test_scale_of_the_input_does_not_matter(gpu_lib, scale):
    import torch
    G = draw(150, 333, 6, torch.float32)
    O, P = torch.empty_like(G), torch.empty_like(G)
    gpu_lib.orthogonalize(G, O)
    gpu_lib.orthogonalize(G * scale, P)
    assert rel(P, ns64((G * scale).double(), [Q] * 5)) <= TOL32
    assert rel(P, O.double()) <= TOL32


def test_zero_and_non_finite(gpu_lib):
    import torch
    shapes = [(70, 40), (40, 70), (70, 40), (70, 40), (300, 200)]
    Gs = [draw(m, n, 7 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    Gs[0].zero_()
    Gs[2][69, 39] = float("inf")
    Gs[3][0, 0] = float("nan")
    Os = [torch.full(s, 3.0, device="cuda") for s in shapes]
    ws = gpu_lib.orthogonalize_batched(list(zip(Gs, Os)))
    code, per = gpu_lib.status(ws, len(shapes))
    bad = gpu_lib.STATUS_NONFINITE
    assert code == gpu_lib.ERR_BREAKDOWN and per == [0, 0, bad, bad, 0]
    assert torch.count_nonzero(Os[0]) == 0
    for i in (2, 3):
        assert torch.equal(Os[i], torch.full_like(Os[i], 3.0))
    for i in (1, 4):
        assert rel(Os[i], ns64(Gs[i].double(), [Q] * 5)) <= TOL32
    # the workspace holds nothing of the failed call
    Gs[2][69, 39] = 0.5
    Gs[3][0, 0] = 0.5
    ws = gpu_lib.orthogonalize_batched(list(zip(Gs, Os)), workspace=ws)
    gpu_lib.check_status(ws, len(shapes))
    for i in (1, 2, 3, 4):
        assert rel(Os[i], ns64(Gs[i].double(), [Q] * 5)) <= TOL32


@pytest.mark.parametrize("mode", ["f32", "f16"])
def test_list_equals_single_calls_and_repeats(gpu_lib, mode):
    """A list of eleven shapes (more than one launch holds) gives the bits of
    single calls, twice."""
    import torch
    shapes = [(40 + 13 * i, 300 - 21 * i) for i in range(10)] + [(520, 260), (40, 300)]
    Gs = [draw(m, n, 30 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    Os = [torch.empty_like(g) for g in Gs]
    gpu_lib.orthogonalize_batched(list(zip(Gs, Os)), math=mode)
    for G, O in zip(Gs, Os):
        P = torch.empty_like(G)
        gpu_lib.orthogonalize(G, P, math=mode)
        assert torch.equal(O, P)
    Rs = [torch.empty_like(g) for g in Gs]
    gpu_lib.orthogonalize_batched(list(zip(Gs, Rs)), math=mode)
    assert all(torch.equal(a, b) for a, b in zip(Os, Rs))


@pytest.mark.parametrize("m,n", [(130, 200), (200, 130), (1, 9), (300, 77)])
def test_row_pitches(gpu_lib, m, n):
    """Pitches that are odd, and outputs between rows that stay untouched."""
    import torch
    for extra in (1, 5, 8):
        big = draw(m, n + extra, 9, torch.bfloat16)
        G = big[:, :n]
        out = torch.full((m, n + extra), 7.0, device="cuda")
        gpu_lib.orthogonalize(G, out[:, extra:], Q, 5, "f32")
        assert rel(out[:, extra:], ns64(G.double(), [Q] * 5)) <= TOL32
        assert torch.all(out[:, :extra] == 7.0)


def test_large_tiles_and_another_stream(gpu_lib):
    """Enough matrices for the 256 x 256 tiles, on a side stream."""
    import torch
    shapes = [(768, 768)] * 30 + [(700, 1500)] * 6
    Gs = [draw(m, n, 50 + i, torch.bfloat16) for i, (m, n) in enumerate(shapes)]
    Os = [torch.empty(s, device="cuda") for s in shapes]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for mode, tol in (("f32", TOL32), ("f16", TOL16)):
        ws = gpu_lib.orthogonalize_batched(list(zip(Gs, Os)), math=mode, stream=side)
        gpu_lib.check_status(ws, len(shapes), stream=side)
        torch.cuda.current_stream().wait_stream(side)
        for i in (0, 17, 29, 30, 35):
            assert rel(Os[i], ns64(Gs[i].double(), [Q] * 5)) <= tol


def test_graph_replays(gpu_lib):
    import torch
    Gs = [draw(150, 90, 1, torch.float32), draw(90, 300, 2, torch.float32)]
    Os = [torch.empty_like(g) for g in Gs]
    ws = gpu_lib.orthogonalize_batched(list(zip(Gs, Os)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.orthogonalize_batched(list(zip(Gs, Os)), workspace=ws)
    for rep in range(4):
        for i, g in enumerate(Gs):
            g.copy_(draw(*g.shape, 60 + 2 * rep + i, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in Os]
        gpu_lib.orthogonalize_batched(list(zip(Gs, Os)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, Os))


# --- the step --------------------------------------------------------------

def muon64(X, G, M, lr, mu, nesterov, wd, s, coeffs):
    lr, mu, wd = f32(lr), f32(mu), f32(wd)
    M = mu * M + G
    D = G + mu * M if nesterov else M
    return (1 - lr * wd) * X - lr * s * ns64(D, coeffs), M


@pytest.mark.parametrize("m,n", [(1, 5), (64, 200), (200, 64), (257, 129), (500, 640)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
def test_muon_step(gpu_lib, m, n, nesterov, gdt):
    """Three steps; each from the state the GPU holds.  The update is lr s O
    with |O| at most sqrt(p) in norm, so X is off by TOL32 of that and by its
    own rounding."""
    import torch
    say(f"muon {m}x{n} {nesterov} {gdt}")
    X, M = draw(m, n, 1, torch.float32) * 0.02, torch.zeros(m, n, device="cuda")
    for t, scale in enumerate(("spectral", "rms", 0.7)):
        G = draw(m, n, 10 + t, getattr(torch, gdt))
        s = {"spectral": max(1.0, m / n) ** 0.5, "rms": 0.2 * max(m, n) ** 0.5}.get(scale, 0.7)
        x, mm = muon64(X.double(), G.double(), M.double(), 0.02, 0.9, nesterov, 0.1, s, [Q] * 5)
        ws = gpu_lib.muon_step(X, G, M, 0.02, 0.9, nesterov, 0.1, scale, Q, 5)
        gpu_lib.check_status(ws, 1)
        assert rel(M, mm) <= 2.0 ** -22
        step = 0.02 * s * min(m, n) ** 0.5 * 1.2
        bound = TOL32 * step + 2.0 ** -22 * float(torch.linalg.vector_norm(x))
        assert float(torch.linalg.vector_norm(X.double() - x)) <= bound


def test_muon_list_non_finite_and_zero(gpu_lib):
    """A matrix whose momentum or gradient is not finite keeps X and M bit
    for bit; one whose gradient and momentum are zero only decays."""
    import torch
    shapes = [(64, 200), (64, 200), (200, 64), (130, 130)]
    X = [draw(m, n, i, torch.float32) * 0.02 for i, (m, n) in enumerate(shapes)]
    M = [draw(m, n, 20 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    G = [draw(m, n, 40 + i, torch.bfloat16) for i, (m, n) in enumerate(shapes)]
    G[0][3, 4] = float("inf")
    M[2][0, 0] = float("nan")
    M[3].zero_()
    G[3].zero_()
    x0, m0 = [x.clone() for x in X], [m.clone() for m in M]
    ws = gpu_lib.muon_step_batched(list(zip(X, G, M)), 0.02, weight_decay=0.5)
    bad = gpu_lib.STATUS_NONFINITE
    assert gpu_lib.status(ws, 4)[1] == [bad, 0, bad, 0]
    for i in (0, 2):
        assert torch.equal(X[i], x0[i])
        assert torch.equal(M[i].view(torch.int32), m0[i].view(torch.int32))
    x, mm = muon64(x0[1].double(), G[1].double(), m0[1].double(), 0.02, 0.95, True, 0.5, 1.0, [Q] * 5)
    assert rel(X[1], x) <= TOL32 and rel(M[1], mm) <= 2.0 ** -22
    assert rel(X[3], x0[3].double() * (1 - f32(0.02) * 0.5)) <= 2.0 ** -22
    assert torch.count_nonzero(M[3]) == 0


# sides around the limits of the one-workgroup form (64 x 512, 128 x 256) and
# the two-plane products of a short side
LIMITS = [(64, 512), (64, 513), (65, 256), (65, 257), (128, 257), (100, 700), (17, 400), (512, 64), (257, 128),
          (33, 129), (64, 129), (127, 128)]


@pytest.mark.parametrize("m,n", LIMITS)
def test_limits_of_the_schedules(gpu_lib, m, n):
    import torch
    say(f"ns limits {m}x{n}")
    G = draw(m, n, 300 + m + n, torch.float32)
    O = torch.full((m, n), float("nan"), device="cuda")
    for cs in ([Q] * 5, [CUBIC] * 3, [Q, CUBIC]):
        gpu_lib.orthogonalize(G, O, cs, len(cs), "f32")
        assert rel(O, ns64(G.double(), cs)) <= TOL32
    Ob = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gpu_lib.orthogonalize(G, Ob, Q, 5, "f16")
    assert rel(Ob, ns64(G.double(), [Q] * 5)) <= TOL16 + TOL_BF


@pytest.mark.parametrize("m,n", [(64, 513), (257, 129), (100, 700), (40, 500), (128, 200)])
def test_muon_schedules(gpu_lib, m, n):
    import torch
    X, M = draw(m, n, 1, torch.float32) * 0.02, draw(m, n, 2, torch.float32)
    G = draw(m, n, 3, torch.bfloat16)
    x, mm = muon64(X.double(), G.double(), M.double(), 0.02, 0.95, True, 0.1, 1.5, [Q] * 5)
    gpu_lib.muon_step(X, G, M, 0.02, 0.95, True, 0.1, 1.5, Q, 5)
    assert rel(M, mm) <= 2.0 ** -22
    bound = TOL32 * 0.02 * 1.5 * min(m, n) ** 0.5 * 1.2 + 2.0 ** -22 * float(torch.linalg.vector_norm(x))
    assert float(torch.linalg.vector_norm(X.double() - x)) <= bound


def test_large_reductions_are_cut(gpu_lib):
    """Few tiles and a long reduction: the tiles' slices are joined; twice the
    same bits."""
    import torch
    for m, n, mode, tol in ((300, 6000, "f16", TOL16), (6000, 300, "f32", TOL32), (1500, 1700, "f32", TOL32)):
        say(f"ns cut {m}x{n} {mode}")
        G = draw(m, n, m, torch.float32)
        O, P = torch.empty_like(G), torch.empty_like(G)
        gpu_lib.orthogonalize(G, O, math=mode)
        gpu_lib.orthogonalize(G, P, math=mode)
        assert rel(O, ns64(G.double(), [Q] * 5)) <= tol
        assert torch.equal(O, P)


@pytest.mark.parametrize("m,n", [(1, 32768), (1, 32769), (16, 2048), (16, 2049), (2048, 16), (3, 6000), (9, 9), (16, 16),
                                 (17, 17), (8, 1000), (1000, 2)])
def test_few_rows(gpu_lib, m, n):
    """Matrices of few singular values, whose roundings do not average: the
    float32 form (up to 16 rows that fit the LDS) and its neighbours."""
    import torch
    say(f"ns few rows {m}x{n}")
    for dt in (torch.float32, torch.bfloat16):
        G = draw(m, n, 400 + m + n, dt)
        O = torch.full((m, n), float("nan"), device="cuda")
        for cs in ([Q] * 5, [CUBIC] * 4):
            ws = gpu_lib.orthogonalize(G, O, cs, len(cs), "f32")
            gpu_lib.check_status(ws, 1)
            assert rel(O, ns64(G.double(), cs)) <= TOL32
    X, M = draw(m, n, 1, torch.float32) * 0.02, draw(m, n, 2, torch.float32)
    x, mm = muon64(X.double(), G.double(), M.double(), 0.02, 0.95, False, 0.1, 1.0, [Q] * 5)
    gpu_lib.muon_step(X, G, M, 0.02, 0.95, False, 0.1, "none", Q, 5)
    assert rel(M, mm) <= 2.0 ** -22
    bound = TOL32 * 0.02 * min(m, n) ** 0.5 * 1.2 + 2.0 ** -22 * float(torch.linalg.vector_norm(x))
    assert float(torch.linalg.vector_norm(X.double() - x)) <= bound
