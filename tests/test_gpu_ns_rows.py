"""Matrices of at most 16 rows or columns that do not fit one workgroup (GPU):
plain float32 in several, against the formulas in float64.

Tolerance (relative Frobenius error): an iteration rounds the sums of A, B and
the new X, of which a few reach the result, at most a few tens of times the
size (the ratio of the polynomial's slopes): 64 * 2^-24, half of what two
planes of 22 bits are allowed."""
import pytest

from .gpuhelp import say
from .test_gpu_ns import CUBIC, Q, draw, f32, muon64, ns64, rel

pytestmark = pytest.mark.gpu

TOL = 64 * 2.0 ** -24
# one column past the one-workgroup form; odd sizes; chunks of one and of many
# columns per thread, the last chunk short; every number of rows from 1 to 16
SHAPES = [(1, 32769), (2, 16385), (3, 10923), (4, 10000), (5, 7000), (6, 5463), (7, 4999), (8, 4097), (9, 3641),
          (11, 3001), (13, 140001), (15, 2185), (16, 2049), (16, 131073), (1, 1048576), (2, 300001)]


@pytest.mark.parametrize("p,q", SHAPES)
@pytest.mark.parametrize("tall", [False, True])
def test_accuracy(gpu_lib, p, q, tall):
    import torch
    m, n = (q, p) if tall else (p, q)
    say(f"ns rows {m}x{n}")
    for dt in (torch.float32, torch.bfloat16):
        G = draw(m, n, 500 + p + q, dt)
        O = torch.full((m, n), float("nan"), device="cuda")
        for cs in ([Q] * 5, [CUBIC] * 4, [Q]):
            ws = gpu_lib.orthogonalize(G, O, cs, len(cs), "f32")
            gpu_lib.check_status(ws, 1)
            assert rel(O, ns64(G.double(), cs)) <= TOL
    gpu_lib.orthogonalize(G, O, Q, 5, "f32")
    Ob = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    gpu_lib.orthogonalize(G, Ob, Q, 5, "f16")     # one arithmetic in both modes
    assert torch.equal(Ob, O.bfloat16())


@pytest.mark.parametrize("m,n", [(3, 11000), (11000, 3), (16, 2500), (40000, 1), (9, 70001)])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
def test_muon(gpu_lib, m, n, gdt):
    import torch
    for nesterov in (True, False):
        X, M = draw(m, n, 1, torch.float32) * 0.02, draw(m, n, 2, torch.float32)
        G = draw(m, n, 3, getattr(torch, gdt))
        x, mm = muon64(X.double(), G.double(), M.double(), 0.02, 0.95, nesterov, 0.1, 1.5, [Q] * 5)
        ws = gpu_lib.muon_step(X, G, M, 0.02, 0.95, nesterov, 0.1, 1.5, Q, 5)
        gpu_lib.check_status(ws, 1)
        assert rel(M, mm) <= 2.0 ** -22
        bound = TOL * 0.02 * 1.5 * min(m, n) ** 0.5 * 1.2 + 2.0 ** -22 * float(torch.linalg.vector_norm(x))
        assert float(torch.linalg.vector_norm(X.double() - x)) <= bound


def test_pitches_scales_and_zero(gpu_lib):
    import torch
    for m, n in ((5, 7000), (7000, 5)):
        for extra in (1, 3, 8):
            big = draw(m, n + extra, 9, torch.bfloat16)
            out = torch.full((m, n + extra), 7.0, device="cuda")
            gpu_lib.orthogonalize(big[:, :n], out[:, extra:])
            assert rel(out[:, extra:], ns64(big[:, :n].double(), [Q] * 5)) <= TOL
            assert torch.all(out[:, :extra] == 7.0)
        for scale in (1e-30, 1e30):
            G, O = draw(m, n, 4, torch.float32) * scale, torch.empty(m, n, device="cuda")
            gpu_lib.orthogonalize(G, O)
            assert rel(O, ns64(G.double(), [Q] * 5)) <= TOL
        Z = torch.zeros(m, n, device="cuda")
        ws = gpu_lib.orthogonalize(Z, O)
        gpu_lib.check_status(ws, 1)
        assert torch.count_nonzero(O) == 0


def test_list_with_bad_matrices(gpu_lib):
    """Several of the form among others, some not finite: those keep O, X and
    M bit for bit, the others are as in calls of their own; then again on the
    same workspace with every matrix sound."""
    import torch
    shapes = [(3, 20000), (200, 300), (20000, 3), (3, 20000), (16, 4000), (12, 3000), (30, 40), (1, 50000)]
    bad = (0, 2, 4)
    want = [gpu_lib.STATUS_NONFINITE if i in bad else 0 for i in range(len(shapes))]
    G = [draw(m, n, 70 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    keep = [g.clone() for g in G]
    G[0][2, 19999] = float("inf")
    G[2][0, 0] = float("nan")
    G[4][7, 5] = float("-inf")
    O = [torch.full(s, 3.0, device="cuda") for s in shapes]
    ws = gpu_lib.orthogonalize_batched(list(zip(G, O)))
    assert gpu_lib.status(ws, len(shapes))[1] == want
    for i, g in enumerate(G):
        if i in bad:
            assert torch.all(O[i] == 3.0)
        else:
            alone = torch.empty_like(O[i])
            gpu_lib.orthogonalize(g, alone)
            assert rel(O[i], ns64(g.double(), [Q] * 5)) <= 2 * TOL and rel(O[i], alone.double()) <= 2 * TOL
    X = [torch.full(s, 0.5, device="cuda") for s in shapes]
    M = [k * 0.25 for k in keep]
    m0 = [v.clone() for v in M]
    ws = gpu_lib.muon_step_batched(list(zip(X, G, M)), 0.02, workspace=ws)
    assert gpu_lib.status(ws, len(shapes))[1] == want
    for i in range(len(shapes)):
        if i in bad:
            assert torch.all(X[i] == 0.5) and torch.equal(M[i], m0[i])
        else:
            assert rel(M[i], f32(0.95) * m0[i].double() + G[i].double()) <= 2.0 ** -22
    gpu_lib.orthogonalize_batched(list(zip(keep, O)), workspace=ws)
    gpu_lib.check_status(ws, len(shapes))
    for g, o in zip(keep, O):
        assert rel(o, ns64(g.double(), [Q] * 5)) <= 2 * TOL


def test_same_bits_and_graph(gpu_lib):
    import torch
    Gs = [draw(4, 30000, 1, torch.float32), draw(16, 9000, 2, torch.float32), draw(50000, 2, 3, torch.float32)]
    Os = [torch.empty_like(g) for g in Gs]
    ws = gpu_lib.orthogonalize_batched(list(zip(Gs, Os)))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.orthogonalize_batched(list(zip(Gs, Os)), workspace=ws)
    for rep in range(4):
        for i, g in enumerate(Gs):
            g.copy_(draw(*g.shape, 60 + 3 * rep + i, torch.float32))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in Os]
        gpu_lib.orthogonalize_batched(list(zip(Gs, Os)))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, Os))
        single = torch.empty_like(Gs[0])
        gpu_lib.orthogonalize(Gs[0], single)
        assert torch.equal(single, Os[0])
