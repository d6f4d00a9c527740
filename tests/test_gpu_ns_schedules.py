"""Orthogonalization and the Muon step (GPU) where lists mix schedules: the
grouped launches with tiles cut along the reduction, large tiles, the
one-workgroup forms.  Tolerances as in test_gpu_ns."""
import pytest

from .gpuhelp import say
from .test_gpu_ns import Q, TOL16, TOL32, draw, muon64, ns64, rel

pytestmark = pytest.mark.gpu

TOLS = {"f32": TOL32, "f16": TOL16}
BAD = (float("inf"), float("nan"), float("-inf"))
# few tiles and long reductions (cut along them), one-workgroup forms, and
# next to each a sound one; shape, whether it is bad
MIXED = [((300, 6000), True), ((300, 6000), False), ((6000, 300), True), ((6000, 300), False), ((1500, 1700), True),
         ((1500, 1700), False), ((520, 260), False), ((520, 260), True), ((3, 50), True), ((3, 50), False),
         ((70, 40), True), ((70, 40), False), ((130, 1000), True), ((130, 1000), False)]
# enough 256 x 256 tiles, one matrix bad
MANY = [((768, 768), i == 5) for i in range(48)] + [((700, 1500), i == 2) for i in range(6)]


def spoil(t, seed):
    """One entry that is not finite: the first, the last, or one between."""
    r, c = [(0, 0), (t.shape[0] - 1, t.shape[1] - 1), (t.shape[0] // 2, t.shape[1] // 3)][seed % 3]
    t[r, c] = BAD[(seed // 3 + seed) % 3]


def bits(t):
    import torch
    return t.view(torch.int32)


@pytest.mark.parametrize("mode", ["f32", "f16"])
@pytest.mark.parametrize("cases", [MIXED, MANY], ids=["mixed", "many"])
def test_orthogonalize_keeps_bad_matrices_out(gpu_lib, cases, mode):
    import torch
    say(f"ns bad {len(cases)} {mode}")
    n = len(cases)
    want = [gpu_lib.STATUS_NONFINITE if bad else 0 for _, bad in cases]
    sound = [draw(*s, 600 + i, torch.float32) for i, (s, _) in enumerate(cases)]
    G = [g.clone() for g in sound]
    for i, (_, bad) in enumerate(cases):
        if bad:
            spoil(G[i], i)
    O = [torch.full(s, 3.0, device="cuda") for s, _ in cases]
    ws = gpu_lib.orthogonalize_batched(list(zip(G, O)), math=mode)
    for rep in range(2):   # the second time on the workspace that the first left
        assert gpu_lib.status(ws, n)[1] == want
        for i, (_, bad) in enumerate(cases):
            if bad:
                assert torch.all(O[i] == 3.0), i
            elif n < 20 or i % 9 in (4, 6) or i >= 48:
                assert rel(O[i], ns64(G[i].double(), [Q] * 5)) <= TOLS[mode], i
            if not bad:
                O[i].fill_(float("nan"))
        ws = gpu_lib.orthogonalize_batched(list(zip(G, O)), math=mode, workspace=ws)
    # and nothing of them is left when all are sound
    gpu_lib.orthogonalize_batched(list(zip(sound, O)), math=mode, workspace=ws)
    gpu_lib.check_status(ws, n)
    for i in range(n):
        if cases[i][1] or n < 20:
            assert rel(O[i], ns64(sound[i].double(), [Q] * 5)) <= TOLS[mode], i


@pytest.mark.parametrize("mode", ["f32", "f16"])
@pytest.mark.parametrize("where", ["G", "M"])
def test_muon_keeps_bad_matrices_out(gpu_lib, mode, where):
    import torch
    cases = MIXED + [((768, 768), False)] * 2 + [((768, 768), True)]
    n = len(cases)
    X = [draw(*s, 700 + i, torch.float32) * 0.02 for i, (s, _) in enumerate(cases)]
    M = [draw(*s, 800 + i, torch.float32) for i, (s, _) in enumerate(cases)]
    G = [draw(*s, 900 + i, torch.float32) for i, (s, _) in enumerate(cases)]
    for i, (_, bad) in enumerate(cases):
        if bad:
            spoil((G if where == "G" else M)[i], i)
    x0, m0 = [x.clone() for x in X], [m.clone() for m in M]
    ws = gpu_lib.muon_step_batched(list(zip(X, G, M)), 0.02, 0.9, True, 0.1, 1.5, math=mode)
    assert gpu_lib.status(ws, n)[1] == [gpu_lib.STATUS_NONFINITE if bad else 0 for _, bad in cases]
    for i, ((m, k), bad) in enumerate(cases):
        if bad:
            assert torch.equal(bits(X[i]), bits(x0[i])) and torch.equal(bits(M[i]), bits(m0[i])), i
            continue
        x, mm = muon64(x0[i].double(), G[i].double(), m0[i].double(), 0.02, 0.9, True, 0.1, 1.5, [Q] * 5)
        assert rel(M[i], mm) <= 2.0 ** -22
        bound = TOLS[mode] * 0.02 * 1.5 * min(m, k) ** 0.5 * 1.2 + 2.0 ** -22 * float(torch.linalg.vector_norm(x))
        assert float(torch.linalg.vector_norm(X[i].double() - x)) <= bound, i


def step_case(lib, shapes, mode, gdt, nesterov=True):
    """One Muon step over a list, every matrix against float64."""
    import torch
    X = [draw(m, n, 20 + i, torch.float32) * 0.02 for i, (m, n) in enumerate(shapes)]
    M = [draw(m, n, 120 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    G = [draw(m, n, 220 + i, gdt) for i, (m, n) in enumerate(shapes)]
    want = [muon64(x.double(), g.double(), mm.double(), 0.02, 0.95, nesterov, 0.1, 1.5, [Q] * 5)
            for x, g, mm in zip(X, G, M)]
    ws = lib.muon_step_batched(list(zip(X, G, M)), 0.02, 0.95, nesterov, 0.1, 1.5, math=mode)
    lib.check_status(ws, len(shapes))
    for s, x, mm, (ex, em) in zip(shapes, X, M, want):
        assert rel(mm, em) <= 2.0 ** -22, s
        bound = TOLS[mode] * 0.02 * 1.5 * min(s) ** 0.5 * 1.2 + 2.0 ** -22 * float(torch.linalg.vector_norm(ex))
        assert float(torch.linalg.vector_norm(x.double() - ex)) <= bound, s


@pytest.mark.parametrize("m,n", [(130, 1000), (1000, 130), (257, 129), (300, 6000), (6000, 300), (600, 520), (1031, 773)])
@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
def test_muon_float16_products(gpu_lib, m, n, gdt):
    import torch
    say(f"muon f16 {m}x{n} {gdt}")
    for nesterov in (True, False):
        step_case(gpu_lib, [(m, n)], "f16", getattr(torch, gdt), nesterov)


@pytest.mark.parametrize("mode", ["f32", "f16"])
def test_muon_large_tiles(gpu_lib, mode):
    """256 x 256 tiles in every product, wide and tall, ragged edges: 28 upper
    tiles of a 1543-row matrix, ten of them."""
    import torch
    shapes = [(1543, 1600), (1600, 1543)] * 5
    say(f"muon large tiles {mode}")
    step_case(gpu_lib, shapes, mode, torch.bfloat16)


@pytest.mark.parametrize("mode", ["f32", "f16"])
def test_muon_list_of_mixed_shapes(gpu_lib, mode):
    import torch
    say(f"muon mixed {mode}")
    step_case(gpu_lib, [s for s, _ in MIXED] + [(900, 1400), (1400, 900), (2, 40000)], mode, torch.float32)


@pytest.mark.parametrize("m,n", [(4, 9), (70, 40), (130, 300), (2, 30000)])
def test_single_matrix_entry_points(gpu_lib, m, n):
    """dion_orthogonalize and dion_muon_step give the bits of lists of one."""
    import ctypes
    import torch
    lib = gpu_lib.load()
    coeffs = (ctypes.c_float * 15)(*(Q * 5))
    stream = torch.cuda.current_stream().cuda_stream
    for mode in ("f32", "f16"):
        for gdt in (torch.float32, torch.bfloat16):
            big = draw(m, n + 3, 1, gdt)
            G, g = big[:, :n], 1 if gdt == torch.bfloat16 else 0
            for odt in (torch.float32, torch.bfloat16):
                want = torch.empty(m, n, dtype=odt, device="cuda")
                ws = gpu_lib.orthogonalize(G, want, math=mode)
                got = torch.zeros(m, n + 1, dtype=odt, device="cuda")
                rc = lib.dion_orthogonalize(big.data_ptr(), n + 3, got.data_ptr(), n + 1, m, n, coeffs, 5,
                                            gpu_lib.MATH_NS[mode], g, 1 if odt == torch.bfloat16 else 0,
                                            ws.data_ptr(), ws.numel(), stream)
                assert rc == gpu_lib.OK and torch.equal(got[:, :n], want)
                assert torch.count_nonzero(got[:, n]) == 0
            G = G.contiguous()
            X, M = draw(m, n, 2, torch.float32), draw(m, n, 3, torch.float32)
            x, mm = X.clone(), M.clone()
            ws = gpu_lib.muon_step(X, G, M, 0.02, 0.9, True, 0.1, 0.7, math=mode)
            rc = lib.dion_muon_step(x.data_ptr(), G.data_ptr(), mm.data_ptr(), m, n, 0.7, 0.02, 0.9, 1, 0.1, coeffs,
                                    5, gpu_lib.MATH_NS[mode], g, ws.data_ptr(), ws.numel(), stream)
            assert rc == gpu_lib.OK and torch.equal(X, x) and torch.equal(M, mm)


@pytest.mark.parametrize("mode", ["f32", "f16"])
def test_many_shapes(gpu_lib, mode):
    """61 matrices, each of its own shape, in every form: three uploads of the
    descriptor table and several launches per product."""
    import torch
    shapes = [(3 + 17 * i, 5 + (29 * i * i) % 1100) for i in range(45)]
    shapes += [(2 + i, 20000 - 900 * i) for i in range(8)] + [(17000 + i, 1 + 2 * i) for i in range(8)]
    assert len(set(shapes)) == 61
    say(f"ns many shapes {mode}")
    G = [draw(m, n, 1000 + i, torch.float32) for i, (m, n) in enumerate(shapes)]
    O = [torch.full(s, float("nan"), device="cuda") for s in shapes]
    ws = gpu_lib.orthogonalize_batched(list(zip(G, O)), math=mode)
    gpu_lib.check_status(ws, len(shapes))
    for s, g, o in zip(shapes, G, O):
        assert rel(o, ns64(g.double(), [Q] * 5)) <= TOLS[mode], s
    step_case(gpu_lib, shapes, mode, torch.bfloat16)
