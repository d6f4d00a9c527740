"""Further refusals and acceptances of the training operators' entry points:
before any HIP call, so on a machine without a GPU too.  An accepted call
shows as ERR_WORKSPACE on a workspace of no bytes."""
import ctypes

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

A, B, C, W = (k << 40 for k in range(1, 5))   # fake, aligned device addresses
Q = (ctypes.c_float * 15)(*([3.4445, -4.7750, 2.0315] * 5))


@pytest.fixture(scope="module")
def lib():
    return dion.load()


@pytest.mark.parametrize("lr,wd,scale", [(1e30, 1e30, 1.0), (-1e30, 1e30, 1.0), (1e30, 0.0, 1e30)])
def test_muon_refuses_factors_that_overflow(lib, lr, wd, scale):
    """1 - lr weight_decay and lr scale are formed in float32: where they are
    not finite, every weight would become infinite or NaN."""
    rc = lib.dion_muon_step(A, B, C, 64, 32, scale, lr, 0.95, 1, wd, Q, 5, 0, 0, W, 0, None)
    assert rc == dion.ERR_INVALID_ARG
    rc = lib.dion_muon_step(A, B, C, 64, 32, 1.0, 1e20, 0.95, 1, 1e10, Q, 5, 0, 0, W, 0, None)
    assert rc == dion.ERR_WORKSPACE


def orth(lib, G, O, n, ldg, ldo, m=40, gd=0, od=0):
    return lib.dion_orthogonalize(G, ldg, O, ldo, m, n, Q, 5, 0, gd, od, W, 0, None)


def linear(lib, name, **kw):
    base = dict(t=100, n=32, k=64, x=A, ldx=64, w=B, ldw=64, y=C, ldy=32, dy=C, lddy=32, act=0, dtype=0)
    base.update(kw)
    return getattr(lib, f"dion_linear_{name}")(ctypes.byref(dion.dion_linear(**base)), W, 0, None)


def test_columns_of_one_buffer(lib):
    """Column blocks of one buffer interleave in memory without sharing an
    element: outputs may lie beside inputs and beside each other."""
    ok, no = dion.ERR_WORKSPACE, dion.ERR_INVALID_ARG
    # G | O, O | G; one column in common, either side; other pitches
    assert orth(lib, A, A + 4 * 32, 32, 64, 64) == ok
    assert orth(lib, A + 4 * 32, A, 32, 64, 64) == ok
    assert orth(lib, A, A + 4 * 31, 32, 64, 64) == no
    assert orth(lib, A, A + 4 * 33, 32, 64, 64) == no
    assert orth(lib, A, A + 4 * 32, 32, 64, 65) == no
    # the same block some rows further down
    assert orth(lib, A, A + 4 * (64 * 7 + 32), 32, 64, 64) == ok
    assert orth(lib, A, A + 4 * 64 * 7, 32, 64, 64) == no
    assert orth(lib, A, A + 4 * 64 * 40, 32, 64, 64) == ok
    # bfloat16 and float32 of the same byte pitch
    assert orth(lib, A, A + 2 * 32, 32, 128, 64, gd=1) == ok
    assert orth(lib, A, A + 2 * 30, 32, 128, 64, gd=1) == no
    # a single row of G in a gap between O's rows
    assert orth(lib, A + 4 * 32, A, 32, 64, 64, m=1) == ok

    ld = 160   # x (64) | y (32) | z (32) | residual (32)
    y, z, r = A + 4 * 64, A + 4 * 96, A + 4 * 128
    assert linear(lib, "forward", ldx=ld, y=y, ldy=ld, z=z, ldz=ld, residual=r, ldr=ld) == ok
    assert linear(lib, "forward", ldx=ld, y=y - 4, ldy=ld) == no
    assert linear(lib, "forward", ldx=ld, y=y, ldy=ld, z=z - 4, ldz=ld) == no
    assert linear(lib, "forward", ldx=ld, y=y, ldy=ld, residual=y + 4, ldr=ld) == no
    # dy | dx beside each other (x elsewhere)
    assert linear(lib, "backward", x=W, dy=A, lddy=96, dx=A + 4 * 32, lddx=96) == ok
    assert linear(lib, "backward", x=W, dy=A, lddy=96, dx=A + 4 * 33, lddx=96) == no


@pytest.mark.parametrize("p,q", [(1, 32769), (1, 1 << 20), (4, 10000), (16, 2049), (16, 100000)])
def test_few_rows_workspace(lib, p, q):
    """A matrix of at most 16 rows or columns takes a float32 copy of itself and
    partial sums (less than half a megabyte), not planes padded to 64 rows."""
    for m, n in ((p, q), (q, p)):
        a = dion.dion_ns_matrix(A, B, m, n, n, n)
        for math in dion.MATH_NS.values():
            assert 0 < lib.dion_orthogonalize_workspace_size(ctypes.byref(a), 1, math) <= 8 * p * q + (1 << 19)
