"""Refusals of the orthogonalization and Muon entry points: before any HIP
call, so on a machine without a GPU too."""
import ctypes
import math

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

A, B, C, W = (k << 40 for k in range(1, 5))   # fake, aligned device addresses
Q = (ctypes.c_float * 15)(*([3.4445, -4.7750, 2.0315] * 5))


@pytest.fixture(scope="module")
def lib():
    return dion.load()


def orth(lib, G=A, O=B, m=64, n=32, ldg=None, ldo=None, coeffs=Q, steps=5, math_=0, gd=0, od=0,
         ws=W, nbytes=1 << 30):
    return lib.dion_orthogonalize(G, n if ldg is None else ldg, O, n if ldo is None else ldo, m, n,
                                  coeffs, steps, math_, gd, od, ws, nbytes, None)


def bad_coeffs(*v):
    return (ctypes.c_float * 15)(*(list(v) * 5))


@pytest.mark.parametrize("kw", [
    dict(G=None), dict(O=None), dict(m=0), dict(n=0), dict(m=-1), dict(m=1 << 21),
    dict(m=1 << 16, n=1 << 16), dict(ldg=31), dict(ldo=31), dict(ldg=1 << 32),
    dict(G=A + 2), dict(G=A + 1, gd=1), dict(O=B + 2), dict(O=B + 1, od=1),
    dict(O=A + 64), dict(coeffs=None), dict(steps=0), dict(steps=33), dict(math_=0x100),
    dict(math_=1), dict(gd=2), dict(od=-1),
    dict(coeffs=bad_coeffs(math.nan, 0, 0)), dict(coeffs=bad_coeffs(1, math.inf, 0)),
    dict(coeffs=bad_coeffs(100.0, 0.0, 0.0)),       # singular values grow past 64
])
def test_orthogonalize_refuses(lib, kw):
    assert orth(lib, **kw) == dion.ERR_INVALID_ARG


def test_orthogonalize_workspace(lib):
    arr = (dion.dion_ns_matrix * 2)(dion.dion_ns_matrix(A, B, 64, 32, 32, 32),
                                    dion.dion_ns_matrix(C, W, 300, 700, 700, 700))
    one = lib.dion_orthogonalize_workspace_size(arr, 1, 0)
    two = lib.dion_orthogonalize_workspace_size(arr, 2, 0)
    half = lib.dion_orthogonalize_workspace_size(arr, 2, dion.MATH_NS["f16"])
    assert 0 < one < two and half < two
    assert orth(lib, nbytes=one - 1) == dion.ERR_WORKSPACE
    assert orth(lib, ws=None) == dion.ERR_WORKSPACE
    assert orth(lib, ws=W + 8) == dion.ERR_WORKSPACE
    assert lib.dion_orthogonalize_workspace_size(arr, 0, 0) == 0
    assert lib.dion_orthogonalize_workspace_size(None, 1, 0) == 0
    assert lib.dion_orthogonalize_workspace_size(arr, 1, 2) == 0
    assert lib.dion_orthogonalize_batched(arr, -1, Q, 5, 0, 0, 0, W, 1 << 30, None) == \
        dion.ERR_INVALID_ARG
    assert lib.dion_orthogonalize_batched(None, 1, Q, 5, 0, 0, 0, W, 1 << 30, None) == \
        dion.ERR_INVALID_ARG


def muon(lib, X=A, G=B, M=C, m=64, n=32, scale=1.0, lr=0.02, mu=0.95, wd=0.0, ws=W, nbytes=1 << 30):
    return lib.dion_muon_step(X, G, M, m, n, scale, lr, mu, 1, wd, Q, 5, 0, 0, ws, nbytes, None)


@pytest.mark.parametrize("kw", [
    dict(X=None), dict(G=None), dict(M=None), dict(m=0), dict(n=0), dict(X=A + 2), dict(M=C + 1),
    dict(M=A + 128), dict(M=B + 128), dict(X=B), dict(scale=math.nan), dict(lr=math.inf),
    dict(mu=math.nan), dict(wd=math.inf),
])
def test_muon_refuses(lib, kw):
    assert muon(lib, **kw) == dion.ERR_INVALID_ARG


def test_muon_workspace(lib):
    arr = (dion.dion_muon_matrix * 1)(dion.dion_muon_matrix(A, B, C, 64, 32, 1.0))
    need = lib.dion_muon_workspace_size(arr, 1, 0)
    assert need > 0 and muon(lib, nbytes=need - 1) == dion.ERR_WORKSPACE


def test_binding_refuses():
    import torch
    g = torch.zeros(4, 4)
    with pytest.raises(ValueError):
        dion.orthogonalize(g, g.clone())            # not on a GPU
    with pytest.raises(ValueError):
        dion.orthogonalize_batched([])
    with pytest.raises(ValueError):
        dion._ns_coeffs([(1, 2, 3)], 2)
    with pytest.raises(ValueError):
        dion._ns_math("bf16x3")
    with pytest.raises(ValueError):
        dion._muon_scale("other", 3, 4)


def test_constants_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "dion.h")).read()
    defs = {k: int(v, 0) for k, v in re.findall(r"#define\s+(DION_\w+)\s+\(?(-?(?:0x)?[0-9a-fA-F]+)\)?", text)}
    assert defs["DION_MATH_F16"] == dion.MATH_NS["f16"] and defs["DION_MATH_F32"] == dion.MATH_NS["f32"]
    assert defs["DION_STATUS_NONFINITE"] == dion.STATUS_NONFINITE
