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
