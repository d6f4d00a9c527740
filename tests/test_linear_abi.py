"""Refusals of the linear layer's entry points, before any HIP call."""
import ctypes

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

X, WT, Y, Z, R, DY, DX, DW, DB, B, S = (k << 40 for k in range(1, 12))


@pytest.fixture(scope="module")
def lib():
    return dion.load()


def args(**kw):
    base = dict(t=100, n=32, k=64, x=X, ldx=64, w=WT, ldw=64, y=Y, ldy=32, act=0, dtype=1,
                dy=DY, lddy=32, dx=DX, lddx=64, dw=DW, lddw=64, db=DB)
    base.update(kw)
    return dion.dion_linear(**base)


SHARED = [dict(t=-1), dict(n=0), dict(k=0), dict(t=1 << 25), dict(n=1 << 21), dict(act=5), dict(act=-1),
          dict(dtype=2), dict(x=None), dict(w=None), dict(ldx=63), dict(ldw=63), dict(x=X + 1)]


@pytest.mark.parametrize("kw", SHARED + [
    dict(y=None), dict(ldy=31), dict(y=X + 128), dict(y=WT), dict(z=Y + 64, ldz=32), dict(z=Z, ldz=31),
    dict(residual=Y + 64, ldr=32), dict(residual=Y, ldr=40), dict(residual=R, ldr=31),
    dict(bias=B + 2), dict(z=X, ldz=32),
])
def test_forward_refuses(lib, kw):
    a = args(**kw)
    assert lib.dion_linear_forward_workspace_size(ctypes.byref(a)) == 0
    assert lib.dion_linear_forward(ctypes.byref(a), S, 1 << 40, None) == dion.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SHARED + [
    dict(dy=None), dict(lddy=31), dict(act=3), dict(act=3, z=Z, ldz=31), dict(dx=DY), dict(dw=X),
    dict(dx=WT + 2), dict(db=DY), dict(lddx=63), dict(lddw=63), dict(dw=DX), dict(db=DB + 1),
])
def test_backward_refuses(lib, kw):
    a = args(**kw)
    assert lib.dion_linear_backward_workspace_size(ctypes.byref(a)) == 0
    assert lib.dion_linear_backward(ctypes.byref(a), S, 1 << 40, None) == dion.ERR_INVALID_ARG


def test_null_and_workspace(lib):
    assert lib.dion_linear_forward(None, S, 1 << 40, None) == dion.ERR_INVALID_ARG
    assert lib.dion_linear_backward(None, S, 1 << 40, None) == dion.ERR_INVALID_ARG
    assert lib.dion_linear_forward_workspace_size(None) == 0
    a = args(dtype=0)       # float32: split copies in the workspace
    need = lib.dion_linear_forward_workspace_size(ctypes.byref(a))
    assert need >= 2 * 3 * (100 * 64 + 32 * 64)
    for ws, nb in ((S, 1024), (None, need), (S + 8, need)):
        assert lib.dion_linear_forward(ctypes.byref(a), ws, nb, None) == dion.ERR_WORKSPACE
    need = lib.dion_linear_backward_workspace_size(ctypes.byref(a))
    assert lib.dion_linear_backward(ctypes.byref(a), S, 1024, None) == dion.ERR_WORKSPACE
    assert need > 0
    # nothing to do for no tokens: accepted without a GPU
    none = args(t=0, x=None, y=None)
    assert lib.dion_linear_forward(ctypes.byref(none), None, 0, None) == dion.OK


def test_binding_refuses():
    import torch
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        dion.linear_forward(x, x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        dion.linear_backward(x, act="gelu")
    with pytest.raises(ValueError):
        dion.linear_backward(x, dx=x)
    with pytest.raises(TypeError):
        dion.linear_forward(x.double(), x, x)
    with pytest.raises(ValueError):
        dion._act("tanh")


def test_act_codes_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "dion.h")).read()
    defs = {k.lower(): int(v) for k, v in re.findall(r"#define\s+DION_ACT_(\w+)\s+(\d+)", text)}
    assert defs == dion.ACTS
