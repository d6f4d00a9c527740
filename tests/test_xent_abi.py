"""Refusals of the cross entropy's entry points, before any HIP call."""
import ctypes
import math

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

X, WT, Y, L, E, D, DX, DW, S = (k << 40 for k in range(1, 10))


@pytest.fixture(scope="module")
def lib():
    return dion.load()


def args(**kw):
    base = dict(t=100, n=320, k=64, x=X, ldx=64, w=WT, ldw=64, target=Y, loss=L, lse=E, dloss=D, dx=DX, lddx=64,
                dw=DW, lddw=64, ignore_index=-100, dtype=1)
    base.update(kw)
    return dion.dion_cross_entropy(**base)


SHARED = [dict(t=-1), dict(n=0), dict(k=0), dict(t=1 << 25), dict(n=1 << 21), dict(k=1 << 21), dict(dtype=2),
          dict(x=None), dict(w=None), dict(target=None), dict(ldx=63), dict(ldw=63), dict(ldx=1 << 31), dict(x=X + 1),
          dict(w=WT + 1), dict(target=Y + 4), dict(label_smoothing=-0.1), dict(label_smoothing=1.1),
          dict(label_smoothing=math.nan), dict(z_loss=math.inf), dict(lse=E + 2)]


@pytest.mark.parametrize("kw", SHARED + [
    dict(loss=None, lse=None), dict(loss=L + 1), dict(loss=E), dict(loss=X + 64), dict(lse=WT + 128), dict(lse=Y),
    dict(loss=E + 396),
])
def test_forward_refuses(lib, kw):
    a = args(**kw)
    assert lib.dion_cross_entropy_forward_workspace_size(ctypes.byref(a)) == 0
    assert lib.dion_cross_entropy_forward(ctypes.byref(a), S, 1 << 40, None) == dion.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SHARED + [
    dict(lse=None), dict(dloss=None), dict(dloss=D + 2), dict(lddx=63), dict(lddw=63), dict(dx=X), dict(dx=WT + 2),
    dict(dw=X + 64), dict(dw=DX), dict(dw=D), dict(dx=Y), dict(dw=E - 4), dict(dx=DX + 1),
])
def test_backward_refuses(lib, kw):
    a = args(**kw)
    assert lib.dion_cross_entropy_backward_workspace_size(ctypes.byref(a)) == 0
    assert lib.dion_cross_entropy_backward(ctypes.byref(a), S, 1 << 40, None) == dion.ERR_INVALID_ARG


@pytest.mark.parametrize("name", ["forward", "backward"])
@pytest.mark.parametrize("kw", [dict(), dict(dtype=0), dict(t=5), dict(k=63), dict(t=5, k=63), dict(ignore_index=7)])
def test_workspace(lib, name, kw):
    size = getattr(lib, f"dion_cross_entropy_{name}_workspace_size")
    run = getattr(lib, f"dion_cross_entropy_{name}")
    a = args(**kw)
    need = size(ctypes.byref(a))
    assert need > 0
    for ws, nb in ((S, need - 1), (None, need), (S + 8, need)):
        assert run(ctypes.byref(a), ws, nb, None) == dion.ERR_WORKSPACE
    assert size(None) == 0 and run(None, S, need, None) == dion.ERR_INVALID_ARG


def test_workspace_is_bounded(lib):
    """Pieces of the vocabulary, not all of its logits: 8192 tokens of a
    vocabulary of 2^18 have 4 GiB of bfloat16 logits."""
    a = args(t=8192, n=1 << 18, k=4096, ldx=4096, ldw=4096, lddx=4096, lddw=4096)
    assert lib.dion_cross_entropy_forward_workspace_size(ctypes.byref(a)) < (1 << 31) / 8 + (1 << 24)
    # dz, dx's sums (128 MiB), slices of tiles
    assert lib.dion_cross_entropy_backward_workspace_size(ctypes.byref(a)) < (256 + 128 + 256) << 20
    a = args(t=8192, n=1 << 18, k=4096, ldx=4096, ldw=4096, lddx=4096, lddw=4096, dtype=0)
    assert lib.dion_cross_entropy_backward_workspace_size(ctypes.byref(a)) < (256 + 256 + 192 + 256) << 20


def test_nothing_to_do_needs_no_gpu(lib):
    a = args(t=0, x=None, target=None, loss=None, lse=None, dloss=None)
    need = lib.dion_cross_entropy_forward_workspace_size(ctypes.byref(a))
    assert lib.dion_cross_entropy_forward(ctypes.byref(a), S, need, None) == dion.OK
    a = args(t=0, x=None, target=None, lse=None, dloss=None, dw=None)
    need = lib.dion_cross_entropy_backward_workspace_size(ctypes.byref(a))
    assert lib.dion_cross_entropy_backward(ctypes.byref(a), S, need, None) == dion.OK
    a = args(dx=None, dw=None)
    assert lib.dion_cross_entropy_backward(ctypes.byref(a), S, 1 << 40, None) == dion.OK


def test_binding_refuses():
    import torch
    x, y = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        dion.cross_entropy_forward(x, x, y, torch.zeros(4))        # not on a GPU
    with pytest.raises(TypeError):
        dion.cross_entropy_forward(x.double(), x, y, torch.zeros(4))
    with pytest.raises(ValueError):
        dion.cross_entropy_forward(x, x[0], y, torch.zeros(4))
    with pytest.raises(ValueError):
        dion.cross_entropy_backward(torch.zeros(4), x[0], x, y, torch.zeros(4))
