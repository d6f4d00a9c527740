"""Refusals of the AdamW step's entry points, before any HIP call, and the
mean of the 8-bit states' rounding (numpy model of the header's formulas)."""
import ctypes
import math

import numpy as np
import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

X, G, M, V, S, C = (k << 40 for k in range(1, 7))


@pytest.fixture(scope="module")
def lib():
    return dion.load()


def call(lib, count=1, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, step=1, c=None, bits=32, gd=0, more=(), **kw):
    base = dict(X=X, G=G, M=M, V=V, S=S, n=0, weight_decay=0.1)
    base.update(kw)
    rows = [base] + [dict(base, **m) for m in more]
    arr = (dion.dion_adamw_tensor * len(rows))(*[dion.dion_adamw_tensor(**r) for r in rows])
    return lib.dion_adamw_step_batched(arr, count, lr, b1, b2, eps, step, c, bits, 0, gd, None)


@pytest.mark.parametrize("kw", [
    dict(count=0), dict(count=-1), dict(count=65537), dict(bits=16), dict(bits=0), dict(gd=2), dict(step=0),
    dict(step=-3), dict(b1=1.0), dict(b1=-0.1), dict(b2=1.0), dict(b2=math.nan), dict(lr=math.inf), dict(lr=math.nan),
    dict(eps=0.0), dict(eps=-1e-8), dict(eps=math.inf), dict(eps=1e-39), dict(weight_decay=math.nan),
    dict(lr=1e30, weight_decay=1e30), dict(lr=1e300, b1=0.5), dict(c=C + 2),
    dict(n=-1), dict(n=(1 << 33) + 1), dict(n=8, X=None), dict(n=8, G=None), dict(n=8, M=None), dict(n=8, V=None),
    dict(n=8, S=None, bits=8), dict(n=8, X=X + 2), dict(n=8, G=G + 2), dict(n=8, G=G + 1, gd=1), dict(n=8, M=M + 1),
    dict(n=8, V=V + 2), dict(n=8, G=X + 28), dict(n=8, M=X + 28), dict(n=8, V=M + 28), dict(n=8, V=G),
    dict(n=8, c=X + 28), dict(n=8, c=M), dict(n=65, bits=8, c=S),
    dict(n=65, bits=8, S=M + 64), dict(n=65, bits=8, V=S + 3), dict(n=65, bits=8, S=X + 259),
])
def test_refuses(lib, kw):
    assert call(lib, **kw) == dion.ERR_INVALID_ARG


def test_second_tensor_is_checked_before_the_first_runs(lib):
    assert call(lib, count=2, more=[dict(n=8, X=None)], n=8) == dion.ERR_INVALID_ARG


def test_nothing_to_do_needs_no_gpu(lib):
    assert call(lib) == dion.OK
    assert call(lib, X=None, G=None, M=None, V=None, S=None, bits=8) == dion.OK
    assert call(lib, count=3, more=[dict(X=None), dict(G=G + 1)]) == dion.OK
    assert lib.dion_adamw_step(X, G, M, V, None, 0, 1e-3, 0.9, 0.999, 1e-8, 0.0, 1, None, 32, 0, 0, None) == dion.OK


def test_null_list(lib):
    assert lib.dion_adamw_step_batched(None, 1, 1e-3, 0.9, 0.999, 1e-8, 1, None, 32, 0, 0, None) == dion.ERR_INVALID_ARG


def test_binding_refuses():
    import torch
    z = torch.zeros(8)
    for bad in ([], [(z, z, z)]):
        with pytest.raises(ValueError):
            dion.AdamWPlan(bad)
    with pytest.raises(ValueError):
        dion.AdamWPlan([(z, z, z, z)])            # not on a GPU
    with pytest.raises(ValueError):
        dion.AdamWPlan([(z, z, z, z)], weight_decay=[0.1, 0.2])
    with pytest.raises(TypeError):
        dion.AdamWPlan([(z, z.double(), z, z)])


def test_constants_match_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "include", "dion.h")).read()
    assert int(re.search(r"#define DION_ADAMW_BLOCK (\d+)", text).group(1)) == dion.ADAMW_BLOCK
    assert ctypes.sizeof(dion.dion_adamw_tensor) == 56


def dither(index, seed):
    h = ((index.astype(np.uint64) + np.uint64(0x632be5ab * seed % 2 ** 32)) & np.uint64(0xffffffff))
    h = h * np.uint64(0x9e3779b1) & np.uint64(0xffffffff)
    h = (h ^ (h >> np.uint64(15))) * np.uint64(0x85ebca77) & np.uint64(0xffffffff)
    h = h ^ (h >> np.uint64(13))
    return (h & np.uint64(0xffff)).astype(float) / 65536, (h >> np.uint64(16)).astype(float) / 65536


@pytest.mark.parametrize("which", [0, 1])
def test_dither_is_uniform_and_uncorrelated(which):
    """Over the elements of one step, and over the steps of one element: mean
    1/2 and variance 1/12 of a uniform variable, and neighbours (in index, in
    step, and the two halves) without correlation.  With N = 2^18 samples the
    mean's standard error is 0.29 / 512 and a correlation's 1 / 512; bounds at
    five of those."""
    n = 1 << 18
    index = np.arange(n)
    rows = {"step": [dither(index, s) for s in (1, 2)],
            "element": [dither(np.full(n, i), 0) for i in (0, 1)]}
    seeds = np.arange(n, dtype=np.uint64)
    by_step = []
    for i in (0, 1):      # the same formula with the seed running
        h = (np.uint64(i) + seeds * np.uint64(0x632be5ab)) & np.uint64(0xffffffff)
        h = h * np.uint64(0x9e3779b1) & np.uint64(0xffffffff)
        h = (h ^ (h >> np.uint64(15))) * np.uint64(0x85ebca77) & np.uint64(0xffffffff)
        h = h ^ (h >> np.uint64(13))
        by_step.append(((h & np.uint64(0xffff)).astype(float) / 65536, (h >> np.uint64(16)).astype(float) / 65536))
    rows["element"] = by_step
    for name, (a, b) in rows.items():
        u, other = a[which], a[1 - which]
        assert abs(u.mean() - 0.5) < 5 * 0.29 / 512, name
        assert abs(u.var() - 1 / 12) < 5 / 512 / 6, name
        for x, y in ((u[1:], u[:-1]), (u, b[which]), (u, other)):
            assert abs(np.corrcoef(x, y)[0, 1]) < 5 / 512, name
