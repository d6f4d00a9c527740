"""The linear layer (GPU) against the same formulas in float64.

Tolerances (relative Frobenius error): bfloat16 outputs carry one rounding,
2^-8 of an element at most and 2^-9 in the root mean square (the sizes of one
element stay below that too with these seeds); dx and dw of an activation
carry the rounding of dz as well, another 2^-9 in the mean; float32 sums over K terms of exact products add sqrt(K) 2^-24
at the sizes here (below 2^-18).  float32 tensors: three-way split products,
3 * 2^-24 per product and the sums' roundings: 2^-19.  db is a float32 sum of
unrounded dz: 2^-18.
"""
import math

import pytest

from .gpuhelp import say

pytestmark = pytest.mark.gpu

ACTS = ("none", "relu", "relu2", "gelu", "silu")
TOL = {"bfloat16": 2.0 ** -9 + 2.0 ** -18, "float32": 2.0 ** -19}
TOL_GRAD = {"bfloat16": 2.0 ** -8 + 2.0 ** -18, "float32": 2.0 ** -19}


def act64(z, act):
    import torch
    if act == "relu":
        return torch.relu(z)
    if act == "relu2":
        return torch.relu(z) ** 2
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(-z / math.sqrt(2))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def rel(x, y):
    import torch
    n = float(torch.linalg.vector_norm(y))
    d = float(torch.linalg.vector_norm(x.double() - y))
    return d / n if n else d


def rand(shape, seed, dtype, pad=0, scale=1.0):
    """Seeded N(0, 1); pad: extra columns of pitch, filled with NaN."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)
    if not pad:
        return v
    big = torch.full((shape[0], shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    big[:, :shape[1]] = v
    return big[:, :shape[1]]


def forward_case(lib, t, k, n, dtype, act, bias, residual, keep, pad=0):
    import torch
    dt = getattr(torch, dtype)
    x, w = rand((t, k), 1, dt, pad), rand((n, k), 2, dt, pad, k ** -0.5)
    b = rand((n,), 3, torch.float32) if bias else None
    r = rand((t, n), 4, dt, pad) if residual else None
    y = rand((t, n), 5, dt, pad)
    z = rand((t, n), 6, dt, pad) if keep else None
    lib.linear_forward(x, w, y, bias=b, act=act, residual=r, preact=z)
    ez = x.double() @ w.double().T
    if bias:
        ez = ez + b.double()
    ey = act64(ez, act)
    if residual:
        ey = ey + r.double()
    assert rel(y, ey) <= TOL[dtype], (t, k, n, dtype, act)
    if keep:
        assert rel(z, ez) <= TOL[dtype]


# one token to several tiles; reductions of one element to several slices;
# odd sizes everywhere
SIZES = [(1, 1, 1), (1, 64, 64), (1, 3072, 1024), (3, 77, 50), (7, 130, 33), (8, 256, 300),
         (16, 640, 256), (17, 520, 264), (33, 1024, 136), (64, 200, 96), (65, 72, 64),
         (100, 1000, 200), (129, 136, 257), (300, 513, 129), (515, 64, 1025), (1025, 768, 520)]


@pytest.mark.parametrize("t,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_sizes(gpu_lib, t, k, n, dtype):
    say(f"linear forward {t} {k} {n} {dtype}")
    forward_case(gpu_lib, t, k, n, dtype, "none", False, False, False)
    forward_case(gpu_lib, t, k, n, dtype, "gelu", True, True, True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_activations(gpu_lib, act, dtype):
    for t in (5, 40, 200):
        say(f"linear act {act} {dtype} {t}")
        forward_case(gpu_lib, t, 192, 144, dtype, act, True, False, True)
        forward_case(gpu_lib, t, 192, 144, dtype, act, False, True, False)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_pitches(gpu_lib, pad, dtype):
    """Rows with NaN between them: nothing outside the tensors is used."""
    for t, k, n in ((1, 96, 40), (20, 96, 40), (140, 200, 160), (140, 201, 161)):
        say(f"linear pitch {t} {k} {n} {pad} {dtype}")
        forward_case(gpu_lib, t, k, n, dtype, "silu", True, True, True, pad)


def backward_case(lib, t, k, n, dtype, act, pad=0, accumulate=False):
    import torch
    dt = getattr(torch, dtype)
    x, w = rand((t, k), 1, dt, pad), rand((n, k), 2, dt, pad, k ** -0.5)
    dy = rand((t, n), 3, dt, pad)
    z = rand((t, n), 4, dt, pad) if act != "none" else None
    dx, dw, db = rand((t, k), 5, dt, pad), rand((n, k), 6, dt, pad), rand((n,), 7, torch.float32)
    w0, b0 = dw.double().clone(), db.double().clone()
    lib.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, act=act, preact=z, accumulate=accumulate)
    dz = dy.double()
    if z is not None:
        zz = z.double().requires_grad_(True)
        act64(zz, act).backward(dz)
        dz = zz.grad
    ew, eb = dz.T @ x.double(), dz.sum(0)
    if accumulate:
        ew, eb = ew + w0, eb + b0
    assert rel(dx, dz @ w.double()) <= TOL_GRAD[dtype], (t, k, n, dtype, act)
    assert rel(dw, ew) <= TOL_GRAD[dtype]
    assert rel(db, eb) <= 2.0 ** -18


@pytest.mark.parametrize("t,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_sizes(gpu_lib, t, k, n, dtype):
    say(f"linear backward {t} {k} {n} {dtype}")
    backward_case(gpu_lib, t, k, n, dtype, "none")
    backward_case(gpu_lib, t, k, n, dtype, "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_activations(gpu_lib, act, dtype):
    say(f"linear backward {act} {dtype}")
    backward_case(gpu_lib, 200, 144, 192, dtype, act)
    backward_case(gpu_lib, 200, 144, 192, dtype, act, accumulate=True)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_backward_pitches(gpu_lib, pad, dtype):
    for act in ("none", "silu"):
        for t, k, n in ((9, 96, 40), (140, 200, 160), (140, 201, 161)):
            say(f"linear backward pitch {t} {k} {n} {pad} {dtype} {act}")
            backward_case(gpu_lib, t, k, n, dtype, act, pad)


def test_parts_of_the_backward(gpu_lib):
    """dx, dw and db each alone give the bits they have together."""
    import torch
    x, w, dy = rand((130, 72), 1, torch.bfloat16), rand((96, 72), 2, torch.bfloat16), rand((130, 96), 3, torch.bfloat16)
    z = rand((130, 96), 4, torch.bfloat16)
    for act in ("none", "gelu"):
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(96, device="cuda")
        gpu_lib.linear_backward(dy, x, w, dx=dx, dw=dw, db=db, act=act, preact=z)
        dx2, dw2, db2 = torch.empty_like(x), torch.empty_like(w), torch.empty(96, device="cuda")
        gpu_lib.linear_backward(dy, weight=w, dx=dx2, act=act, preact=z)
        gpu_lib.linear_backward(dy, x, dw=dw2, act=act, preact=z)
        gpu_lib.linear_backward(dy, db=db2, act=act, preact=z)
        assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_no_tokens(gpu_lib, dtype):
    import torch
    dt = getattr(torch, dtype)
    x, w = torch.empty(0, 40, dtype=dt, device="cuda"), rand((24, 40), 2, dt)
    y = torch.empty(0, 24, dtype=dt, device="cuda")
    gpu_lib.linear_forward(x, w, y)
    dw, db = rand((24, 40), 3, dt), rand((24,), 4, torch.float32)
    keep_w, keep_b = dw.clone(), db.clone()
    gpu_lib.linear_backward(y, x, w, dx=torch.empty_like(x), dw=dw, db=db, accumulate=True)
    assert torch.equal(dw, keep_w) and torch.equal(db, keep_b)
    gpu_lib.linear_backward(y, x, w, dx=torch.empty_like(x), dw=dw, db=db)
    assert torch.count_nonzero(dw) == 0 and torch.count_nonzero(db) == 0


def test_residual_in_place_and_stream(gpu_lib):
    import torch
    x, w = rand((140, 96), 1, torch.bfloat16), rand((72, 96), 2, torch.bfloat16, scale=0.1)
    r = rand((140, 72), 3, torch.bfloat16)
    y, want = r.clone(), torch.empty_like(r)
    gpu_lib.linear_forward(x, w, want, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gpu_lib.linear_forward(x, w, y, residual=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)


def test_non_finite_stays_in_its_rows(gpu_lib):
    """A NaN or infinite token reaches its own row of y and dx only."""
    import torch
    for dtype in (torch.bfloat16, torch.float32):
        for t in (4, 40, 150):
            x, w = rand((t, 80), 1, dtype), rand((48, 80), 2, dtype)
            y = torch.empty(t, 48, dtype=dtype, device="cuda")
            x[1, 5], x[2, 7] = float("nan"), float("inf")
            gpu_lib.linear_forward(x, w, y)
            bad = ~torch.isfinite(y).all(1)
            assert bad.nonzero().flatten().tolist() == [1, 2]
            dy, dx = rand((t, 48), 3, dtype), torch.empty(t, 80, dtype=dtype, device="cuda")
            dy[3, 0] = float("nan")
            gpu_lib.linear_backward(dy, weight=w, dx=dx)
            assert (~torch.isfinite(dx).all(1)).nonzero().flatten().tolist() == [3]


def test_gradient_by_differences(gpu_lib):
    """<dL/dW, D> against the central difference of L(W) = <y, C> along D.
    float32, L in float64 from the layer's own y; step h = 2^-6: the
    difference's own error is h^2 / 6 of a third derivative of order one
    (4e-5) and 2^-23 / h (8e-6) of y's roundings."""
    import torch
    t, k, n = 70, 90, 50
    x, w, b = rand((t, k), 1, torch.float32), rand((n, k), 2, torch.float32, scale=k ** -0.5), rand((n,), 3, torch.float32)
    c, d = rand((t, n), 4, torch.float32), rand((n, k), 5, torch.float32, scale=k ** -0.5)
    for act in ("gelu", "silu", "none"):
        def loss(weight):
            y = torch.empty(t, n, device="cuda")
            gpu_lib.linear_forward(x, weight, y, bias=b, act=act)
            return float((y.double() * c.double()).sum())
        z, y = torch.empty(t, n, device="cuda"), torch.empty(t, n, device="cuda")
        gpu_lib.linear_forward(x, w, y, bias=b, act=act, preact=z)
        dw = torch.empty_like(w)
        gpu_lib.linear_backward(c, x, dw=dw, act=act, preact=z)
        h = 2.0 ** -6
        diff = (loss(w + h * d) - loss(w - h * d)) / (2 * h)
        scale = float(torch.linalg.vector_norm(dw.double()) * torch.linalg.vector_norm(d.double()))
        assert abs(float((dw.double() * d.double()).sum()) - diff) <= 1e-4 * scale


def test_repeats_are_equal_and_graphs_replay(gpu_lib):
    import torch
    x, w = rand((333, 520), 1, torch.bfloat16), rand((264, 520), 2, torch.bfloat16)
    dy = rand((333, 264), 3, torch.bfloat16)
    outs = [torch.empty_like(x), torch.empty_like(w), torch.empty(264, device="cuda")]
    ws = gpu_lib.linear_backward(dy, x, w, dx=outs[0], dw=outs[1], db=outs[2])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.linear_backward(dy, x, w, dx=outs[0], dw=outs[1], db=outs[2], workspace=ws)
    for rep in range(4):
        x.copy_(rand(x.shape, 10 + rep, torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        fresh = [torch.empty_like(o) for o in outs]
        gpu_lib.linear_backward(dy, x, w, dx=fresh[0], dw=fresh[1], db=fresh[2])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, fresh))


def test_large_tiles(gpu_lib):
    """Sizes that take the 256 x 256 tiles in every product, ragged at every
    edge."""
    for dtype in ("bfloat16", "float32"):
        t, k, n = 4104, 4136, 4120
        say(f"linear large {dtype}")
        forward_case(gpu_lib, t, k, n, dtype, "gelu", True, True, True)
        backward_case(gpu_lib, t, k, n, dtype, "silu")
