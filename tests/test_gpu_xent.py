"""The output head's cross entropy (GPU) against its formulas in float64.

Errors, with N = max ||x_t|| max ||w_j||, which bounds every partial sum of a
logit: bfloat16 products are exact and a matrix instruction adds 32 of them,
so a logit takes K / 32 roundings of 2^-24 N that add like a random walk;
float32 operands lose 3 2^-24 per product and take six times the instructions:
dz(K) = (sqrt(6 K / 32) + 4) 2^-24 N bounds both.  The exponentials add 2^-21
(two ulps, and the rounding of an argument up to 16; smaller terms do not
count), the sums and the final differences a few ulps of lse and of the loss.
Gradients, element by element: dz is off by its logit's error, by lse's given
rounding (none: lse is an input), by exp's 2^-21 and by its own rounding, half a
step of bfloat16 (2^-9) or of two or three planes (2^-17, 2^-25); an output by
the sum of |dz| |w| times that, by its sum's roundings in float32 and by its
own rounding (2^-9; the tie to half a step's end is 2^-8 of the smallest
mantissa: 2^-8 relative)."""
import math

import pytest

from .gpuhelp import say

pytestmark = pytest.mark.gpu

IGNORE = -100


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


def inputs(t, k, n, dtype, pad=0, ignored=0.2, seed=1, spread=2.0):
    import torch
    dt = getattr(torch, dtype)
    x, w = rand((t, k), seed, dt, pad), rand((n, k), seed + 1, dt, pad, spread * k ** -0.5)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    y = torch.randint(0, n, (t,), generator=g, device="cuda")
    if t > 2:
        y[0], y[-1], y[1] = 0, n - 1, n - 1      # the vocabulary's ends, one of them twice
        drop = torch.rand(t, generator=g, device="cuda") < ignored
        drop[0] = drop[-1] = drop[1] = False
        y = torch.where(drop, IGNORE, y)
    dloss = torch.rand(t, generator=g, device="cuda") / t + 0.1 / t
    return x, w, y, dloss


def z_error(x, w):
    import torch
    K = x.shape[1]
    N = float(torch.linalg.vector_norm(x.double(), dim=1).max()) * float(torch.linalg.vector_norm(w.double(), dim=1).max())
    return (math.sqrt(6 * K / 32) + 4) * 2.0 ** -24 * N


def reference(x, w, y, e, zc, lse=None, dloss=None, ignore=IGNORE):
    import torch
    z = torch.mm(x.double(), w.double().t().contiguous())
    taken = y != ignore
    at = y.clamp(min=0)[:, None]
    if dloss is None:
        lse = torch.logsumexp(z, 1)
        loss = lse - (1 - e) * z.gather(1, at)[:, 0] - e * z.mean(1) + zc * lse ** 2
        return torch.where(taken, loss, 0.0), lse
    lse = lse.double()[:, None]
    p = torch.exp(z - lse) * (1 + 2 * zc * lse)
    d = (dloss.double() * taken)[:, None]
    dz = d * (p - e / z.shape[1])
    dz.scatter_add_(1, at, -(1 - e) * d)
    size = d * (p + e / z.shape[1])          # terms' magnitudes: what errors are relative to
    size.scatter_add_(1, at, (1 - e) * d)
    return dz, size


def check_forward(lib, x, w, y, e=0.0, zc=0.0, want_loss=True, want_lse=True, ignore=IGNORE, **kw):
    import torch
    t = x.shape[0]
    loss = torch.full((t,), float("nan"), device="cuda") if want_loss else None
    lse = torch.full((t,), float("nan"), device="cuda") if want_lse else None
    ws = lib.cross_entropy_forward(x, w, y, loss, lse=lse, label_smoothing=e, z_loss=zc, ignore_index=ignore, **kw)
    eloss, else_ = reference(x, w, y, e, zc, ignore=ignore)
    dz = z_error(x, w) + 2.0 ** -21
    if want_lse:
        tol = dz + 2.0 ** -23 * (1 + else_.abs())
        assert bool(((lse.double() - else_).abs() <= tol).all()), float(((lse.double() - else_).abs() / tol).max())
    if want_loss:
        tol = 2 * dz + 2.0 ** -22 * (1 + eloss.abs()) + abs(zc) * (2 * else_.abs() * dz + 2.0 ** -21 * else_ ** 2)
        if e:     # the largest logit and the mean enter by their difference
            tol = tol + 2.0 ** -22 * else_.abs()
        d = (loss.double() - eloss).abs()
        assert bool((d <= tol).all()), float((d / tol).max())
        assert bool((loss[y == ignore] == 0).all())
    return lse, ws


def check_backward(lib, x, w, y, dloss, lse, e=0.0, zc=0.0, accumulate=False, pad=0, which="both", ignore=IGNORE, **kw):
    import torch
    t, k = x.shape
    n = w.shape[0]
    bf = x.dtype == torch.bfloat16
    dx = rand((t, k), 5, x.dtype, pad) if which != "dw" else None
    dw = rand((n, k), 6, x.dtype, pad) if which != "dx" else None
    w0 = dw.double().clone() if dw is not None else None
    ws = lib.cross_entropy_backward(dloss, x, w, y, lse, dx=dx, dw=dw, label_smoothing=e, z_loss=zc,
                                    accumulate=accumulate, ignore_index=ignore, **kw)
    dz, size = reference(x, w, y, e, zc, lse, dloss, ignore)
    # dz's rounding: half a step, at most 2^-8 of the value in one plane, 2^-16 in
    # the two that the header gives up to 32 tokens
    half = (2.0 ** -16 if t <= 32 else 2.0 ** -8) if bf else 2.0 ** -24
    err = dz.abs() * half + size * (z_error(x, w) + 2.0 ** -21 + 2.0 ** -22)
    out = 2.0 ** -8 if bf else 2.0 ** -24
    slip = size * (z_error(x, w) + 2.0 ** -21)
    def near(got, want, terms, worst, length, lost):
        tol = out * want.abs() + worst * 1.01 + terms * 2.0 ** -24 * (math.sqrt(6 * length / 32) + 8) + 1e-38
        d = (got.double() - want).abs()
        assert bool((d <= tol).all()), float((d / tol).max())
        # and as a whole: roundings add like a random walk.  dz is a difference of
        # terms of magnitude `size`: where they cancel (a vocabulary of one word has
        # p = 1 and dz = 0 but for lse's rounding) what is left is their error, which
        # is relative to them
        norm = float(torch.linalg.vector_norm(want))
        if norm and want.numel() > 1000:
            whole = (2.0 ** -8 if bf else 2.0 ** -20) * norm
            assert float(torch.linalg.vector_norm(got.double() - want)) <= whole + 2 * float(torch.linalg.vector_norm(lost))
    if dx is not None:
        wd, wa = w.double(), w.double().abs()
        near(dx, torch.mm(dz, wd), torch.mm(dz.abs(), wa), torch.mm(err, wa), n, torch.mm(slip, wa))
        assert not bool(dx[y == ignore].any())
    if dw is not None:
        dzt, xd = dz.t().contiguous(), x.double()
        want, terms = torch.mm(dzt, xd), torch.mm(dzt.abs(), xd.abs())
        worst = torch.mm(err.t().contiguous(), xd.abs())
        if accumulate:
            want, terms = want + w0, terms + w0.abs()
        near(dw, want, terms, worst, t, torch.mm(slip.t().contiguous(), xd.abs()))
    return ws


def both(lib, t, k, n, dtype, e=0.0, zc=0.0, pad=0, **kw):
    x, w, y, dloss = inputs(t, k, n, dtype, pad)
    lse, _ = check_forward(lib, x, w, y, e, zc)
    check_backward(lib, x, w, y, dloss, lse, e, zc, pad=pad, **kw)


# one token to several tiles, vocabularies of one word to several tiles, odd
# sizes everywhere; rows, skinny products, tiles of both sizes, cut tiles
SIZES = [(1, 1, 1), (1, 64, 1), (1, 3, 2), (1, 64, 1000), (2, 65, 17), (4, 130, 33), (8, 256, 300), (9, 64, 63),
         (16, 640, 255), (17, 520, 1030), (32, 512, 65), (33, 1024, 136), (64, 200, 2001), (65, 72, 64), (65, 8, 1),
         (100, 1000, 300), (127, 136, 129), (129, 264, 257), (300, 513, 1030), (515, 64, 4097), (1025, 768, 520),
         (200, 2048, 130)]


@pytest.mark.parametrize("t,k,n", SIZES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_sizes(gpu_lib, t, k, n, dtype):
    say(f"cross entropy {t} {k} {n} {dtype}")
    both(gpu_lib, t, k, n, dtype)
    both(gpu_lib, t, k, n, dtype, 0.1, 1e-2)


@pytest.mark.parametrize("t,k,n,dtype", [(4200, 64, 8200, "bfloat16"), (4097, 200, 4100, "bfloat16"),
                                         (2050, 96, 8300, "float32")])
def test_large_tiles(gpu_lib, t, k, n, dtype):
    say(f"cross entropy large {t} {k} {n} {dtype}")
    both(gpu_lib, t, k, n, dtype)
    both(gpu_lib, t, k, n, dtype, 0.05, -1e-3)


@pytest.mark.parametrize("t,k,n,dtype", [(8192, 64, 33000, "bfloat16"), (8200, 72, 17001, "bfloat16"),
                                         (8192, 40, 11001, "float32"), (70, 8192, 11000, "float32"),
                                         (4100, 63, 40000, "bfloat16")])
def test_pieces(gpu_lib, t, k, n, dtype):
    """Several pieces of the vocabulary, the last one short."""
    say(f"cross entropy pieces {t} {k} {n} {dtype}")
    both(gpu_lib, t, k, n, dtype, 0.1)
    both(gpu_lib, t, k, n, dtype, accumulate=True)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_pitches(gpu_lib, pad, dtype):
    """Rows with NaN between them: nothing outside the tensors is used."""
    for t, k, n in ((1, 96, 40), (7, 97, 41), (20, 96, 40), (140, 200, 160), (140, 201, 161)):
        say(f"cross entropy pitch {t} {k} {n} {pad} {dtype}")
        both(gpu_lib, t, k, n, dtype, 0.1, 1e-3, pad)


@pytest.mark.parametrize("t", [5, 40, 300])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_outputs_one_by_one(gpu_lib, t, dtype):
    x, w, y, dloss = inputs(t, 72, 130, dtype)
    check_forward(gpu_lib, x, w, y, want_loss=False)
    check_forward(gpu_lib, x, w, y, want_lse=False)
    lse, _ = check_forward(gpu_lib, x, w, y)
    for which in ("dx", "dw"):
        check_backward(gpu_lib, x, w, y, dloss, lse, which=which)
    check_backward(gpu_lib, x, w, y, dloss, lse, accumulate=True)
    # a word of the vocabulary as the ignored target
    check_forward(gpu_lib, x, w, torch_where_ignored(y), ignore=3)
    check_backward(gpu_lib, x, w, torch_where_ignored(y), dloss, lse, ignore=3)


def torch_where_ignored(y):
    import torch
    return torch.where(y == IGNORE, 3, y)


@pytest.mark.parametrize("t", [3, 30, 200])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_masked_and_bad_rows(gpu_lib, t, dtype):
    """All rows ignored; a logit that is not finite in an ignored row; targets
    outside the vocabulary."""
    import torch
    k, n = 64, 150
    x, w, y, dloss = inputs(t, k, n, dtype, ignored=0.0)
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    none = torch.full_like(y, IGNORE)
    gpu_lib.cross_entropy_forward(x, w, none, loss, lse=lse)
    gpu_lib.cross_entropy_backward(dloss, x, w, none, lse, dx=dx, dw=dw)
    assert not bool(loss.any()) and not bool(dx.any()) and not bool(dw.any())
    assert bool(torch.isfinite(lse).all())
    # an ignored row of infinities and NaN: its loss and dx are zero, other rows as without it
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse)
    gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dx=dx)
    l0, d0 = loss.clone(), dx.clone()
    bad, yb = x.clone(), y.clone()
    bad[1, 0], bad[1, 5], yb[1] = math.nan, math.inf, IGNORE
    gpu_lib.cross_entropy_forward(bad, w, yb, loss, lse=lse)
    gpu_lib.cross_entropy_backward(dloss, bad, w, yb, lse, dx=dx)
    assert float(loss[1]) == 0 and not bool(dx[1].any())
    keep = torch.arange(t, device="cuda") != 1
    assert torch.equal(loss[keep], l0[keep]) and torch.equal(dx[keep], d0[keep])
    # not ignored: NaN, in that row
    gpu_lib.cross_entropy_forward(bad, w, y, loss, lse=lse)
    assert bool(torch.isnan(loss[1])) and torch.equal(loss[keep], l0[keep])
    for wrong in (n, -1, 1 << 40, -(1 << 62)):
        yb = y.clone()
        yb[1] = wrong
        gpu_lib.cross_entropy_forward(x, w, yb, loss, lse=lse)
        gpu_lib.cross_entropy_backward(dloss, x, w, yb, lse, dx=dx)
        assert bool(torch.isnan(loss[1])) and torch.equal(loss[keep], l0[keep])
        assert bool(torch.isnan(dx[1]).all()) and torch.equal(dx[keep], d0[keep])


@pytest.mark.parametrize("t", [6, 50, 260])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_range_of_logits(gpu_lib, t, dtype):
    """Logits of hundreds (a shift would overflow exp), all equal, and one that
    carries all of the probability: a loss of exp(-30) keeps its digits."""
    import torch
    k, n = 64, 700
    x, w, y, dloss = inputs(t, k, n, dtype, spread=200.0)
    lse, _ = check_forward(gpu_lib, x, w, y)
    check_backward(gpu_lib, x, w, y, dloss, lse)
    z = torch.zeros_like(x)
    lse, _ = check_forward(gpu_lib, z, w, y)
    check_backward(gpu_lib, z, w, y, dloss, lse)
    x.zero_(), w.zero_()
    x[:, 3] = 30.0
    y.fill_(699)
    w[699, 3] = 1.0
    loss = torch.empty(t, device="cuda")
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse)
    # log(1 + s) with s = 699 exp(-30) = 6.5e-11, below float32's step at 1: the sum
    # of 700 terms is 1 and the loss 0, where lse - z_y would be off by up to 2e-6
    assert float(loss.abs().max()) <= 699 * math.exp(-30) * 1.01
    x[:, 3] = 12.0
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse)
    want = math.log1p(699 * math.exp(-12))
    assert float((loss - want).abs().max()) <= 700 / 64 * 2.0 ** -24 + 2.0 ** -20 * want


@pytest.mark.parametrize("e,zc", [(0.0, 0.0), (0.2, 0.0), (0.1, 1e-2)])
def test_gradient_against_differences(gpu_lib, e, zc):
    """Central differences of the summed loss along random directions.  The
    losses are off by 2^-20 each, 2^-20 sqrt(t) in the sum, over a distance of 2h;
    the differences' own error is h^2 / 6 times the third derivative along the
    direction, below sum_t dloss |dz|_max^3 with |dz| < 8 h-units here."""
    import torch
    t, k, n, h = 90, 64, 210, 2.0 ** -7
    x, w, y, dloss = inputs(t, k, n, "float32")
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse, label_smoothing=e, z_loss=zc)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dx=dx, dw=dw, label_smoothing=e, z_loss=zc)
    u, v = rand((t, k), 21, torch.float32, scale=k ** -0.5), rand((n, k), 22, torch.float32, scale=k ** -0.5)
    def total(a, b):
        gpu_lib.cross_entropy_forward(x + a * u, w + b * v, y, loss, label_smoothing=e, z_loss=zc)
        return float((loss.double() * dloss.double()).sum())
    noise = 2.0 ** -20 * float(torch.linalg.vector_norm(dloss)) * 8 / h
    third = h * h / 6 * float(dloss.sum()) * 8 ** 3
    for a, b, want in ((h, 0.0, float((dx.double() * u.double()).sum())), (0.0, h, float((dw.double() * v.double()).sum()))):
        got = (total(a, b) - total(-a, -b)) / (2 * h)
        assert abs(got - want) <= noise + third, (got, want, noise, third)
        assert abs(want) > 4 * (noise + third) or abs(got - want) < 0.3 * abs(want) + noise


@pytest.mark.parametrize("t,k,n,dtype", [(5, 72, 300, "float32"), (20, 72, 300, "bfloat16"), (300, 520, 1000, "bfloat16"),
                                         (300, 77, 1000, "float32")])
def test_same_bits_streams_and_graphs(gpu_lib, t, k, n, dtype):
    """Workspaces of any content; another stream; two captured graphs that share
    a workspace, replayed in turn with eager work between."""
    import torch
    x, w, y, dloss = inputs(t, k, n, dtype)
    def fresh():
        return (torch.empty(t, device="cuda"), torch.empty(t, device="cuda"), torch.empty_like(x), torch.empty_like(w))
    def step(o, ws1=None, ws2=None, stream=None):
        a = gpu_lib.cross_entropy_forward(x, w, y, o[0], lse=o[1], label_smoothing=0.1, workspace=ws1, stream=stream)
        b = gpu_lib.cross_entropy_backward(dloss, x, w, y, o[1], dx=o[2], dw=o[3], label_smoothing=0.1, workspace=ws2,
                                           stream=stream)
        return a, b
    first = fresh()
    ws = step(first)
    for u in ws:
        u.fill_(0xff)
    again = fresh()
    step(again, *ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = fresh()
    step(other, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for a, b, c in zip(first, again, other):
        assert torch.equal(a, b) and torch.equal(a, c)
    graphs, outs = [], []
    shared = torch.empty(max(u.numel() for u in ws), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        g, o = torch.cuda.CUDAGraph(), fresh()
        with torch.cuda.graph(g):
            step(o, shared, shared)
        graphs.append(g)
        outs.append(o)
    for turn in range(3):
        for g, o in zip(graphs, outs):
            for a in o:
                a.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(first, o):
                assert torch.equal(a, b), turn
        step(again, *ws)


def test_rows_behind_the_last_stay(gpu_lib):
    """Outputs in larger buffers: nothing past the last row, nor between rows."""
    import torch
    for dtype in ("bfloat16", "float32"):
        for t in (3, 33, 130):
            k, n = 72, 140
            x, w, y, dloss = inputs(t, k, n, dtype)
            lse, _ = check_forward(gpu_lib, x, w, y)
            bx = torch.full((t + 3, k + 8), 7.0, dtype=x.dtype, device="cuda")
            bw = torch.full((n + 3, k + 8), 7.0, dtype=x.dtype, device="cuda")
            bl = torch.full((t + 5,), 7.0, device="cuda")
            gpu_lib.cross_entropy_forward(x, w, y, bl[1:t + 1], lse=None)
            gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dx=bx[:t, :k], dw=bw[:n, :k])
            for b, m in ((bx, t), (bw, n)):
                assert bool((b[m:] == 7).all()) and bool((b[:, k:] == 7).all())
            assert bool((bl[t + 1:] == 7).all()) and float(bl[0]) == 7


def test_no_tokens(gpu_lib):
    import torch
    for dtype in (torch.bfloat16, torch.float32):
        x, w = torch.empty(0, 64, dtype=dtype, device="cuda"), rand((300, 64), 1, dtype)
        y, l = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda")
        gpu_lib.cross_entropy_forward(x, w, y, l, lse=l)
        dx, dw = torch.empty_like(x), torch.full_like(w, math.nan)
        gpu_lib.cross_entropy_backward(l, x, w, y, l, dx=dx, dw=dw)
        assert not bool(dw.any())
        dw.fill_(3.0)
        gpu_lib.cross_entropy_backward(l, x, w, y, l, dx=dx, dw=dw, accumulate=True)
        assert bool((dw == 3).all())


def test_offsets_past_32_bits(gpu_lib):
    """A weight of more than 2^31 elements, its last rows hit."""
    import torch
    n, k, t = (1 << 19) + 77, 4104, 70
    w = torch.zeros(n, k, dtype=torch.bfloat16, device="cuda")
    w[-50:] = rand((50, k), 3, torch.bfloat16, scale=4 * k ** -0.5)
    x = rand((t, k), 4, torch.bfloat16)
    y = n - 1 - torch.arange(t, device="cuda") % 50
    loss, lse = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
    dloss = torch.full((t,), 1.0 / t, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    for rows in (t, 30):     # tiles, skinny products
        a = slice(0, rows)
        gpu_lib.cross_entropy_forward(x[a], w, y[a], loss[a], lse=lse[a])
        gpu_lib.cross_entropy_backward(dloss[a], x[a], w, y[a], lse[a], dx=dx[a], dw=dw)
        z = torch.mm(x[a].double(), w[-50:].double().t().contiguous())
        els = torch.log(torch.exp(z).sum(1) + (n - 50))
        assert torch.allclose(lse[a].double(), els, rtol=1e-6, atol=1e-5)
        hit = z.gather(1, (y[a] - (n - 50))[:, None])[:, 0]
        assert torch.allclose(loss[a].double(), els - hit, rtol=1e-5, atol=1e-5)
        dz = torch.exp(z - els[:, None])
        dz.scatter_add_(1, (y[a] - (n - 50))[:, None], -torch.ones(rows, 1, dtype=torch.float64, device="cuda"))
        dz /= t
        want = torch.mm(dz.t().contiguous(), x[a].double())
        assert float(torch.linalg.vector_norm(dw[-50:].double() - want) / torch.linalg.vector_norm(want)) < 2.0 ** -7
        rest = torch.exp(-els) / t
        want = torch.mm(rest[None], x[a].double())[0]
        got = dw[12345].double()
        assert float(torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want)) < 2.0 ** -7
        want = torch.mm(dz, w[-50:].double())
        assert float(torch.linalg.vector_norm(dx[a].double() - want) / torch.linalg.vector_norm(want)) < 2.0 ** -7


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_more_tiles_than_a_launch(gpu_lib, dtype):
    """2^20 tokens on 65836 words: the forward pass takes the vocabulary in pieces."""
    import torch
    t, k, n = 1 << 20, 8, 65836
    say("cross entropy, many tiles", t, k, n, dtype)
    x, w, y, _ = inputs(t, k, n, dtype)
    loss = torch.full((t,), float("nan"), device="cuda")
    lse = torch.full_like(loss, float("nan"))
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse, ignore_index=IGNORE)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())
    some = torch.cat([torch.arange(0, t, 20011, device="cuda"), torch.arange(t - 5, t, device="cuda")])
    dz = z_error(x[some], w) + 2.0 ** -21
    eloss, else_ = reference(x[some], w, y[some], 0.0, 0.0)
    assert bool(((lse[some].double() - else_).abs() <= dz + 2.0 ** -23 * (1 + else_.abs())).all())
    assert bool(((loss[some].double() - eloss).abs() <= 2 * dz + 2.0 ** -22 * (1 + eloss.abs())).all())


def test_binding_refuses(gpu_lib):
    import torch
    x, w, y, dloss = inputs(4, 16, 20, "float32")
    f = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        gpu_lib.cross_entropy_forward(x, w, y.int(), f)
    with pytest.raises(TypeError):
        gpu_lib.cross_entropy_forward(x, w.bfloat16(), y, f)
    with pytest.raises(ValueError):
        gpu_lib.cross_entropy_forward(x, w, y[:3], f)
    with pytest.raises(ValueError):
        gpu_lib.cross_entropy_forward(x, w[:, :8], y, f)
    with pytest.raises(TypeError):
        gpu_lib.cross_entropy_forward(x, w, y, f.double())
    with pytest.raises(gpu_lib.DionError):
        gpu_lib.cross_entropy_forward(x, w, y)
    with pytest.raises(gpu_lib.DionError):
        gpu_lib.cross_entropy_forward(x, w, y, f, label_smoothing=1.5)
    with pytest.raises(ValueError):
        gpu_lib.cross_entropy_backward(dloss, x, w, y, f, dx=torch.empty(4, 8, device="cuda"))
    with pytest.raises(ValueError):
        gpu_lib.cross_entropy_forward(x, w, y, f, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
