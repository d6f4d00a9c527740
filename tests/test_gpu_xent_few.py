"""The cross entropy of few tokens (GPU): its own kernels up to 32 tokens (64
where the tiles would need copies of x and W), on both sides of each of their block
sizes, at every alignment, with short and long vocabularies and reductions.
Same checks and tolerances as the other sizes."""
import pytest

from .gpuhelp import say
from .test_gpu_xent import both, check_backward, check_forward, inputs, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 31, 32, 33, 48, 63, 64, 65, 96, 97, 127, 128, 129])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_tokens(gpu_lib, t, dtype):
    for k, n in ((64, 97), (200, 1000), (777, 301), (1030, 64)):
        say(f"few tokens {t} {k} {n} {dtype}")
        both(gpu_lib, t, k, n, dtype, 0.1, 1e-3)


@pytest.mark.parametrize("k", [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 127, 129, 511, 513, 4103])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_reductions(gpu_lib, k, dtype):
    for t, n in ((3, 40), (20, 129), (50, 33)):
        say(f"few tokens reduction {t} {k} {n} {dtype}")
        both(gpu_lib, t, k, n, dtype)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 65, 127, 128, 129, 255, 257, 16383, 16385, 40001])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_vocabularies(gpu_lib, n, dtype):
    for t, k in ((1, 72), (30, 100), (64, 64)):
        say(f"few tokens vocabulary {t} {k} {n} {dtype}")
        both(gpu_lib, t, k, n, dtype, 0.05)


@pytest.mark.parametrize("pad", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_alignment(gpu_lib, pad, dtype):
    """Rows at every offset, NaN between them; accumulated too."""
    for t, k, n in ((1, 130, 65), (33, 129, 65), (64, 72, 200)):
        say(f"few tokens pitch {pad} {t} {dtype}")
        both(gpu_lib, t, k, n, dtype, pad=pad)
        both(gpu_lib, t, k, n, dtype, pad=pad, accumulate=True)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_last_row_of_the_weight_not_finite(gpu_lib, dtype):
    """Blocks past the vocabulary's end re-read its last row: what they make of
    it is dropped also where that row is not finite (all tokens ignored: dz is
    zero, and only that row's own products with it are NaN in dx)."""
    import torch
    t, k, n = 20, 96, 65
    x, w, y, dloss = inputs(t, k, n, dtype, ignored=0.0)
    loss, lse = torch.empty(t, device="cuda"), torch.zeros(t, device="cuda")
    dw = torch.empty_like(w)
    w[n - 1, 3] = float("inf")
    y.fill_(-100)
    gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dw=dw)
    assert not bool(dw.any())
    v = w.clone()
    w[n - 1] = 0
    dx = torch.empty_like(x)
    gpu_lib.cross_entropy_backward(dloss, x, w, y, lse, dx=dx)
    assert not bool(dx.any())
    # a piece of the vocabulary that ends before a row that is not finite
    gpu_lib.cross_entropy_forward(x, v[:n - 1], y, loss, lse=lse)
    assert bool(torch.isfinite(lse).all())
    gpu_lib.cross_entropy_backward(dloss, x, v[:n - 1], y, lse, dx=dx)
    assert not bool(dx.any())


@pytest.mark.parametrize("t", [4, 5, 16, 17, 32])
@pytest.mark.parametrize("n", [16384, 17001, 32000])
@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_rows_per_workgroup(gpu_lib, t, n, dtype):
    """Both sides of the vocabularies and tokens that share W's rows differently,
    widths that end inside a workgroup's columns."""
    say(f"cross entropy few, rows {t} {n} {dtype}")
    both(gpu_lib, t, 200, n, dtype, 0.1)
    both(gpu_lib, t, 131, n, dtype)


@pytest.mark.parametrize("t,k,n,dtype", [(3, 4100, 17000, "float32"), (20, 2050, 33000, "float32"), (4, 4097, 33000, "bfloat16"),
                                         (13, 4104, 33000, "bfloat16"), (50, 4097, 33000, "bfloat16")])
def test_weights_larger_than_the_caches(gpu_lib, t, k, n, dtype):
    say(f"cross entropy few, large weight {t} {k} {n} {dtype}")
    both(gpu_lib, t, k, n, dtype, 0.1)


def test_long_vocabulary_in_pieces(gpu_lib):
    """dz of 128 tokens in three planes, by rows and transposed, is bounded by
    pieces of the vocabulary."""
    say("few tokens pieces")
    x, w, y, dloss = inputs(128, 16, 400003, "float32")
    lse, _ = check_forward(gpu_lib, x, w, y)
    check_backward(gpu_lib, x, w, y, dloss, lse)
