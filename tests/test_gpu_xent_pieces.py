"""The cross entropy over several pieces of the vocabulary (GPU) in each of its
forms: few tokens, float32 and bfloat16 tiles, copied operands, and the forward
where a launch would have too many threads.  Every case first shows that it has
several pieces: its workspace is smaller than what one piece would hold."""
import ctypes

import pytest

from .gpuhelp import say
from .test_gpu_xent import check_backward, check_forward, inputs, z_error

pytestmark = pytest.mark.gpu


def workspace(lib, name, x, w):
    """The call's, with both outputs."""
    import torch
    t, k = x.shape
    base = 1 << 44
    a = lib.dion_cross_entropy(t=t, n=w.shape[0], k=k, x=x.data_ptr(), ldx=x.stride(0), w=w.data_ptr(), ldw=w.stride(0),
                               target=base, loss=2 * base, lse=3 * base, dloss=4 * base, dx=5 * base, lddx=k, dw=6 * base,
                               lddw=k, ignore_index=-100, dtype=1 if x.dtype == torch.bfloat16 else 0)
    size = getattr(lib.load(), f"dion_cross_entropy_{name}_workspace_size")(ctypes.byref(a))
    assert size > 0
    return size


# tokens, inputs, vocabulary, type, pad, and the bytes per word that the backward
# holds of a piece: dz, and few tokens its transpose (padded to 32 or 64 tokens), in
# their planes; for W that is copied, its row
BACKWARD = [
    (11, 7, 1048576, "float32", 2, 6 * (11 + 32)), (32, 16, 1000003, "float32", 0, 6 * (32 + 32)),
    (64, 17, 600001, "bfloat16", 0, 4 * (64 + 64)), (64, 16, 600001, "bfloat16", 0, 4 * (64 + 64)),
    (40, 24, 900001, "bfloat16", 8, 4 * (40 + 64)), (33, 9, 1000001, "bfloat16", 3, 4 * (33 + 64)),
    (200, 8, 1000003, "float32", 0, 4 * 200), (3000, 33, 50001, "float32", 1, 4 * 3000),
    (1000, 16, 200001, "bfloat16", 0, 2 * 1024), (70, 4097, 100003, "bfloat16", 0, 2 * 4160),
]


@pytest.mark.parametrize("t,k,n,dtype,pad,row", BACKWARD)
def test_backward(gpu_lib, t, k, n, dtype, pad, row):
    x, w, y, dloss = inputs(t, k, n, dtype, pad)
    assert workspace(gpu_lib, "backward", x, w) < row * n
    say(f"cross entropy pieces {t} {k} {n} {dtype} {pad}")
    lse, _ = check_forward(gpu_lib, x, w, y, 0.1, 1e-3)
    check_backward(gpu_lib, x, w, y, dloss, lse, 0.1, 1e-3, pad=pad)
    check_backward(gpu_lib, x, w, y, dloss, lse, 0.1, 1e-3, pad=pad, accumulate=True)
    for which in ("dx", "dw"):
        check_backward(gpu_lib, x, w, y, dloss, lse, 0.1, 1e-3, pad=pad, which=which)


@pytest.mark.parametrize("t,k,n,pad", [(70, 4097, 70003, 0), (129, 8191, 40001, 1), (300, 4104, 66000, 3)])
@pytest.mark.parametrize("e", [0.0, 0.1])
def test_forward_of_copied_pieces(gpu_lib, t, k, n, pad, e):
    x, w, y, _ = inputs(t, k, n, "bfloat16", pad)
    assert workspace(gpu_lib, "forward", x, w) < 2 * n * k
    say(f"cross entropy forward pieces {t} {k} {n} {pad}")
    check_forward(gpu_lib, x, w, y, e, 1e-3)


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_forward_of_more_tiles_than_a_grid(gpu_lib, dtype):
    """2^20 tokens by 70001 words: more than 2^22 tiles of 128 x 128 (2^32 threads);
    the words from 65536 on are a piece of their own.  A sample of the tokens is
    compared, the first and the last of them included."""
    import torch
    t, k, n = 1 << 20, 8, 70001
    say(f"cross entropy forward {t} {k} {n} {dtype}")
    assert -(-t // 128) * -(-n // 128) > 1 << 22
    x, w, y, _ = inputs(t, k, n, dtype)
    loss, lse = (torch.full((t,), float("nan"), device="cuda") for _ in range(2))
    gpu_lib.cross_entropy_forward(x, w, y, loss, lse=lse)
    assert bool(torch.isfinite(loss).all()) and bool(torch.isfinite(lse).all())
    at = torch.cat([torch.arange(0, t, 1023, device="cuda"), torch.tensor([1, t - 1], device="cuda")])
    z = torch.mm(x[at].double(), w.double().t().contiguous())
    want = torch.logsumexp(z, 1)
    ys = y[at]
    wl = torch.where(ys != -100, want - z.gather(1, ys.clamp(min=0)[:, None])[:, 0], 0.0)
    dz = z_error(x, w) + 2.0 ** -21
    assert bool(((lse[at].double() - want).abs() <= dz + 2.0 ** -23 * (1 + want.abs())).all())
    assert bool(((loss[at].double() - wl).abs() <= 2 * dz + 2.0 ** -22 * (1 + wl.abs())).all())
