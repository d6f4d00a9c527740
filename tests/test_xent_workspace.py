"""The cross entropy's workspace (CPU: size queries) against the bounds that the
header states, over the whole range of sizes, types and alignments."""
import ctypes
import math
import random

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

MiB = 1 << 20
X, WT, Y, L, E, D, DX, DW = (k << 44 for k in range(1, 9))


def size(name, t, n, k, pad, dtype, smoothing=0.0, dx=True, dw=True):
    ld = k + pad
    a = dion.dion_cross_entropy(t=t, n=n, k=k, x=X, ldx=ld, w=WT, ldw=ld, target=Y, loss=L, lse=E, dloss=D,
                                dx=DX if dx else None, lddx=ld, dw=DW if dw else None, lddw=ld, ignore_index=-100,
                                label_smoothing=smoothing, dtype=dtype)
    got = getattr(dion.load(), f"dion_cross_entropy_{name}_workspace_size")(ctypes.byref(a))
    assert got > 0
    return got


def copies(t, k):
    """x and a piece of W, padded to whole stages and cells."""
    kp = -(-k // 64) * 64
    return 2 * (t + 31) * kp + max(256 * MiB, 256 * 2 * kp)


def backward_bound(t, n, k, pad, dtype):
    if t <= (64 if dtype else 32):
        return (256 + 64) * MiB + 1024 * (k + 63)
    dz = max(256 * MiB, 256 * (2 * (t + 31) if dtype else 4 * t))
    return dz + 200 * MiB + (4 * t * k + copies(t, k) if dtype else 0)


def forward_bound(t, n, k, pad, dtype, smoothing):
    per = 12 if smoothing else 8
    if t <= (64 if dtype else 32):
        few = per * t * min(-(-n // 16), 1024) + 1024 * (k + 63)
    else:
        few = 0
    tiles = per * t * (n / 64 + 5) + 4 * t + 70 * MiB + (copies(t, k) if dtype else 0)
    return max(few, tiles)


def cases():
    rng = random.Random(5)
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    for _ in range(6000):
        t, n, k = log_int(1, 1 << 24), log_int(1, 1 << 20), log_int(1, 1 << 20)
        if rng.random() < 0.5:
            k = min(-(-k // 64) * 64, 1 << 20)
        if (t + n) * (k + 8) < 1 << 40:      # more than any memory
            yield t, n, k, rng.choice((0, 0, 1, 8)), rng.choice((0, 1))
    for t in (1, 32, 33, 64, 65, 1 << 18, 1 << 19, 1 << 24):
        for n in (1, 255, 257, 1 << 20):
            for k in (1, 64, 4097, (1 << 18) + 1, 1 << 20):
                if (t + n) * k < 1 << 40:
                    for dtype in (0, 1):
                        yield t, n, k, 0, dtype


def test_backward_is_bounded():
    for case in cases():
        got, bound = size("backward", *case), backward_bound(*case)
        assert got <= bound, (case, got / bound)


@pytest.mark.parametrize("smoothing", [0.0, 0.1])
def test_forward_is_bounded(smoothing):
    for case in cases():
        got, bound = size("forward", *case, smoothing), forward_bound(*case, smoothing)
        assert got <= bound, (case, got / bound)


def test_narrow_pieces_keep_an_eighth_of_a_byte_per_logit():
    """Copied pieces of 256 words (2^20 + 1 inputs are too many; 2^20 - 1 are not):
    the columns of statistics are still one per 64 words."""
    t, n, k = 1 << 16, 1 << 16, (1 << 20) - 1
    assert size("forward", t, n, k, 0, 1) <= t * n / 8 + 2 * (t + 31) * (k + 1) + (512 + 70) * MiB + 64 * t


def test_what_grows_and_what_does_not():
    """Beyond a piece of the vocabulary the backward's workspace stays as it is."""
    for t, k, pad, dtype, n in ((8192, 4096, 0, 1, 1 << 17), (8192, 4096, 0, 0, 1 << 17), (100, 4097, 1, 1, 1 << 18)):
        assert size("backward", t, 2 * n, k, pad, dtype) <= size("backward", t, n, k, pad, dtype) + MiB
