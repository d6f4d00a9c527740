"""AdamWPlan keeps the memory of its tensors for as long as it lives (without a
GPU): a step after ``X.data`` or ``X.set_`` replaced a tensor's storage would
otherwise write to memory that has been handed out again."""
import gc
import weakref

import numpy as np
import pytest

import rank_orthonormalized_optimizer_dion_amd as dion


def on_gpu(a):
    """A tensor over the numpy array a that the checks take for a GPU tensor."""
    import torch

    class Fake(torch.Tensor):
        is_cuda = property(lambda self: True)

    return torch.Tensor._make_subclass(Fake, torch.from_numpy(a))


@pytest.mark.parametrize("how", ["data", "set", "drop"])
@pytest.mark.parametrize("which", range(4))
def test_memory_outlives_the_tensors_storage(how, which):
    import torch
    arrays = [np.full(16, i, np.float32) for i in range(4)]
    refs = [weakref.ref(a) for a in arrays]
    address = [a.ctypes.data for a in arrays]
    tensors = [on_gpu(a) for a in arrays]
    plan = dion.AdamWPlan([tuple(tensors)])
    row = plan._table[0]
    assert [row.X, row.G, row.M, row.V] == address
    if how == "data":
        tensors[which].data = on_gpu(np.zeros(16, np.float32))
    elif how == "set":
        with torch.no_grad():
            tensors[which].set_(torch.zeros(16))
    if how != "drop":
        assert tensors[which].data_ptr() != address[which]
    del arrays, tensors
    gc.collect()
    assert all(r() is not None for r in refs)
    del plan, row
    gc.collect()
    assert all(r() is None for r in refs)


def test_one_call_keeps_nothing(monkeypatch):
    """adamw_step_batched needs its tensors only until it returns: it makes no
    object per tensor (lists have hundreds of them)."""
    import torch
    made = []
    for name in ("detach", "untyped_storage"):
        monkeypatch.setattr(torch.Tensor, name, lambda t, old=getattr(torch.Tensor, name): made.append(t) or old(t))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    a = [np.zeros(16, np.float32) for _ in range(4)]
    refs = [weakref.ref(v) for v in a]
    stream = type("Stream", (), {"cuda_stream": 0})
    with pytest.raises(dion.DionError):     # step number 0 is refused before any launch
        dion.adamw_step_batched([tuple(on_gpu(v) for v in a)], 1e-3, 0, stream=stream)
    assert not made
    del a
    gc.collect()
    assert all(r() is None for r in refs)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_steps_after_other_memory(gpu_lib, bits):
    """The plan goes on with its own memory: the tensors that replaced it, and
    those that are allocated later, stay as they are."""
    import torch
    n = 5000
    X, G = torch.randn(n, device="cuda"), torch.randn(n, device="cuda")
    state = (torch.zeros_like(X), torch.zeros_like(X)) if bits == 32 else gpu_lib.adamw_state8(X)
    before, old = X.clone(), X.data_ptr()
    plan = gpu_lib.AdamWPlan([(X, G) + tuple(state)])
    del state
    X.data = torch.full((n,), 5.0, device="cuda")
    later = [torch.full((n,), 3.0, device="cuda") for _ in range(8)]
    assert old not in [t.data_ptr() for t in later]
    plan.step(0.1, 1)
    assert bool((X == 5.0).all()) and all(bool((t == 3.0).all()) for t in later)
    stepped = torch.empty(0, device="cuda").set_(plan._memory[0])
    assert torch.allclose(before - stepped[:n], 0.1 * G.sign(), rtol=1e-3, atol=1e-6)
