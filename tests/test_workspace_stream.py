"""A workspace that the binding allocates for a call on another stream than the
current one comes from that stream's own memory (without a GPU: torch's
allocator is a recorder).

Memory taken from the current stream's pool may still be in use by work pending
there, which nothing orders before the other stream's kernels."""
import contextlib
import types

import pytest

import rank_orthonormalized_optimizer_dion_amd as dion

MAIN, SIDE = types.SimpleNamespace(cuda_stream=1), types.SimpleNamespace(cuda_stream=2)
DEVICE = types.SimpleNamespace(index=0)


class Buffer:
    device = DEVICE

    def __init__(self, nbytes, stream):
        self.nbytes, self.stream = nbytes, stream

    def data_ptr(self):
        return 1 << 40

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1

    def record_stream(self, stream):
        pass


class Cuda:
    def __init__(self):
        self.now = MAIN

    def current_stream(self, device=None):
        return self.now

    def current_device(self):
        return 0

    @contextlib.contextmanager
    def stream(self, stream):
        old, self.now = self.now, stream if stream is not None else self.now
        try:
            yield
        finally:
            self.now = old


class Torch:
    uint8 = "uint8"

    def __init__(self):
        self.cuda, self.made = Cuda(), []

    def empty(self, nbytes, dtype=None, device=None):
        self.made.append(Buffer(nbytes, self.cuda.now))
        return self.made[-1]


@pytest.fixture
def torch(monkeypatch):
    fake = Torch()
    monkeypatch.setattr(dion, "_torch", lambda: fake)
    return fake


@pytest.mark.parametrize("stream,where", [(None, MAIN), (MAIN, MAIN), (SIDE, SIDE)])
def test_training_operators(torch, stream, where):
    seen = []
    ws = dion._launch(lambda: 640, lambda p, nbytes, st: seen.append((p, nbytes, st)) or dion.OK,
                      DEVICE, None, stream)
    assert torch.made == [ws] and ws.stream is where
    assert seen == [(ws.data_ptr(), 640, where.cuda_stream)]
    assert torch.cuda.now is MAIN
    # a workspace that is handed in is used as it is
    assert dion._launch(lambda: 640, lambda *a: dion.OK, DEVICE, ws, stream) is ws
    assert len(torch.made) == 1


@pytest.mark.parametrize("stream,where", [(None, MAIN), (SIDE, SIDE)])
@pytest.mark.parametrize("call", ["step", "step_batched", "plan"])
def test_optimizer_step(torch, monkeypatch, call, stream, where):
    class Lib:
        dion_workspace_size = dion_workspace_size_batched = dion_plan_workspace_size = \
            staticmethod(lambda *a: 640)
        dion_step = dion_step_batched = dion_plan_create = staticmethod(lambda *a: dion.OK)
        dion_plan_destroy = staticmethod(lambda h: None)

    mat = types.SimpleNamespace(device=DEVICE, data_ptr=lambda: 1 << 20)
    monkeypatch.setattr(dion, "load", lambda: Lib)
    monkeypatch.setattr(dion, "_check", lambda X, G, R, V: (8, 8, 4))
    monkeypatch.setattr(dion, "_gdtype", lambda G: 0)
    if call == "step":
        ws = dion.step(mat, mat, mat, mat, 0.1, 0.9, stream=stream)
    elif call == "step_batched":
        ws = dion.step_batched([(mat,) * 4], 0.1, 0.9, stream=stream)
    else:
        ws = dion.Plan([(mat,) * 4]).new_workspace(stream)
    assert ws.stream is where and torch.cuda.now is MAIN


@pytest.mark.gpu
def test_on_the_gpu(gpu_lib):
    """The allocator's own record: the block belongs to the call's stream."""
    import torch as t
    side = t.cuda.Stream()
    x, w, y = t.zeros(100, 96, device="cuda"), t.zeros(100, 96, device="cuda"), t.empty(100, 100, device="cuda")
    g, o = t.randn(200, 300, device="cuda"), t.empty(200, 300, device="cuda")
    side.wait_stream(t.cuda.current_stream())
    for ws in (gpu_lib.linear_forward(x, w, y, stream=side),
               gpu_lib.orthogonalize(g, o, stream=side)):
        owner = [s["stream"] for s in t.cuda.memory_snapshot()
                 if s["address"] <= ws.data_ptr() < s["address"] + s["total_size"]]
        assert owner == [side.cuda_stream]
    side.synchronize()
