"""A decode graph is captured and replayed with its tensors' device current,
whichever one the caller has: played on the CPU with a library, devices and
tensors of the test's own."""
import contextlib

import pytest
import torch

from gated_group_rmsnorm_gb300 import binding


class Tensor:
    """What a call of a graph looks at."""

    def __init__(self, device, shape=(1, 64)):
        self.device, self.shape, self.dtype = torch.device(device), shape, torch.bfloat16

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape[0] * self.shape[1]

    def stride(self, i=None):
        return (self.shape[1], 1)[i]

    def data_ptr(self):
        return 4096


class Library:
    def __init__(self, devices):
        self.devices, self.seen = devices, []

    def ggrn_graph_create_steps(self, steps, n, handle):
        self.seen.append(("create", self.devices[-1]))
        return binding.OK

    def ggrn_graph_launch(self, handle, stream):
        self.seen.append(("launch", self.devices[-1], stream.value))
        return binding.OK

    def ggrn_graph_destroy(self, handle):
        return binding.OK


@pytest.fixture
def cuda(monkeypatch):
    devices = [0]  # the current one last

    @contextlib.contextmanager
    def use(device):
        devices.append(torch.device(device).index)
        yield
        devices.pop()

    class Stream:
        def __init__(self, device):
            self.cuda_stream = 1000 + torch.device(device).index

    lib = Library(devices)
    monkeypatch.setattr(torch.cuda, "device", use)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: devices[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", Stream)
    monkeypatch.setattr(binding, "load", lambda *a: lib)
    return lib


def _call(device):
    t = {n: Tensor(device) for n in ("y", "gate", "w", "out")}
    return dict(t, group_size=64, eps=1e-5)


@pytest.mark.parametrize("index", [0, 1])
@pytest.mark.parametrize("n", [1, 3])
def test_graph_runs_on_its_tensors_device(cuda, index, n):
    graph = binding.DecodeGraph([_call(f"cuda:{index}")] * n)
    graph.replay()
    assert cuda.seen == [("create", index), ("launch", index, 1000 + index)]
    assert cuda.devices == [0]


def test_no_calls_are_the_librarys_to_refuse(cuda):
    binding.DecodeGraph([])
    assert cuda.seen == [("create", 0)]


def test_buffers_in_host_memory_take_the_callers_device(cuda):
    """Pinned buffers are read and written over the host link, on the stream given."""
    class Given:
        cuda_stream = 77

    graph = binding.DecodeGraph([_call("cpu")])
    graph.replay(Given())
    assert cuda.seen == [("create", 0), ("launch", 0, 77)]
