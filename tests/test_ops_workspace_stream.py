"""On which stream verify_probs takes its workspace when a stream is given
(CPU only: the tensors only claim to be on a GPU, the native call is recorded).

The workspace is given back when the call returns, before its kernels have run:
only memory of the stream that runs them is safe from the next allocation."""

import contextlib
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from speculative_decoding_sampling_amd import ops  # noqa: E402

CUDA = torch.device("cuda", 0)


class OnGpu(torch.Tensor):
    is_cuda = True
    device = CUDA

    def get_device(self):
        return 0


class Stream:
    device = CUDA

    def __init__(self, handle):
        self.cuda_stream = handle
        self.waited = []

    def wait_stream(self, other):
        self.waited.append(other)


class Calls:
    """The native module and torch's stream state, recorded."""

    def __init__(self, monkeypatch, current):
        self.current, self.workspaces, self.recorded, self.passed = current, [], [], None
        monkeypatch.setattr(ops, "_native", SimpleNamespace(verify_probs=self.verify_probs))
        monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: self.current)
        monkeypatch.setattr(torch.cuda, "stream", self.stream)
        monkeypatch.setattr(torch, "empty", self.empty)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, self.current if s is None else s
        yield
        self.current = before

    def empty(self, n, **kw):
        ws = SimpleNamespace(nbytes=n, stream=self.current)
        self.workspaces.append(ws)
        return ws

    def verify_probs(self, *args):
        self.passed = args
        return tuple(SimpleNamespace(record_stream=self.recorded.append) for _ in range(2))


def call(stream, V, **kw):
    t = torch.zeros(1, 1, V).as_subclass(OnGpu)
    return ops.verify_probs(t, None, None, None, None, None, stream=stream, **kw)


# torch's default stream has the raw handle 0
@pytest.mark.parametrize("given", [0, 1 << 40])
@pytest.mark.parametrize("current", [0, 1 << 41])
def test_workspace_is_of_the_given_stream(monkeypatch, given, current):
    given, current = Stream(given), Stream(current)
    c = Calls(monkeypatch, current)
    call(given, 40000)
    assert c.passed[11] == given.cuda_stream and given.waited == [current]
    assert [w.stream for w in c.workspaces] == [given]
    assert c.passed[9] is c.workspaces[0] and c.workspaces[0].nbytes > 0
    assert c.recorded == [given, given]


@pytest.mark.parametrize("given", [0, 1 << 40])
def test_workspace_of_the_callers(monkeypatch, given):
    c, own = Calls(monkeypatch, Stream(1 << 41)), object()
    call(Stream(given), 40000, workspace=own)
    assert c.passed[9] is own and not c.workspaces


@pytest.mark.parametrize("given", [0, 1 << 40])
def test_what_is_no_gpu_tensor_reaches_the_checks(monkeypatch, given):
    c = Calls(monkeypatch, Stream(1 << 41))
    for t in (None, [1.0], torch.zeros(1, 1, 40000), torch.zeros(1, 40000).as_subclass(OnGpu)):
        ops.verify_probs(t, None, None, None, None, None, stream=Stream(given))
        assert c.passed[0] is t and c.passed[9] is None and not c.workspaces
