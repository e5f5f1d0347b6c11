"""Where the feed-forward helpers get the memory that they allocate, without a GPU:
torch's streams are stood in for by names, and an allocation notes which one
is current."""
import contextlib
import inspect
import re

import pytest

torch = pytest.importorskip("torch")
from fp32_gemm_tuning_amd import ffn  # noqa: E402


class Allocated:
    def __init__(self, on):
        self.on, self.device, self.used_on = on, "cuda:0", []

    def record_stream(self, s):
        self.used_on.append(s)


class Like:
    device = "cuda:0"

    def __init__(self, current):
        self.current = current

    def new_empty(self, shape, dtype=None):
        return Allocated(self.current[-1])


@pytest.fixture
def current(monkeypatch):
    stack = ["current"]

    @contextlib.contextmanager
    def stream(s):
        stack.append(s)
        yield
        stack.pop()

    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: stack[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda address, device=None: f"stream at {address}")
    return stack


@pytest.mark.parametrize("stream,name", [("another", "another"), (4096, "stream at 4096")])
def test_memory_is_the_streams_own(current, stream, name):
    t = ffn._new(Like(current), 2, 3, stream)
    assert t.on == name                 # ordered with the work that will write it
    assert "current" in t.used_on       # and kept while the caller's stream uses it
    assert current == ["current"]


def test_a_workspace_is_the_streams_alone(current):
    t = ffn._new(Like(current), 1, 64, "another", torch.uint8, returned=False)
    assert t.on == "another" and t.used_on == []


def test_without_a_stream_it_is_the_current_ones(current):
    t = ffn._new(Like(current), 2, 3)
    assert t.on == "current" and t.used_on == []


def test_nothing_is_allocated_another_way():
    source = inspect.getsource(ffn)
    assert not re.search(r"torch\.(empty|zeros|ones|full)\w*\(", source)
    assert source.count("new_empty(") == inspect.getsource(ffn._new).count("new_empty(")


class GpuTensor:
    """What the helpers look at before they look at a stream."""
    is_cuda, dtype = True, torch.bfloat16

    def __init__(self, *shape):
        self.shape, self.device = shape, torch.device("cuda:0")

    def dim(self):
        return 2


class Elsewhere:
    device = torch.device("cuda:1")
    cuda_stream = 4096


W = ffn.W4(GpuTensor(8, 32), GpuTensor(8, 1), None, 64, 64)
X = GpuTensor(4, 64)


@pytest.mark.parametrize("call", [
    lambda s: ffn.glu(X, GpuTensor(8, 64), GpuTensor(8, 64), stream=s),
    lambda s: ffn.glu_backward(GpuTensor(4, 8), X, GpuTensor(8, 64), GpuTensor(8, 64), None, stream=s),
    lambda s: ffn.w4_quantize(GpuTensor(8, 64), stream=s), lambda s: ffn.w4_dequantize(W, stream=s),
    lambda s: ffn.w4_matmul(X, W, stream=s), lambda s: ffn.w4_glu(X, W, W, stream=s)],
    ids=["glu", "glu_backward", "w4_quantize", "w4_dequantize", "w4_matmul", "w4_glu"])
def test_another_devices_stream_is_refused(call):
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(Elsewhere())
