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
