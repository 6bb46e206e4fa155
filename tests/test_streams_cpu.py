"""Buffers that a prepared call made for itself, on streams and tensors that
only record what is asked of them."""
import pytest


class Stream:
    def __init__(self, handle, capturing=False):
        self.cuda_stream, self.capturing, self.waits = handle, capturing, []

    def wait_stream(self, other):
        self.waits.append(other)


class Tensor:
    device = "cuda:0"

    def __init__(self):
        self.streams = []

    def record_stream(self, s):
        self.streams.append(s)


@pytest.fixture()
def made(monkeypatch):
    from paged_kv_continuous_gb300 import build
    build.build()
    from paged_kv_continuous_gb300 import ops
    home = Stream(1)
    monkeypatch.setattr(ops.torch.cuda, "current_stream", lambda device=None: home)
    monkeypatch.setattr(ops, "_capturing", lambda s: s.capturing)
    tensors = [Tensor(), Tensor()]
    return ops._Defaults(tensors), tensors, home


def test_another_stream_waits_once_and_is_told_of(made):
    d, tensors, home = made
    assert d.known == {1}
    side = Stream(2)
    d.share(side)
    assert side.waits == [home] and d.known == {1, 2}
    assert all(t.streams == [side] for t in tensors)


def test_no_wait_enters_a_capture(made):
    d, tensors, home = made
    side = Stream(2, capturing=True)
    d.share(side)
    assert not side.waits and d.known == {1}
    assert all(t.streams == [side] for t in tensors)
    home.capturing, other = True, Stream(3)
    d.share(other)
    assert not other.waits and d.known == {1}
