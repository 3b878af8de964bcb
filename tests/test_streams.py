"""stream= keeps the memory of a call's tensors until that stream is done with them (CPU only: the streams and the call are
stand-ins)."""
import contextlib

import pytest
import torch

from hyper_connection_rank_gb300 import _paged


class Tensor(torch.Tensor):
    """A tensor that says it lies on GPU 0 and notes the streams that its memory is kept for."""
    is_cuda = True

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.__dict__.setdefault("kept_for", []).append(stream)


class Stream:
    device = torch.device("cuda", 0)


def tensor():
    return torch.zeros(2).as_subclass(Tensor)


@pytest.fixture
def here(monkeypatch):
    stream = Stream()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: stream)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return stream


def test_every_tensor_of_a_call_is_kept(here):
    """Inputs by place and by name, out and workspace for the call's stream, results for the caller's."""
    inputs, named, out, work, result = [tensor() for _ in range(3)], tensor(), tensor(), tensor(), tensor()
    seen = {}

    def call(*args, out=None, workspace=None, **kw):
        seen.update(args=args, out=out, workspace=workspace, kw=kw)
        return result, out
    side = Stream()
    got = _paged._on_stream(side, call, *inputs, 3, None, out=out, workspace=work, bias=named, scale=2.0, live=None)
    assert got[0] is result and got[1] is out
    assert seen["args"] == (*inputs, 3, None) and seen["out"] is out and seen["workspace"] is work
    assert seen["kw"]["bias"] is named and seen["kw"]["scale"] == 2.0 and seen["kw"]["live"] is None
    for t in (*inputs, named, work):
        assert t.kept_for == [side]
    assert out.kept_for == [side, here] and result.kept_for == [here]


def test_tensors_elsewhere_are_left_to_the_call(here):
    """A tensor on the host has no stream to be kept for: the call refuses it with its own words."""
    def call(a, b):
        raise ValueError("b must be a CUDA tensor")
    with pytest.raises(ValueError, match="b must be"):
        _paged._on_stream(Stream(), call, tensor(), torch.zeros(2))
