"""A torch stream belongs to a device: work of tensors on another one is refused (a
raw handle is the caller's)."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from logit_source_projection_amd import sb


def test_a_stream_of_another_device():
    one, two = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(ValueError, match="a stream of cuda:1 for tensors on cuda:0"):
        sb._stream_on(SimpleNamespace(device=two, cuda_stream=64), one)
    assert sb._stream_on(64, one).value == 64


def test_refused_before_a_workspace_is_allocated(monkeypatch):
    """A call that makes its own workspace would allocate it on the other device's stream."""
    def allocated(*args):
        raise AssertionError("a workspace was allocated")

    monkeypatch.setattr(sb, "_workspace", allocated)
    monkeypatch.setattr(sb, "_on", lambda device: contextlib.nullcontext())
    with pytest.raises(ValueError, match="a stream of cuda:1 for tensors on cuda:0"):
        sb._space(None, lambda: 16, 0, SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=64))
