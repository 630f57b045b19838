"""A torch stream belongs to a device: work of tensors on another one is refused (a
raw handle is the caller's)."""
from types import SimpleNamespace

import pytest
import torch

from logit_source_projection_amd import sb


def test_a_stream_of_another_device():
    one, two = torch.device("cuda", 0), torch.device("cuda", 1)
    with pytest.raises(ValueError, match="a stream of cuda:1 for tensors on cuda:0"):
        sb._stream_on(SimpleNamespace(device=two, cuda_stream=64), one)
    assert sb._stream_on(64, one).value == 64
