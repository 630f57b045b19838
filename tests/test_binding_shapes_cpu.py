"""A head whose tensors are smaller than its descriptor says: its loss, gradient and
quantiser would read past them.  (The device check comes first in the calls; the
shapes are checked with the operands' device.)"""
import pytest
import torch

from logit_source_projection_amd import sb


def bf16(*shape):
    return torch.empty(*shape, dtype=torch.bfloat16)


def test_shapes_of_one_weight():
    assert sb.Head(bf16(4, 64), bf16(64, 304), [0, 304]).device() == torch.device("cpu")
    assert sb.Head(bf16(4, 64)[:2], bf16(80, 304), [0, 104, 296]).device() == torch.device("cpu")
    with pytest.raises(ValueError, match=r"w must be a \[>= 64, >= 304\] matrix, not \[56, 304\]"):
        sb.Head(bf16(4, 64), bf16(56, 304), [0, 304]).device()
    with pytest.raises(ValueError, match=r"w must be a \[>= 64, >= 312\]"):
        sb.Head(bf16(4, 64), bf16(64, 304), [0, 312]).device()
    with pytest.raises(ValueError, match=r"x must be a \[>= 5, >= 64\]"):
        sb.Head(bf16(4, 64), bf16(64, 304), [0, 304], B=5).device()


def test_shapes_of_lanes():
    assert sb.Head(bf16(4, 64), [bf16(64, 104)[:, :100], bf16(64, 104)], [0, 100, 204]).device()
    with pytest.raises(ValueError, match=r"w\[1\] must be a \[>= 64, >= 105\]"):
        sb.Head(bf16(4, 64), [bf16(64, 104), bf16(64, 104)], [0, 104, 209]).device()
    with pytest.raises(ValueError, match="one tensor per lane, 3"):
        sb.Head(bf16(4, 64), [bf16(64, 104), bf16(64, 104)], [0, 104, 208, 216]).device()
    with pytest.raises(ValueError, match="one row stride"):
        sb.Head(bf16(4, 64), [bf16(64, 104), bf16(64, 112)], [0, 104, 208]).device()


def test_raw_pointers_are_the_callers():
    assert sb.Head(bf16(0, 0), bf16(0, 0), [0, 8], B=4, H=8, ldx=8, ldw=8, x_ptr=16, w_ptrs=[16]).device() is None
