"""Layer norm, embedding and verification calls on tensors of several devices are
refused, each argument by its name of devices, before the library is called.  The
tensors are fake ones (torch keeps their device and shape, and no data), so that no
second GPU is needed, or a first."""
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from logit_source_projection_amd import sb

F, I32 = torch.float32, torch.int32


@pytest.fixture
def fake(monkeypatch):
    def called(*args):
        raise AssertionError("the library was called")

    monkeypatch.setattr(sb, "_call", called)
    monkeypatch.setattr(sb, "_space", lambda ws, fn, index, stream: (sb._buffer(ws, "ws", torch.uint8, 0, index), 0, ws))
    with warnings.catch_warnings():
        warnings.simplefilter("ignore")  # (an address of a fake tensor is 0)
        with FakeTensorMode():
            yield


def norm(on):
    n = sb.Norm(on("x", 4, 16), on("weight", 16), on("bias", 16))
    sb.sb_layer_norm(n, on("y", 4, 16), on("mean", 4), on("rstd", 4))


def norm_grad(on):
    n = sb.Norm(on("x", 4, 16), on("weight", 16), on("bias", 16))
    sb.sb_layer_norm_grad(n, on("dy", 4, 16), on("mean", 4), on("rstd", 4), on("dx", 4, 16), on("dweight", 16),
                          on("dbias", 16), ws=on("ws", 64, dtype=torch.uint8))


def embed(on):
    sb.sb_embed(sb.Table([on("w", 10, 16), on("lane", 10, 16)]), on("ids", 4, dtype=I32), on("out", 4, 16))


def embed_grad(on):
    sb.sb_embed_grad(sb.Table([on("w", 10, 16), on("lane", 10, 16)]), on("ids", 4, dtype=I32), on("dout", 4, 16),
                     ws=on("ws", 64, dtype=torch.uint8))


def verify(on):
    d = sb.Drafts(on("target", 6, 40), on("tokens", 4, dtype=I32), on("offsets", 3, dtype=I32), 2, on("draft", 4, 40),
                  on("temperature", 2))
    sb.sb_verify_drafts(d, on("u", 4), on("u_next", 2), on("out", 2, 3, dtype=I32), on("accepted", 2, dtype=I32),
                        ws=on("ws", 64, dtype=torch.uint8))


CALLS = {norm: "x weight bias y mean rstd", norm_grad: "x weight bias dy mean rstd dx dweight dbias ws",
         embed: "w lane ids out", embed_grad: "w lane ids dout ws",
         verify: "target tokens offsets draft temperature u u_next out accepted ws"}


@pytest.mark.parametrize("call,name", [(f, n) for f, names in CALLS.items() for n in names.split()],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_one_tensor_on_another_device(fake, call, name):
    seen = []

    def on(which, *shape, dtype=F):
        seen.append(which)
        return torch.empty(*shape, dtype=dtype, device="cuda:1" if which == name else "cuda:0")

    with pytest.raises(ValueError, match="tensors on different devices"):
        call(on)
    assert name in seen


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("device", ["cuda:0", "cuda:1"])
def test_one_device(fake, call, device):
    with pytest.raises(AssertionError, match="the library was called"):
        call(lambda which, *shape, dtype=F: torch.empty(*shape, dtype=dtype, device=device))
