"""Validation of sb_layer_norm and sb_layer_norm_grad on the host: every bad
argument is refused with the documented status before any GPU work."""
import ctypes

import pytest
import torch

from logit_source_projection_amd import sb
from tests.test_abi_cpu import FAKE

BIG = 1 << 40
NAN, INF = float("nan"), float("inf")


def desc(B=4, H=512, x=FAKE, x_type=sb.SB_BF16, ldx=512, weight=FAKE, bias=FAKE, param_type=sb.SB_FP32, eps=1e-5):
    return sb.sb_norm_desc(B=B, H=H, x=x, x_type=x_type, ldx=ldx, weight=weight, bias=bias,
                           param_type=param_type, eps=eps)


def forward(d, y=FAKE, y_type=sb.SB_BF16, ldy=512, mean=FAKE, rstd=FAKE):
    return sb.lib().sb_layer_norm(ctypes.byref(d), y, y_type, ldy, mean, rstd, None)


def grad(d, dy=FAKE, dy_type=sb.SB_BF16, lddy=512, mean=FAKE, rstd=FAKE, dx=FAKE, lddx=512, dw=FAKE, db=FAKE,
         ws=FAKE, n=BIG):
    return sb.lib().sb_layer_norm_grad(ctypes.byref(d), dy, dy_type, lddy, mean, rstd, dx, lddx, dw, db, ws, n, None)


def ws_status(d):
    st = ctypes.c_int(0)
    n = sb.lib().sb_layer_norm_grad_workspace_bytes(ctypes.byref(d), ctypes.byref(st))
    assert n == 0 or st.value == sb.SB_OK
    return st.value


BAD_DESC = [
    (dict(B=-1), sb.SB_ERR_SHAPE), (dict(H=0), sb.SB_ERR_SHAPE), (dict(H=-3), sb.SB_ERR_SHAPE),
    (dict(x_type=2), sb.SB_ERR_SHAPE), (dict(x_type=-1), sb.SB_ERR_SHAPE), (dict(param_type=7), sb.SB_ERR_SHAPE),
    (dict(eps=-1e-9), sb.SB_ERR_SHAPE), (dict(eps=NAN), sb.SB_ERR_SHAPE), (dict(eps=INF), sb.SB_ERR_SHAPE),
    (dict(ldx=504), sb.SB_ERR_SHAPE), (dict(ldx=-512), sb.SB_ERR_SHAPE), (dict(ldx=0), sb.SB_ERR_SHAPE),
    (dict(x=0), sb.SB_ERR_NULL),
    (dict(x=FAKE + 8), sb.SB_ERR_ALIGN), (dict(ldx=516), sb.SB_ERR_ALIGN),
    (dict(ldx=514, x_type=sb.SB_FP32), sb.SB_ERR_ALIGN),
    (dict(weight=FAKE + 4), sb.SB_ERR_ALIGN), (dict(bias=FAKE + 2), sb.SB_ERR_ALIGN),
    (dict(H=(1 << 24) + 1, ldx=(1 << 24) + 8), sb.SB_ERR_UNSUPPORTED),
    (dict(ldx=1 << 45), sb.SB_ERR_UNSUPPORTED), (dict(ldx=1 << 62), sb.SB_ERR_UNSUPPORTED),
]


@pytest.mark.parametrize("kw,want", BAD_DESC)
def test_descriptor(kw, want):
    assert ws_status(desc(**kw)) == want
    assert forward(desc(**kw), ldy=1 << 25) == want
    assert grad(desc(**kw), lddy=1 << 25, lddx=1 << 25) == want


def test_null_descriptor():
    assert sb.lib().sb_layer_norm(None, FAKE, 0, 512, None, None, None) == sb.SB_ERR_NULL
    assert sb.lib().sb_layer_norm_grad_workspace_bytes(None, None) == 0


def test_forward_arguments():
    for kw, want in ((dict(y=0), sb.SB_ERR_NULL), (dict(y_type=5), sb.SB_ERR_SHAPE), (dict(ldy=511), sb.SB_ERR_SHAPE),
                     (dict(ldy=516), sb.SB_ERR_ALIGN), (dict(y=FAKE + 4), sb.SB_ERR_ALIGN),
                     (dict(mean=FAKE + 1), sb.SB_ERR_ALIGN), (dict(rstd=FAKE + 2), sb.SB_ERR_ALIGN),
                     (dict(ldy=1 << 60), sb.SB_ERR_UNSUPPORTED)):
        assert forward(desc(), **kw) == want, kw


def test_gradient_arguments():
    for kw, want in ((dict(dy=0), sb.SB_ERR_NULL), (dict(dy_type=2), sb.SB_ERR_SHAPE), (dict(lddy=511), sb.SB_ERR_SHAPE),
                     (dict(lddy=516), sb.SB_ERR_ALIGN), (dict(dy=FAKE + 4), sb.SB_ERR_ALIGN),
                     (dict(mean=0), sb.SB_ERR_NULL), (dict(rstd=0), sb.SB_ERR_NULL),
                     (dict(mean=FAKE + 1), sb.SB_ERR_ALIGN),
                     (dict(lddx=511), sb.SB_ERR_SHAPE), (dict(lddx=516), sb.SB_ERR_ALIGN),
                     (dict(dx=FAKE + 8), sb.SB_ERR_ALIGN), (dict(lddx=1 << 60), sb.SB_ERR_UNSUPPORTED),
                     (dict(dw=FAKE + 8), sb.SB_ERR_ALIGN), (dict(db=FAKE + 8), sb.SB_ERR_ALIGN),
                     (dict(dx=0, dw=0, db=0), sb.SB_ERR_NULL)):
        assert grad(desc(), **kw) == want, kw
    for kw, want in ((dict(ws=0), sb.SB_ERR_NULL), (dict(ws=FAKE + 8), sb.SB_ERR_ALIGN), (dict(n=16), sb.SB_ERR_WORKSPACE)):
        assert grad(desc(B=1000), **kw) == want, kw


def test_gradient_workspace():
    def n(**kw):
        return sb.lib().sb_layer_norm_grad_workspace_bytes(ctypes.byref(desc(**kw)), None)

    # one launch of few rows, partial sums of more or longer ones
    assert n(B=1) == n(B=256) == n(B=256, H=8192, ldx=8192) == 0
    assert n(B=257) > 0 and n(B=1, H=8193, ldx=8200) > 0


def test_no_rows():
    # nothing to do, and nothing is launched
    d = desc(B=0, x=0)
    assert forward(d, y=0) == sb.SB_OK
    assert grad(d, dy=0, mean=0, rstd=0, dw=0, db=0, ws=0, n=0) == sb.SB_OK
    assert sb.lib().sb_layer_norm_grad_workspace_bytes(ctypes.byref(d), None) == 0


def test_host_tensors_are_refused():
    x, y = torch.zeros(2, 8), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_layer_norm(sb.Norm(x), y)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_layer_norm_grad(sb.Norm(x), y, None, None, dx=y)
