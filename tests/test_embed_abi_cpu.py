"""Validation of sb_embed and sb_embed_grad on the host: every bad argument is
refused with the documented status before any GPU work."""
import ctypes

import pytest
import torch

from logit_source_projection_amd import sb
from tests.test_abi_cpu import FAKE

BIG = 1 << 40


def table(V=4096, H=512, off=(0, 1000, 4096), w=(FAKE, FAKE), ldw=512, type=sb.SB_BF16):
    return sb.Table(torch.empty(0, 0), off, V=V, H=H, ldw=ldw, type=type, w_ptrs=w)


def embed(t, ids=FAKE, B=4, scale=1.0, out=FAKE, out_type=sb.SB_BF16, ldo=512):
    return sb.lib().sb_embed(t.ref(), ids, B, scale, out, out_type, ldo, None)


def grad(t, ids=FAKE, B=4, scale=1.0, dout=FAKE, dout_type=sb.SB_BF16, lddo=512, add=0, ws=FAKE, n=BIG):
    return sb.lib().sb_embed_grad(t.ref(), ids, B, scale, dout, dout_type, lddo, add, ws, n, None)


def ws_status(t, B=4, add=0):
    st = ctypes.c_int(0)
    n = sb.lib().sb_embed_grad_workspace_bytes(t.ref(), B, add, ctypes.byref(st))
    assert n == 0 or st.value == sb.SB_OK
    return st.value


@pytest.mark.parametrize("kw,want", [
    (dict(V=0, off=(0, 0), w=(FAKE,)), sb.SB_ERR_SHAPE), (dict(H=-1), sb.SB_ERR_SHAPE), (dict(type=2), sb.SB_ERR_SHAPE),
    (dict(type=-1), sb.SB_ERR_SHAPE), (dict(ldw=504), sb.SB_ERR_SHAPE), (dict(ldw=-512), sb.SB_ERR_SHAPE),
    (dict(V=5000), sb.SB_ERR_LANES), (dict(off=(8, 1000, 4096)), sb.SB_ERR_LANES),
    (dict(off=(0, 4096, 4096)), sb.SB_ERR_LANES), (dict(off=(0, 5000, 4096)), sb.SB_ERR_LANES),
    (dict(w=(FAKE, 0)), sb.SB_ERR_NULL), (dict(w=(FAKE + 8, FAKE)), sb.SB_ERR_ALIGN), (dict(ldw=516), sb.SB_ERR_ALIGN),
    (dict(ldw=514, type=sb.SB_FP32), sb.SB_ERR_ALIGN),
    (dict(V=(1 << 30) + 1, off=(0, 1000, (1 << 30) + 1)), sb.SB_ERR_UNSUPPORTED),
    (dict(H=(1 << 24) + 1, ldw=1 << 25), sb.SB_ERR_UNSUPPORTED), (dict(ldw=1 << 36), sb.SB_ERR_UNSUPPORTED),
    (dict(ldw=1 << 62), sb.SB_ERR_UNSUPPORTED)])
def test_table(kw, want):
    t = table(**kw)
    assert ws_status(t) == want
    assert embed(t, ldo=1 << 25) == want
    assert grad(t, lddo=1 << 25) == want


def test_lane_counts():
    for k in (0, 65):
        t = table()
        t.desc.k = k
        assert ws_status(t) == sb.SB_ERR_LANES
    assert sb.lib().sb_embed(None, FAKE, 4, 1.0, FAKE, 1, 512, None) == sb.SB_ERR_NULL
    many = list(range(0, 65 * 10, 10))
    assert ws_status(table(V=640, off=many, w=[FAKE] * 64)) == sb.SB_OK


def test_lookup_arguments():
    for kw, want in ((dict(B=-1), sb.SB_ERR_SHAPE), (dict(out_type=3), sb.SB_ERR_SHAPE), (dict(ldo=511), sb.SB_ERR_SHAPE),
                     (dict(scale=float("nan")), sb.SB_ERR_SHAPE), (dict(scale=float("inf")), sb.SB_ERR_SHAPE),
                     (dict(ids=0), sb.SB_ERR_NULL), (dict(out=0), sb.SB_ERR_NULL), (dict(ids=FAKE + 2), sb.SB_ERR_ALIGN),
                     (dict(out=FAKE + 4), sb.SB_ERR_ALIGN), (dict(ldo=516), sb.SB_ERR_ALIGN),
                     (dict(ldo=1 << 60), sb.SB_ERR_UNSUPPORTED)):
        assert embed(table(), **kw) == want, kw
    assert embed(table(V=1 << 28, off=(0, 1000, 1 << 28)), B=-1) == sb.SB_ERR_SHAPE


def test_gradient_arguments():
    for kw, want in ((dict(B=-1), sb.SB_ERR_SHAPE), (dict(dout_type=3), sb.SB_ERR_SHAPE), (dict(lddo=511), sb.SB_ERR_SHAPE),
                     (dict(scale=float("nan")), sb.SB_ERR_SHAPE), (dict(ids=0), sb.SB_ERR_NULL),
                     (dict(dout=0), sb.SB_ERR_NULL), (dict(ids=FAKE + 2), sb.SB_ERR_ALIGN),
                     (dict(dout=FAKE + 4), sb.SB_ERR_ALIGN), (dict(lddo=516), sb.SB_ERR_ALIGN),
                     (dict(lddo=1 << 60), sb.SB_ERR_UNSUPPORTED), (dict(B=(1 << 24) + 1), sb.SB_ERR_UNSUPPORTED),
                     (dict(ws=0), sb.SB_ERR_NULL), (dict(ws=FAKE + 8), sb.SB_ERR_ALIGN), (dict(n=64), sb.SB_ERR_WORKSPACE)):
        assert grad(table(), **kw) == want, kw
    big = table(V=(1 << 24) + 1, off=(0, 1000, (1 << 24) + 1))
    assert ws_status(big) == sb.SB_ERR_UNSUPPORTED and grad(big) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(table(), B=-1) == sb.SB_ERR_SHAPE


def test_nothing_to_do():
    assert embed(table(), B=0, ids=0, out=0) == sb.SB_OK
    empty = table(H=0, ldw=0, w=(0, 0))
    assert embed(empty, ids=0, out=0, ldo=0) == sb.SB_OK
    assert grad(empty, ids=0, dout=0, lddo=0, ws=0, n=0) == sb.SB_OK
    assert grad(table(), B=0, add=1, ids=0, dout=0, ws=0, n=0) == sb.SB_OK


def test_host_tensors_are_refused():
    w, ids = torch.zeros(16, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="w must be a device tensor"):
        sb.sb_embed(sb.Table(w), ids, torch.zeros(2, 8))
    with pytest.raises(ValueError, match="w must be a device tensor"):
        sb.sb_embed_grad(sb.Table(w), ids, torch.zeros(2, 8))
    with pytest.raises(ValueError, match="one tensor per lane, 2"):
        sb.Table([w], [0, 8, 16])


def test_gradients_that_pass_a_grid():
    wide = dict(ldw=1 << 24, type=sb.SB_BF16)
    assert ws_status(table(H=(1 << 24) - 512, **wide), B=1 << 10) == sb.SB_OK
    assert ws_status(table(H=(1 << 24) - 8, **wide)) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(table(H=1 << 16, ldw=1 << 16), B=1 << 24) == sb.SB_ERR_UNSUPPORTED
    # with the zeros' workgroups behind them
    assert ws_status(table(H=1 << 14, ldw=1 << 14), B=1 << 24) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(table(H=1 << 12, ldw=1 << 12), B=1 << 24) == sb.SB_OK
