"""Validation of the 8-bit head's calls on the host: every bad argument is
refused with the documented status before any GPU work."""
import ctypes

import pytest
import torch

from logit_source_projection_amd import sb
from tests.test_abi_cpu import FAKE, fake_head

WS = ctypes.c_void_p(FAKE)
BIG = 1 << 40


def head8(B=16, H=512, V=4096, off=(0, 2048, 4096), ldx=512, ldw=512, x_ptr=FAKE, xs=FAKE,
          w=(FAKE, FAKE), ws=(FAKE, FAKE)):
    e = torch.empty(0)
    return sb.Int8Head(e, e, e, e, off, B=B, H=H, V=V, ldx=ldx, ldw=ldw, x_ptr=x_ptr,
                       x_scale_ptr=xs, w_ptrs=w, w_scale_ptrs=ws)


def status(h, surface=sb.SB_SURF_TOKENS):
    st = ctypes.c_int(0)
    sb.lib().sb_int8_workspace_bytes(h.ref(), surface, ctypes.byref(st))
    return st.value


def tokens(h, ids=FAKE, ws=FAKE, n=BIG):
    return sb.lib().sb_int8_project_tokens(h.ref(), ids, ws, n, None)


def logits(h, out=FAKE, dtype=sb.SB_FP32, ldo=4096, ws=FAKE, n=BIG):
    return sb.lib().sb_int8_logits(h.ref(), out, dtype, ldo, ws, n, None)


def rows(x=FAKE, ldx=512, B=4, H=512, q=FAKE, ldq=512, scale=FAKE):
    return sb.lib().sb_int8_quantize_rows(x, ldx, B, H, q, ldq, scale, None)


def quant(h, q=(FAKE, FAKE), ldq=512, scale=(FAKE, FAKE)):
    pq = None if q is None else (ctypes.c_void_p * len(q))(*q)
    ps = None if scale is None else (ctypes.c_void_p * len(scale))(*scale)
    return sb.lib().sb_int8_quantize_head(h.ref(), pq, ldq, ps, None)


def test_descriptor():
    assert status(head8()) == sb.SB_OK
    assert status(head8(), sb.SB_SURF_FULL_LOGITS) == sb.SB_OK
    assert status(head8(), sb.SB_SURF_LOGPROBS) == sb.SB_ERR_SHAPE
    for kw, want in (
            (dict(B=-1), sb.SB_ERR_SHAPE), (dict(H=-1), sb.SB_ERR_SHAPE),
            (dict(V=0, off=(0, 0)), sb.SB_ERR_SHAPE), (dict(ldx=496), sb.SB_ERR_SHAPE),
            (dict(ldw=496), sb.SB_ERR_SHAPE),
            (dict(off=(0, 4000, 4000)), sb.SB_ERR_LANES), (dict(off=(8, 2048, 4096)), sb.SB_ERR_LANES),
            (dict(off=(0, 3000, 2000)), sb.SB_ERR_LANES), (dict(V=5000), sb.SB_ERR_LANES),
            (dict(x_ptr=0), sb.SB_ERR_NULL), (dict(xs=0), sb.SB_ERR_NULL),
            (dict(w=(FAKE, 0)), sb.SB_ERR_NULL), (dict(ws=(0, FAKE)), sb.SB_ERR_NULL),
            (dict(x_ptr=FAKE + 8), sb.SB_ERR_ALIGN), (dict(w=(FAKE + 4, FAKE)), sb.SB_ERR_ALIGN),
            (dict(xs=FAKE + 2), sb.SB_ERR_ALIGN), (dict(ws=(FAKE, FAKE + 1)), sb.SB_ERR_ALIGN),
            (dict(ldx=520), sb.SB_ERR_ALIGN), (dict(ldw=520), sb.SB_ERR_ALIGN),
            (dict(H=131072, ldx=131072, ldw=131072), sb.SB_ERR_UNSUPPORTED),
            (dict(ldx=1 << 24), sb.SB_ERR_UNSUPPORTED), (dict(ldw=1 << 24), sb.SB_ERR_UNSUPPORTED),
            (dict(V=(1 << 30) + 1, off=(0, 8, (1 << 30) + 1)), sb.SB_ERR_UNSUPPORTED),
            (dict(B=1 << 22), sb.SB_ERR_UNSUPPORTED)):
        assert status(head8(**kw)) == want, kw
    assert status(head8(H=131071, ldx=131072, ldw=131072)) == sb.SB_OK
    assert status(head8(ldx=(1 << 24) - 16, ldw=(1 << 24) - 16)) == sb.SB_OK
    assert sb.lib().sb_int8_workspace_bytes(None, 0, None) == 0


def test_workspace_sizes():
    # 64 tiles of 64 channels cannot fill the card: K slices of partial sums
    assert sb.sb_int8_workspace_bytes(head8(H=5120, ldx=5120, ldw=5120), sb.SB_SURF_FULL_LOGITS) > 0
    # enough tiles, or MFMA tiles: the product needs none, the IDs their pairs
    wide = dict(V=40960, off=(0, 20480, 40960))
    assert sb.sb_int8_workspace_bytes(head8(**wide), sb.SB_SURF_FULL_LOGITS) == 0
    assert sb.sb_int8_workspace_bytes(head8(**wide), sb.SB_SURF_TOKENS) == 640 * 16 * 8
    assert sb.sb_int8_workspace_bytes(head8(B=100, **wide), sb.SB_SURF_FULL_LOGITS) == 0
    for s in (sb.SB_SURF_TOKENS, sb.SB_SURF_FULL_LOGITS):
        assert sb.sb_int8_workspace_bytes(head8(B=0), s) == 0


def test_product_arguments():
    h = head8()
    assert tokens(h, ids=None) == sb.SB_ERR_NULL
    assert tokens(h, ws=None) == sb.SB_ERR_NULL
    need = sb.sb_int8_workspace_bytes(h, sb.SB_SURF_TOKENS)
    assert tokens(h, n=need - 1) == sb.SB_ERR_WORKSPACE
    assert tokens(h, ws=FAKE + 8) == sb.SB_ERR_ALIGN
    assert logits(h, out=None) == sb.SB_ERR_NULL
    assert logits(h, dtype=2) == sb.SB_ERR_SHAPE
    assert logits(h, ldo=4095) == sb.SB_ERR_SHAPE
    assert logits(h, ldo=4098) == sb.SB_ERR_ALIGN
    assert logits(h, dtype=sb.SB_BF16, ldo=4100) == sb.SB_ERR_ALIGN
    assert logits(h, out=FAKE + 8) == sb.SB_ERR_ALIGN
    assert tokens(head8(B=0), None, None, 0) == sb.SB_OK
    assert logits(head8(B=0), None, sb.SB_FP32, 0, None, 0) == sb.SB_OK


def test_row_quantiser_arguments():
    for kw, want in ((dict(B=-1), sb.SB_ERR_SHAPE), (dict(ldx=504), sb.SB_ERR_SHAPE),
                     (dict(ldq=496), sb.SB_ERR_SHAPE), (dict(x=None), sb.SB_ERR_NULL),
                     (dict(q=None), sb.SB_ERR_NULL), (dict(scale=None), sb.SB_ERR_NULL),
                     (dict(x=FAKE + 2), sb.SB_ERR_ALIGN), (dict(ldx=516), sb.SB_ERR_ALIGN),
                     (dict(q=FAKE + 8), sb.SB_ERR_ALIGN), (dict(ldq=520), sb.SB_ERR_ALIGN),
                     (dict(scale=FAKE + 2), sb.SB_ERR_ALIGN),
                     (dict(B=1 << 22), sb.SB_ERR_UNSUPPORTED),
                     (dict(H=131072, ldx=131072, ldq=131072), sb.SB_ERR_UNSUPPORTED)):
        assert rows(**kw) == want, kw
    assert rows(x=None, q=None, scale=None, B=0) == sb.SB_OK


def test_head_quantiser_arguments():
    h = fake_head()
    for kw, want in ((dict(q=None), sb.SB_ERR_NULL), (dict(scale=None), sb.SB_ERR_NULL),
                     (dict(q=(FAKE, 0)), sb.SB_ERR_NULL), (dict(scale=(0, FAKE)), sb.SB_ERR_NULL),
                     (dict(ldq=496), sb.SB_ERR_SHAPE), (dict(ldq=520), sb.SB_ERR_ALIGN),
                     (dict(q=(FAKE, FAKE + 8)), sb.SB_ERR_ALIGN),
                     (dict(scale=(FAKE, FAKE + 2)), sb.SB_ERR_ALIGN)):
        assert quant(h, **kw) == want, kw
    assert quant(fake_head(w_ptrs=[FAKE, FAKE + 8])) == sb.SB_ERR_ALIGN
    assert quant(fake_head(w_ptrs=[FAKE, 0])) == sb.SB_ERR_NULL
    assert quant(fake_head(ldw=4100)) == sb.SB_ERR_ALIGN
    assert quant(fake_head(ldw=1000)) == sb.SB_ERR_SHAPE
    assert quant(fake_head(off=(0, 4096, 2048))) == sb.SB_ERR_LANES
    assert quant(fake_head(H=131072, ldx=131072, ldw=4096), ldq=131072) == sb.SB_ERR_UNSUPPORTED


def test_binding_refuses_arguments_the_abi_cannot_take():
    q, s = torch.zeros(4, 32, dtype=torch.int8), torch.ones(4)
    h = sb.Int8Head(q, s, q, s, [0, 4])
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_int8_project_tokens(h, None)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_int8_logits(h, None)
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_int8_quantize_rows(torch.zeros(4, 32, dtype=torch.bfloat16), q, s)
    with pytest.raises(ValueError, match="one tensor per lane"):
        sb.Int8Head(q, s, [q], [s], [0, 2, 4])
    with pytest.raises(sb.SbError) as e:
        sb.sb_int8_workspace_bytes(head8(B=-1), sb.SB_SURF_TOKENS)
    assert e.value.status == sb.SB_ERR_SHAPE
