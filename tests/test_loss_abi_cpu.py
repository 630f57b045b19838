"""Validation of sb_cross_entropy and sb_cross_entropy_grad on the host: every
bad argument is refused with the documented status before any GPU work."""
import ctypes

import pytest
import torch

from logit_source_projection_amd import sb
from tests.test_abi_cpu import FAKE, fake_head

WS = ctypes.c_void_p(FAKE)
BIG = 1 << 40


def ws_status(h, grad):
    st = ctypes.c_int(0)
    n = sb.lib().sb_cross_entropy_workspace_bytes(h.ref(), grad, ctypes.byref(st))
    assert (n == 0) or st.value == sb.SB_OK
    return st.value


def loss(h, t=FAKE, out=FAKE, lse=FAKE, ws=FAKE, n=BIG):
    return sb.lib().sb_cross_entropy(h.ref(), t, out, lse, ws, n, None)


def grad(h, t=FAKE, lse=FAKE, d=FAKE, dx=FAKE, lddx=512, dw=(FAKE, FAKE), lddw=4096, ws=FAKE, n=BIG):
    arr = None if dw is None else (ctypes.c_void_p * len(dw))(*dw)
    return sb.lib().sb_cross_entropy_grad(h.ref(), t, lse, d, dx, lddx, arr, lddw, ws, n, None)


def test_workspace_sizes():
    # 16 rows, H=512, V=4096 in two lanes of 8 blocks of 256 columns: 32 tiles
    # of 128 columns and one K slice (its 16 steps are not split): a result per row and tile
    h = fake_head()
    assert sb.sb_cross_entropy_workspace_bytes(h, False) == 16 * 32 * 8 + 256
    # with 64 steps, four slices of the logits and one result per 1024 columns
    deep = fake_head(H=2048, ldx=2048)
    assert sb.sb_cross_entropy_workspace_bytes(deep, False) == 4 * 16 * 4096 * 4 + 16 * 4 * 8 + 256
    # dz in two parts, dx in 64 partial sums (one per 64 columns)
    assert sb.sb_cross_entropy_workspace_bytes(h, True) == 2 * 16 * 4096 * 2 + 64 * 16 * 512 * 4
    # small MFMA tiles: a result per row and 128 columns; dz, the masked rows and
    # dx in 16 sums (one per block)
    mid = fake_head(B=100)
    assert sb.sb_cross_entropy_workspace_bytes(mid, False) == 100 * 32 * 8 + 512
    # big ones: per 256 columns
    wide = fake_head(B=300, V=40960, off=(0, 40960), ldw=40960, w_ptrs=[FAKE])
    assert sb.sb_cross_entropy_workspace_bytes(wide, False) == 300 * 160 * 8 + 1280
    assert sb.sb_cross_entropy_workspace_bytes(mid, True) == \
        100 * 4096 * 2 + 100 * 512 * 2 + 16 * 100 * 512 * 4
    for g in (False, True):
        assert sb.sb_cross_entropy_workspace_bytes(fake_head(B=0), g) == 0
    # a large batch: dz in pieces of at most 256 MiB, and no logits anywhere
    big = fake_head(B=8192, H=512, V=151936, off=(0, 151936), ldw=151936)
    assert sb.sb_cross_entropy_workspace_bytes(big, True) < (256 << 20) + (64 << 20)


@pytest.mark.parametrize("g", [0, 1])
def test_head_rules_apply(g):
    assert ws_status(fake_head(B=-1), g) == sb.SB_ERR_SHAPE
    assert ws_status(fake_head(off=(0, 4096, 2048)), g) == sb.SB_ERR_LANES
    assert ws_status(fake_head(x_ptr=FAKE + 8), g) == sb.SB_ERR_ALIGN
    assert ws_status(fake_head(ldx=516), g) == sb.SB_ERR_ALIGN
    assert ws_status(fake_head(ldx=504), g) == sb.SB_ERR_SHAPE
    assert ws_status(fake_head(x_ptr=0), g) == sb.SB_ERR_NULL
    assert ws_status(fake_head(w_ptrs=[FAKE, 0]), g) == sb.SB_ERR_NULL
    assert ws_status(fake_head(B=1 << 24), g) == sb.SB_ERR_UNSUPPORTED


def test_offset_limits():
    # 256 rows of x must span less than 4 GiB; 64 shard rows in the loss and
    # 256 in the gradient
    assert ws_status(fake_head(ldx=1 << 23), 0) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(fake_head(ldx=(1 << 23) - 8), 0) == sb.SB_OK
    assert ws_status(fake_head(ldw=1 << 25), 0) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(fake_head(ldw=(1 << 25) - 8), 0) == sb.SB_OK
    assert ws_status(fake_head(ldw=1 << 23), 1) == sb.SB_ERR_UNSUPPORTED
    assert ws_status(fake_head(ldw=(1 << 23) - 8), 1) == sb.SB_OK


    # few rows: all of dz at once, 256 rows of which must span less than 4 GiB
    for V, want in (((1 << 23) - 256, sb.SB_OK), ((1 << 23) - 255, sb.SB_ERR_UNSUPPORTED)):
        h = fake_head(B=64, H=8, V=V, off=(0, V), ldx=8, ldw=(1 << 23) - 8, w_ptrs=[FAKE])
        assert ws_status(h, 1) == want, V
        assert ws_status(h, 0) == sb.SB_OK


def test_loss_arguments():
    h = fake_head()
    need = sb.sb_cross_entropy_workspace_bytes(h, False)
    for kw in (dict(t=None), dict(out=None), dict(lse=None), dict(ws=None)):
        assert loss(h, **kw) == sb.SB_ERR_NULL, kw
    assert loss(h, n=need - 1) == sb.SB_ERR_WORKSPACE
    assert loss(h, ws=FAKE + 8) == sb.SB_ERR_ALIGN
    assert loss(fake_head(B=-1)) == sb.SB_ERR_SHAPE
    assert loss(fake_head(B=0), None, None, None, None, 0) == sb.SB_OK
    assert sb.lib().sb_cross_entropy(None, None, None, None, None, 0, None) == sb.SB_ERR_NULL


def test_grad_arguments():
    h = fake_head()
    need = sb.sb_cross_entropy_workspace_bytes(h, True)
    for kw in (dict(t=None), dict(lse=None), dict(d=None), dict(ws=None), dict(dx=None, dw=None),
               dict(dw=(FAKE, 0))):
        assert grad(h, **kw) == sb.SB_ERR_NULL, kw
    assert grad(h, n=need - 1) == sb.SB_ERR_WORKSPACE
    for kw in (dict(lddx=504), dict(lddw=2040)):
        assert grad(h, **kw) == sb.SB_ERR_SHAPE, kw
    for kw in (dict(lddx=516), dict(lddw=4100), dict(dx=FAKE + 8), dict(dw=(FAKE, FAKE + 2)),
               dict(ws=FAKE + 4)):
        assert grad(h, **kw) == sb.SB_ERR_ALIGN, kw
    # no rows and only dx wanted: nothing to do
    assert grad(fake_head(B=0), None, None, None, FAKE, 512, None, 0, None, 0) == sb.SB_OK
    # an empty hidden size: both gradients are empty, as their pointers may be
    assert grad(fake_head(H=0, ldx=0)) == sb.SB_OK
    assert grad(fake_head(H=0, ldx=0), None, None, None, None, 0, (0, 0), 4096, None, 0) == sb.SB_OK
    assert grad(fake_head(B=0), None, None, None, None, 512, None, 0, None, 0) == sb.SB_OK


def test_binding_refuses_arguments_the_abi_cannot_take():
    h = fake_head()
    with pytest.raises(ValueError, match="targets must be a device tensor"):
        sb.sb_cross_entropy(h, torch.empty(16, dtype=torch.int32), None, None)
    with pytest.raises(ValueError, match="targets must be a device tensor"):
        sb.sb_cross_entropy_grad(h, torch.empty(16, dtype=torch.int64), None, None)
    host = sb.Head(torch.empty(16, 512, dtype=torch.bfloat16),
                   torch.empty(512, 4096, dtype=torch.bfloat16), [0, 2048, 4096])
    with pytest.raises(ValueError, match="x must be a device tensor"):
        sb.sb_cross_entropy(host, None, None, None)
    with pytest.raises(sb.SbError) as e:
        sb.sb_cross_entropy_workspace_bytes(fake_head(B=-1), True)
    assert e.value.status == sb.SB_ERR_SHAPE


def test_binding_wants_one_device():
    meta, cpu = torch.empty(1, device="meta"), torch.empty(1)
    assert sb._one_device([cpu, None, cpu]) == torch.device("cpu")
    with pytest.raises(ValueError, match="different devices"):
        sb._one_device([cpu, meta])
