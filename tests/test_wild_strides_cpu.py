"""Row strides whose byte spans pass 64 bits are refused, not wrapped round to small ones."""
import ctypes

import pytest

from logit_source_projection_amd import sb
from tests.test_abi_cpu import fake_head, fake_partial, ws_status
from tests.test_int8_abi_cpu import head8
from tests.test_int8_abi_cpu import status as int8_status
from tests.test_loss_abi_cpu import ws_status as loss_status

WILD = [1 << n for n in range(36, 63)] + [(1 << 56) + 16, (1 << 58) + (1 << 40), (1 << 63) - 16]


@pytest.mark.parametrize("B", [1, 16, 100, 300])
@pytest.mark.parametrize("ld", WILD)
def test_refused_everywhere(B, ld):
    for kw in (dict(ldx=ld), dict(ldw=ld), dict(ldx=ld, ldw=ld)):
        assert ws_status(fake_head(B=B, **kw)) == sb.SB_ERR_UNSUPPORTED
        for grad in (0, 1):
            assert loss_status(fake_head(B=B, **kw), grad) == sb.SB_ERR_UNSUPPORTED
        for surface in (sb.SB_SURF_TOKENS, sb.SB_SURF_FULL_LOGITS):
            assert int8_status(head8(B=B, **kw), surface) == sb.SB_ERR_UNSUPPORTED
        st = ctypes.c_int(0)
        sb.lib().sb_partial_workspace_bytes(fake_partial(B=B, **kw).ref(), ctypes.byref(st))
        assert st.value == sb.SB_ERR_UNSUPPORTED
