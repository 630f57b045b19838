"""GPU tests of the loss, gradient and 8-bit calls far out: more rows than one
launch dimension's 65535 groups, operands whose offsets pass 32 bits, outputs of
more than 2^31 values, and the row strides just below what validation accepts."""
import pytest
import torch

from logit_source_projection_amd import sb
from tests.loss_common import check_grad, check_loss
from tests.test_gpu_loss import Case

pytestmark = pytest.mark.gpu


def test_many_rows(require_gpu):
    print("loss of 70001 rows", flush=True)
    c = Case(70001, 24, 300, (0, 120, 300), seed=1)
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B", [5, 300])
def test_largest_row_strides(require_gpu, B):
    """x, w and both gradients with rows of 2^23 - 8 values, 16 MiB apart."""
    H, V, ld = 290, 500, (1 << 23) - 8
    print(f"largest strides B={B}", flush=True)
    c = Case(B, H, V, (0, V), seed=2)
    wide = torch.empty(H, ld, dtype=torch.bfloat16, device="cuda")
    wide[:, :V] = c.w
    xw = torch.empty(B, ld, dtype=torch.bfloat16, device="cuda")
    xw[:, :H] = c.x
    head = sb.Head(xw[:, :H], wide[:, :V], [0, V])
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    sb.sb_cross_entropy(head, c.targets, loss, lse)
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx = torch.zeros(B, ld, dtype=torch.bfloat16, device="cuda")[:, :H]
    dw = torch.zeros(H, ld, dtype=torch.bfloat16, device="cuda")[:, :V]
    sb.sb_cross_entropy_grad(head, c.targets, lse, c.dloss, dx, dw)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B", [6, 300])
def test_int8_channels_past_4_gib(require_gpu, B):
    """70000 channels 64 KiB apart; the codes are compared at both ends."""
    H, V, ld = 80, 70000, 65536
    print(f"int8 channels past 4 GiB B={B}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = torch.empty(V, ld, dtype=torch.int8, device="cuda")[:, :H]
    codes = torch.randint(-127, 128, (V, H), device="cuda", generator=g, dtype=torch.int8)
    w.copy_(codes)
    x = torch.randint(-127, 128, (B, H), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.rand(B, device="cuda", generator=g), torch.rand(V, device="cuda", generator=g)
    head = sb.Int8Head(x, xs, w, ws, [0, 30000, V])
    out = sb.sb_int8_logits(head, torch.empty(B, V, device="cuda"))
    z = ((x.double() @ codes.double().t()).float() * xs[:, None]) * ws
    assert torch.equal(out, z)
    ids = sb.sb_int8_project_tokens(head, torch.empty(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(ids, z.argmax(1).to(torch.int32))


def test_int8_output_past_2_to_the_31(require_gpu):
    """18000 x 120000 logits in bf16: the last rows and columns."""
    B, H, V = 18000, 16, 120000
    print("int8 output of 2.16e9 values", flush=True)
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randint(-127, 128, (B, H), device="cuda", generator=g, dtype=torch.int8)
    w = torch.randint(-127, 128, (V, H), device="cuda", generator=g, dtype=torch.int8)
    xs, ws = torch.rand(B, device="cuda", generator=g), torch.rand(V, device="cuda", generator=g)
    head = sb.Int8Head(x, xs, w, ws, [0, V])
    out = sb.sb_int8_logits(head, torch.empty(B, V, device="cuda", dtype=torch.bfloat16))
    ids = sb.sb_int8_project_tokens(head, torch.empty(B, dtype=torch.int32, device="cuda"))
    for rows in (slice(0, 100), slice(B - 300, B)):
        z = ((x[rows].double() @ w.double().t()).float() * xs[rows, None]) * ws
        assert torch.equal(out[rows], z.to(torch.bfloat16))
        assert torch.equal(ids[rows], z.argmax(1).to(torch.int32))


def test_int8_many_rows(require_gpu):
    print("int8 of 70001 rows", flush=True)
    B, H, V = 70001, 40, 300
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(B, H, device="cuda", generator=g).to(torch.bfloat16)
    q = torch.empty(B, 48, dtype=torch.int8, device="cuda")[:, :H]
    xs = torch.empty(B, device="cuda")
    sb.sb_int8_quantize_rows(x, q, xs)
    w = torch.zeros(V, 48, dtype=torch.int8, device="cuda")[:, :H]
    w.copy_(torch.randint(-127, 128, (V, H), device="cuda", generator=g, dtype=torch.int8))
    ws = torch.rand(V, device="cuda", generator=g)
    head = sb.Int8Head(q, xs, w, ws, [0, 7, V])
    z = ((q.double() @ w.double().t()).float() * xs[:, None]) * ws
    assert torch.equal(sb.sb_int8_logits(head, torch.empty(B, V, device="cuda")), z)
    ids = sb.sb_int8_project_tokens(head, torch.empty(B, dtype=torch.int32, device="cuda"))
    assert torch.equal(ids, z.argmax(1).to(torch.int32))
