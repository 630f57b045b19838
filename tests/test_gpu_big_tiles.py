"""GPU tests of the 256 x 256 tiles through many K stages, ragged in every size:
loss, gradient and the 8-bit product.  Each case first shows, by the rules of the
sources and by the workspace it needs, that it runs those tiles."""
import os
import re

import pytest
import torch

from logit_source_projection_amd import build, sb
from tests.grad_accuracy import check_grad_exactness
from tests.loss_common import HALF_FP32, check_loss
from tests.test_gpu_int8 import Case as Case8
from tests.test_gpu_loss import Case

pytestmark = pytest.mark.gpu


def constant(header, name):
    """An integer constant of a header of the kernels."""
    text = open(os.path.join(build.CSRC, header)).read()
    return int(re.search(rf"\b{name} = (\d+)", text).group(1))


def up(n, m):
    return -(-n // m) * m


def blocks(lanes):
    return sum(-(-(b - a) // 256) for a, b in zip(lanes, lanes[1:]))


def assert_big_logits(c):
    n = blocks(c.lanes)
    assert c.B > constant("loss.h", "kSmallRows")
    assert -(-c.B // 256) * n > constant("loss.h", "kSmallLogitsTiles")
    # one result per row and 256 columns (128 in the small tiles), no slices
    assert sb.sb_cross_entropy_workspace_bytes(c.head, False) == up(8 * c.B * n, 256) + up(4 * c.B, 256)


def assert_big_grad(c, piece_blocks):
    assert_big_logits(c)
    assert -(-c.H // 256) * piece_blocks * -(-c.B // 256) > constant("loss.h", "kSmallGradTiles")


def loss_and_gradient(c):
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad_exactness(dx, dw, c.x, c.w, c.targets, c.dloss, lse)
    return loss, lse, dx, dw


@pytest.mark.parametrize("B,H,V,lanes", [
    (2100, 1111, 4000, (0, 4000)),                  # 18 stages, the last of 23 values
    (2304, 64, 4100, (0, 8, 1032, 4100)),           # one whole stage
    (2049, 65, 4003, (0, 4003)),                    # a stage and one value
    (2100, 192, 3700, (0, 264, 3700)),              # three whole stages
    (300, 257, 17001, (0, 5000, 17001)),
])
def test_loss(require_gpu, B, H, V, lanes):
    print(f"big tiles: loss B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=H, scale=1 / H ** 0.5)
    assert_big_logits(c)
    first = c.loss()
    check_loss(*first, c.x, c.w, c.targets)
    for _ in range(3):
        for a, b in zip(first, c.loss()):
            assert torch.equal(a, b)


def test_gradient_with_one_sum_of_dx(require_gpu):
    """Nine tiles of dX's columns, each stored at once."""
    B, H, V, lanes = 4096, 2100, 2100, (0, 1304, 2100)
    print(f"big tiles: gradient B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=1, scale=0.02)
    assert_big_grad(c, blocks(lanes))
    n = blocks(lanes) * 256
    assert sb.sb_cross_entropy_workspace_bytes(c.head, True) == 2 * B * (n + up(H, 8)) + 2 * B
    first = loss_and_gradient(c)
    for a, b in zip(first[2:], c.grad(first[1])):
        assert torch.equal(a, b)


def test_gradient_with_two_sums_of_dx(require_gpu):
    B, H, V, lanes = 2048, 2100, 8190, (0, 4104, 8190)
    print(f"big tiles: gradient B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=2, scale=0.02)
    assert_big_grad(c, blocks(lanes))
    # two sums of 72 big tiles; 272 small ones would store theirs at once
    n = blocks(lanes) * 256
    assert sb.sb_cross_entropy_workspace_bytes(c.head, True) == 2 * B * (n + up(H, 8)) + 2 * 4 * B * up(H, 4)
    loss_and_gradient(c)


def test_gradient_in_pieces(require_gpu):
    """Two pieces of the vocabulary, two tiles of H, dX in four sums."""
    B, H, V, lanes = 4100, 333, 40003, (0, 16000, 40003)
    print(f"big tiles: pieces B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=3, scale=0.05)
    piece = -(-blocks(lanes) // 2)
    assert_big_grad(c, piece)
    assert sb.sb_cross_entropy_workspace_bytes(c.head, True) == \
        2 * B * (256 * piece) + up(2 * B * up(H, 8), 256) + up(4 * 4 * B * up(H, 4), 256)
    loss_and_gradient(c)


def test_rows_that_hold_anything(require_gpu):
    """Ignored rows of NaN and infinities, a target past the vocabulary, masked
    columns and an infinite loss."""
    B, H, V = 2100, 200, 4000
    print("big tiles: ignored and masked", flush=True)
    c = Case(B, H, V, (0, 1504, V), seed=4, scale=0.05)
    wide = Case(4600, 900, V, (0, 1504, V), seed=5, scale=0.03)
    assert_big_logits(c)
    assert_big_grad(wide, blocks(wide.lanes))
    for case in (c, wide):
        case.targets[0], case.targets[case.B - 1] = V - 1, -1
        ref = loss_and_gradient(case)
        ig = case.targets < 0
        case.x[ig] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38],
                                  device="cuda").repeat(case.H // 4).to(torch.bfloat16)
        loss, lse = case.loss()
        assert bool((loss[ig] == 0).all()) and torch.equal(lse[~ig], ref[1][~ig])
        dx, dw = case.grad(lse)
        assert torch.equal(dx, ref[2]) and torch.equal(dw, ref[3])
        case.targets[5] = V                       # past the vocabulary
        loss, lse = case.loss()
        assert bool(loss[5].isnan()) and bool(lse[5].isfinite())
        dx, dw = case.grad(lse)
        rest = torch.arange(case.B, device="cuda") != 5
        assert bool(dx[5].isnan().all()) and torch.equal(dx[rest], ref[2][rest]) and bool(dw.isnan().all())
    # columns at -inf wherever x's first value is 1
    c.x.fill_(0), c.x[:, 0].fill_(1)
    c.w.zero_()
    c.w[0] = torch.linspace(-3, 3, V, device="cuda").to(torch.bfloat16)
    c.w[0, 100:3000] = float("-inf")
    c.wt.copy_(c.w)
    c.targets.fill_(50)
    c.targets[7] = 2999
    loss, lse = c.loss()
    want = torch.logsumexp(c.w[0].double(), 0)
    assert bool(((lse.double() - want).abs() <= 64 * HALF_FP32 * 8).all())
    assert loss[7].item() == float("inf") and bool(loss[:7].isfinite().all())


@pytest.mark.parametrize("B,H,V,lanes", [
    (2100, 1000, 5000, (0, 300, 2001, 5000)),       # 8 stages, the last of 104 values
    (2304, 128, 4100, (0, 4100)),                   # one whole stage
    (2049, 129, 4003, (0, 7, 4003)),
    (2100, 384, 3700, (0, 3700)),                   # three whole stages
    (1200, 5120, 8000, (0, 2600, 8000)),            # 40 stages
    (300, 300, 17001, (0, 5000, 17001)),
])
def test_int8(require_gpu, B, H, V, lanes):
    print(f"big tiles: int8 B={B} H={H} V={V}", flush=True)
    c = Case8(B, H, V, lanes, seed=H)
    n = blocks(lanes)
    assert B > constant("int8.h", "kInt8TileSmallRows") and B > constant("int8.h", "kInt8SmallRows")
    assert -(-B // 256) * n > constant("int8.h", "kInt8SmallTiles")
    # a pair per row and 256 columns (128 in the small tiles), no slices
    assert sb.sb_int8_workspace_bytes(c.head, sb.SB_SURF_TOKENS) == up(8 * B * n, 256)
    assert sb.sb_int8_workspace_bytes(c.head, sb.SB_SURF_FULL_LOGITS) == 0
    z = c.reference()
    want = z.argmax(1).to(torch.int32)
    for _ in range(2):
        assert torch.equal(c.logits(), z)
        assert torch.equal(c.tokens(), want)
    assert torch.equal(c.logits(torch.bfloat16), z.to(torch.bfloat16))


def test_int8_ties_and_scales_that_are_not_finite(require_gpu):
    B, H, V = 2100, 200, 4100
    c = Case8(B, H, V, (0, 1000, V), seed=3)
    assert sb.sb_int8_workspace_bytes(c.head, sb.SB_SURF_TOKENS) == up(8 * B * blocks((0, 1000, V)), 256)
    top = torch.full((H,), 127, dtype=torch.int8, device="cuda")
    c.x[:, :] = top
    c.ws.fill_(0.5)
    for cols in ([V - 1], [2999, 1001], [1001, 999], [999, 70, 64], [70, 3, 2]):
        c.w[cols] = top
        assert bool((c.tokens() == min(cols)).all()), cols
    c.w.zero_()
    assert bool((c.tokens() == 0).all())
    c.x[:, 0], c.w[:, 0] = 1, 1
    c.x[:, 1:] = 0
    c.xs.fill_(1.0), c.ws.fill_(1.0)
    c.ws[3000], c.ws[2500] = float("nan"), float("inf")
    assert bool((c.tokens() == 3000).all())          # NaN ranks above infinity
    c.ws[3000] = 1
    assert bool((c.tokens() == 2500).all())
    c.xs[1999] = float("nan")
    ids = c.tokens()
    assert ids[1999].item() == 0 and int((ids == 2500).sum()) == B - 1
    assert torch.equal(c.logits().isnan(), c.reference().isnan())


def test_int8_longest_sums(require_gpu):
    """The largest H, 1024 stages, of the largest products."""
    B, H, V = 2100, 131071, 4100
    print("big tiles: longest sums", flush=True)
    c = Case8(B, H, V, (0, V), seed=1, extreme=True)
    assert sb.sb_int8_workspace_bytes(c.head, sb.SB_SURF_TOKENS) == up(8 * B * blocks((0, V)), 256)
    c.x[0], c.w[0] = -128, -128
    out = c.logits()
    rows = torch.tensor([0, 1, 255, 256, 1000, 2047, 2048, 2099], device="cuda")
    sums = c.x[rows].double() @ c.w.double().t()
    assert sums[0, 0].item() == 16384.0 * H
    assert torch.equal(out[rows], (sums.float() * c.xs[rows, None]) * c.ws)
