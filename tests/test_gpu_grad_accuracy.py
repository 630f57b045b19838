"""GPU tests of how exact the gradient is: up to 32 rows, where dz is the sum of two
bf16 numbers, and above, where dz is bf16 but for the targets', whose products are
completed in fp32; on every path (streaming, small and big tiles, K slices, pieces,
one or several sums of dX)."""
import pytest
import torch

from logit_source_projection_amd import inputs, sb
from tests.grad_accuracy import check_grad_exactness
from tests.test_gpu_loss import Case

pytestmark = pytest.mark.gpu


def check(c, want=("dx", "dw")):
    _, lse = c.loss()
    dx, dw = c.grad(lse, want=want)
    check_grad_exactness(dx, dw, c.x, c.w, c.targets, c.dloss, lse)
    return lse, dx, dw


@pytest.mark.parametrize("B,H,V,lanes", [(1, 40, 700, (0, 700)), (5, 65, 2570, (0, 1032, 2570)),
                                         (16, 512, 2600, (0, 2600)), (16, 2100, 1500, (0, 1500)),
                                         (17, 72, 3001, (0, 1000, 3001)), (32, 200, 3000, (0, 3000)),
                                         (30, 2100, 1900, (0, 8, 1900))])
@pytest.mark.parametrize("spread", [0.5, 6])
def test_every_term_is_exact_up_to_32_rows(require_gpu, B, H, V, lanes, spread):
    """Without slices and with; logits close together and so far apart that other
    columns hold as much of a row as the target's."""
    print(f"grad accuracy B={B} H={H} V={V} lanes={lanes} spread={spread}", flush=True)
    c = Case(B, H, V, lanes, seed=B + V, scale=spread / H ** 0.5)
    lse, dx, dw = check(c)
    for want in ("dx", "dw"):
        one = c.grad(lse, want=(want,))[0 if want == "dx" else 1]
        assert torch.equal(one, dx if want == "dx" else dw), want


SHAPES = [
    # B, H, V, lanes
    (33, 200, 3000, (0, 3000)),
    (50, 2100, 1500, (0, 504, 1500)),         # K slices, streaming
    (64, 130, 2051, (0, 1024, 2051)),
    (65, 129, 3003, (0, 3003)),
    (100, 4100, 2003, (0, 136, 600, 2003)),   # K slices, tiles
    (257, 300, 5000, (0, 5000)),
    (600, 520, 6000, (0, 640, 1280, 6000)),
    (2048, 2100, 3000, (0, 1000, 3000)),      # one sum of dX, small tiles
    (4096, 2100, 2100, (0, 1304, 2100)),      # one sum of dX, big tiles
    (4100, 300, 40000, (0, 16000, 40000)),    # two pieces
]


@pytest.mark.parametrize("B,H,V,lanes", SHAPES)
def test_target_terms_are_exact(require_gpu, B, H, V, lanes):
    print(f"grad accuracy B={B} H={H} V={V} lanes={lanes}", flush=True)
    c = Case(B, H, V, lanes, seed=B + V, scale=0.5 / H ** 0.5)
    lse, dx, dw = check(c)
    for want in ("dx", "dw"):                 # each alone: the same bits
        one = c.grad(lse, want=(want,))[0 if want == "dx" else 1]
        assert torch.equal(one, dx if want == "dx" else dw), want


@pytest.mark.parametrize("B,H,V,lanes", [SHAPES[i] for i in (0, 1, 3, 4, 6, 8, 9)])
def test_logits_far_apart(require_gpu, B, H, V, lanes):
    """Columns besides the target's hold as much of a row: their terms are off by
    2^-8 each, and above 64 rows their sum in dx by as much again."""
    print(f"grad accuracy, far apart B={B} H={H} V={V}", flush=True)
    check(Case(B, H, V, lanes, seed=B + V, scale=6 / H ** 0.5))


@pytest.mark.parametrize("B,H,V,k", [(40, 100, 2003, 5), (70, 264, 2003, 3), (300, 64, 1601, 64)])
def test_lanes_in_their_own_allocations(require_gpu, B, H, V, k):
    print(f"grad accuracy, separate lanes B={B} V={V} k={k}", flush=True)
    check(Case(B, H, V, inputs.equal_lanes(V, k), seed=k, separate=True, scale=0.05))


@pytest.mark.parametrize("B", [40, 120, 333, 1500])
def test_rows_that_share_targets(require_gpu, B):
    """All rows on one column, on two of a block and on the ends of lanes: more
    rows to a wave's columns than it lists at once."""
    print(f"shared targets B={B}", flush=True)
    V = 2600
    c = Case(B, 96, V, (0, 520, V), seed=B, ignored=0, scale=0.05)
    i = torch.arange(B, device="cuda", dtype=torch.int32)
    for targets in (torch.full_like(i, 777), 63 + i % 2, (i % 4) * 519 + i % 2, V - 1 - i % 3):
        c.targets.copy_(targets)
        check(c)
    c.targets[::3] = -1
    c.targets[1] = -(1 << 31)
    check(c)


@pytest.mark.parametrize("B", [40, 70, 300])
def test_one_hidden_value(require_gpu, B):
    """H of 1: dx has a single column."""
    c = Case(B, 1, 900, (0, 304, 900), seed=B, scale=0.5)
    check(c)


@pytest.mark.parametrize("B", [40, 200])
def test_infinite_weight_at_a_target(require_gpu, B):
    """An impossible target: dz is -dloss there, and dx the infinity that its
    product with the weight's is, not a NaN of two of them."""
    c = Case(B, 8, 600, (0, 600), seed=1, ignored=0)
    c.x.fill_(0), c.x[:, 0].fill_(1)
    c.w.zero_()
    c.w[0] = torch.linspace(-1, 1, 600, device="cuda").to(torch.bfloat16)
    c.w[0, 100] = float("-inf")
    c.wt.copy_(c.w)
    c.targets.fill_(100)
    c.dloss.fill_(1 / 3)
    loss, lse = c.loss()
    assert bool((loss == float("inf")).all()) and bool(lse.isfinite().all())
    dx, dw = c.grad(lse)
    assert bool((dx[:, 0] == float("inf")).all())
    want = -(c.dloss.double().sum())
    assert abs(dw[0, 100].double() - want) <= 2.0 ** -8 * abs(want)


@pytest.mark.parametrize("B", [48, 96, 2500])
def test_replayed_with_new_targets(require_gpu, B):
    """Captured once; each replay's targets, eager calls between."""
    print(f"captured B={B}", flush=True)
    H, V = 200, 4000
    c = Case(B, H, V, (0, 1600, V), seed=3, scale=0.05)
    ws = sb.cross_entropy_workspace(c.head, grad=True)
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    dx = torch.empty(B, H, device="cuda", dtype=torch.bfloat16)
    dw = torch.empty(H, V, device="cuda", dtype=torch.bfloat16)
    c.loss(), c.grad(lse.zero_())             # kernels loaded before the capture
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sb.sb_cross_entropy(c.head, c.targets, loss, lse, ws=ws)
        sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss, dx, dw, ws=ws)
    for turn in range(3):
        c.targets.copy_(torch.randint(-1, V, (B,), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        check_grad_exactness(dx, dw, c.x, c.w, c.targets, c.dloss, lse)
        eager = c.grad(lse)
        assert torch.equal(dx, eager[0]) and torch.equal(dw, eager[1]), turn


@pytest.mark.parametrize("B", [40, 100, 2100])
def test_infinite_row_weight(require_gpu, B):
    """One row's loss weighted infinitely: dw is infinite, not NaN, wherever that row
    has an x and a probability, and the other rows' dx is theirs alone."""
    V = 3000
    c = Case(B, 16, V, (0, V), seed=B, ignored=0, scale=0.05)
    c.x[1] = 1
    _, lse = c.loss()
    dx, dw = c.grad(lse)
    c.dloss[1] = float("inf")
    dx2, dw2 = c.grad(lse)
    rest = torch.arange(B, device="cuda") != 1
    assert torch.equal(dx2[rest], dx[rest])
    sign = torch.ones(V, device="cuda")
    sign[c.targets[1].long()] = -1
    assert torch.equal(dw2.float(), sign.expand(16, V) * float("inf"))
