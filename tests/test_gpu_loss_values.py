"""GPU tests of single values of the loss on every path: small losses beside large
logits, and rows whose logits are all -inf."""
import pytest
import torch

from logit_source_projection_amd import sb
from tests.loss_common import HALF_FP32
from tests.test_gpu_loss import Case

pytestmark = pytest.mark.gpu

# B, H, V: streaming; with K slices; small tiles; with K slices; big tiles
PATHS = [(3, 8, 300), (20, 8, 1000), (40, 8, 300), (5, 2100, 300), (50, 2100, 300), (70, 8, 300),
         (100, 4100, 300), (2100, 8, 4000)]


@pytest.mark.parametrize("B,H,V", PATHS)
def test_small_losses_beside_large_logits(require_gpu, B, H, V):
    """The target's logit is 1000 and the others' 984: the loss is log(1 + (V - 1)
    e^-16), 3e-5 at V 300, where fp32's step at 1000 is 6e-5.  The logits are
    exact, so what is off is the sum, whose at most 32 additions of values near 1
    are each off by 2^-24, and the logarithm, by as much."""
    print(f"small losses B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, (0, V), seed=1, ignored=0)
    c.x.zero_(), c.w.zero_()
    c.x[:, 0] = 1
    c.w[0] = 984
    c.w[0, V - 7] = 1000
    c.wt.copy_(c.w)
    c.targets.fill_(V - 7)
    c.targets[1] = -1
    c.targets[2] = 3                               # 16 more
    loss, lse = c.loss()
    small = torch.log1p((V - 1) * torch.exp(torch.tensor(-16.0, dtype=torch.float64))).item()
    want = torch.full((B,), small, dtype=torch.float64, device="cuda")
    want[1], want[2] = 0, 16 + small
    bound = 34 * HALF_FP32 + want * 4 * HALF_FP32
    assert bool(((loss.double() - want).abs() <= bound).all()), (loss[:3].tolist(), small)
    assert bool(((lse.double() - 1000 - small).abs() <= 1001 * 2 * HALF_FP32).all())


@pytest.mark.parametrize("B,H,V", PATHS + [(4096, 264, 4000)])
def test_rows_of_minus_infinity(require_gpu, B, H, V):
    """A row whose logits are all -inf has probability 0 everywhere: an infinite
    loss, and of its gradient only the target's term.  That is what an lse far
    above the logits gives, so the gradient has those bits wherever x is finite."""
    print(f"rows of -inf B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, (0, 152, V), seed=2, ignored=0, scale=0.05)
    c.w[0] = 1
    c.wt.copy_(c.w)
    c.x[:, 0] = 0.5
    c.targets[0], c.targets[2] = 5, -1
    masked = [0, 2] + ([B - 1] if B > 3 else [])
    for b in masked:
        c.x[b, 0] = float("-inf")
    loss, lse = c.loss()
    assert bool((lse[masked] == float("-inf")).all()) and loss[2].item() == 0
    assert bool((loss[[b for b in masked if b != 2]] == float("inf")).all())
    rest = torch.ones(B, dtype=torch.bool, device="cuda")
    rest[masked] = False
    assert bool(loss[rest].isfinite().all()) and bool(lse[rest].isfinite().all())
    dx, dw = c.grad(lse)
    assert bool((dx[2] == 0).all())
    c.x[masked, 0] = 0.5
    far = lse.clone()
    far[masked] = 1e4
    dx2, dw2 = c.grad(far)
    assert torch.equal(dx, dx2) and torch.equal(dw[1:], dw2[1:])
    # one NaN among them: a NaN
    c.x[0, 0], c.x[0, 1] = float("-inf"), float("nan")
    loss, lse = c.loss()
    assert bool(loss[0].isnan()) and bool(lse[0].isnan())
