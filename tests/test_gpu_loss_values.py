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
