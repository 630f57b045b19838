"""The 64-bit reference of the loss and its gradient, on the CPU: against
torch's cross entropy and its autograd, and against central differences."""
import pytest
import torch

from tests.loss_common import reference, reference_grad


def _case(B, H, V, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, generator=g, dtype=torch.float64)
    w = 0.3 * torch.randn(H, V, generator=g, dtype=torch.float64)
    t = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    if B > 2:
        t[1] = -100
    return x, w, t, torch.rand(B, generator=g, dtype=torch.float64) + 0.5


@pytest.mark.parametrize("B,H,V", [(1, 1, 1), (4, 7, 13), (9, 16, 300)])
def test_reference_is_torchs_cross_entropy(B, H, V):
    x, w, t, d = _case(B, H, V, 3)
    x.requires_grad_(), w.requires_grad_()
    ref = torch.nn.functional.cross_entropy(x @ w, t.long(), reduction="none", ignore_index=-100)
    gx, gw = torch.autograd.grad((ref * d).sum(), (x, w))
    x, w = x.detach(), w.detach()
    _, lse, loss = reference(x, w, t)
    assert torch.allclose(loss, ref.detach(), rtol=1e-12, atol=1e-12)
    _, dx, dw = reference_grad(x, w, t, d, lse)
    assert torch.allclose(dx, gx, rtol=1e-10, atol=1e-12)
    assert torch.allclose(dw, gw, rtol=1e-10, atol=1e-12)


def test_reference_gradient_against_differences():
    x, w, t, d = _case(5, 6, 11, 4)
    _, lse, _ = reference(x, w, t)
    _, dx, dw = reference_grad(x, w, t, d, lse)
    eps = 1e-5

    def total(x, w):
        return (reference(x, w, t)[2] * d).sum()

    for tensor, grad in ((x, dx), (w, dw)):
        for i in range(tensor.shape[0]):
            for j in range(tensor.shape[1]):
                keep = tensor[i, j].item()
                tensor[i, j] = keep + eps
                up = total(x, w)
                tensor[i, j] = keep - eps
                down = total(x, w)
                tensor[i, j] = keep
                # third-order term below eps^2, cancellation below 1e-15 / eps
                assert abs((up - down) / (2 * eps) - grad[i, j]) < 1e-8
