"""The check of the gradient's exactness, on the CPU: results of the form it
describes pass, and ones that lost part of it do not."""
import pytest
import torch

from tests.grad_accuracy import check_grad_exactness
from tests.loss_common import reference, reference_grad


def results(B, H, V, form, spread=0.5):
    """The gradient's results in bf16 with dz in the given form; the products in 64 bits.
    The logits' standard deviation is `spread`."""
    g = torch.Generator().manual_seed(B)
    x = torch.randn(B, H, generator=g).to(torch.bfloat16)
    w = (torch.randn(H, V, generator=g) * spread / H ** 0.5).to(torch.bfloat16)
    t = torch.randint(0, V, (B,), generator=g, dtype=torch.int32)
    if B > 2:
        t[2] = -100
    d = torch.randn(B, generator=g)
    lse = reference(x, w, t)[1].float()
    dz = reference_grad(x, w, t, d, lse)[0]
    hi = dz.to(torch.bfloat16).double()
    lo = (dz - hi).to(torch.bfloat16).double()
    rows = torch.nonzero(t >= 0)[:, 0]
    at_target = torch.zeros_like(hi)
    at_target[rows, t[rows].long()] = lo[rows, t[rows].long()]
    held = {"two parts": hi + lo, "one part": hi, "target": hi + at_target,
            "parts of other rows": hi + lo.roll(1, 0), "taken off": hi - at_target}[form]
    kept = (t >= 0)[:, None]
    return ((held @ w.double().t()).to(torch.bfloat16),
            (torch.where(kept, x.double(), 0.0).t() @ held).to(torch.bfloat16), x, w, t, d, lse)


FEW, MANY = [(1, 40, 700), (7, 129, 2000), (32, 200, 3000)], [(33, 200, 3000), (300, 96, 4000)]


@pytest.mark.parametrize("size,form", [(s, "two parts") for s in FEW + MANY] + [(s, "target") for s in MANY])
def test_the_forms_pass(size, form):
    check_grad_exactness(*results(*size, form))


@pytest.mark.parametrize("size,form", [(s, "one part") for s in FEW] +
                         [(s, "parts of other rows") for s in FEW[1:]] +
                         [(s, f) for s in MANY for f in ("one part", "taken off")])
def test_a_lost_part_is_seen(size, form):
    dx, dw, *rest = results(*size, form)
    for pair in ((dx, None), (None, dw)):
        with pytest.raises(AssertionError):
            check_grad_exactness(*pair, *rest)


@pytest.mark.parametrize("size", FEW)
def test_a_lost_part_of_other_terms_is_seen(size):
    """Logits so far apart that columns besides the target's hold much of a row."""
    check_grad_exactness(*results(*size, "two parts", spread=6))
    for form in ("one part", "target"):
        dx, dw, *rest = results(*size, form, spread=6)
        for pair in ((dx, None), (None, dw)):
            with pytest.raises(AssertionError):
                check_grad_exactness(*pair, *rest)
