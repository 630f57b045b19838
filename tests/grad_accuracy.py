"""How exact the gradient's dz is held, and a check that tells: bounds that count
one rounding of the bf16 result and, of dz's, only what its form allows.

Up to 32 rows dz is the sum of two bf16 numbers: off by at most 2^-16 of itself.
Above, so is the dz of a row's target; the others are bf16, off by at most 2^-8.
Above 64 rows the target's term of dx is made whole by a factor of the row, within
2^-8 of 1, which the sum of the others takes too.
"""
import torch

from tests.loss_common import HALF_BF16, HALF_FP32, logit_bound, reference_grad

TWO_PARTS = 2.0 ** -16


def dz_rounding(targets, V):
    """Relative bound on the rounding of every dz."""
    B = targets.shape[0]
    half = torch.full((B, V), TWO_PARTS if B <= 32 else HALF_BF16, dtype=torch.float64,
                      device=targets.device)
    rows = torch.nonzero((targets >= 0) & (targets < V))[:, 0]
    half[rows, targets[rows].long()] = TWO_PARTS
    return half


def check_grad_exactness(dx, dw, x, w, targets, dloss, lse):
    """Every element within the worst case, and the errors' norm within that of
    the results' own rounding (measured on the reference; the result rounds other
    values of the same size, whose mean square differs by some 1/sqrt(n) over n
    elements, below 5 % from a few thousand on) and of dz's."""
    dz, rx, rw = reference_grad(x, w, targets, dloss, lse)
    kept = (targets >= 0)[:, None]
    xd, wd = torch.where(kept, x.double(), 0.0), w.double()
    z = x.double() @ wd
    arg = (z - lse.double()[:, None]).abs()
    p = torch.where(kept, torch.exp(z - lse.double()[:, None]), 0.0)
    # exp(z - lse) in fp32: the logit's error, the subtraction's, the exponential's
    ferr = p * dloss.double().abs()[:, None] * \
        (logit_bound(x, w)[:, None] + (arg.clamp(max=104) + 8) * 2 * HALF_FP32)
    ferr = ferr + 4 * HALF_FP32 * dz.abs()
    half = dz_rounding(targets, w.shape[1])
    err = ferr + half * (dz.abs() + ferr)
    rms2 = (half * dz) ** 2 / 3
    moved = torch.zeros_like(rx)  # what the row's factor may move of dx
    if x.shape[0] > 64:
        moved = HALF_BF16 * (torch.where(half == TWO_PARTS, 0.0, dz) @ wd.t()).abs()
    for name, got, ref, worst, terms, square, n, fp32 in (
            ("dx", dx, rx, err @ wd.abs().t() + moved, dz.abs() @ wd.abs().t(),
             rms2 @ (wd ** 2).t() + moved ** 2 / 3, w.shape[1], ferr @ wd.abs().t()),
            ("dw", dw, rw, xd.abs().t() @ err, xd.abs().t() @ dz.abs(), (xd ** 2).t() @ rms2,
             x.shape[0], xd.abs().t() @ ferr)):
        if got is None:
            continue
        sums = (n + 40) * HALF_FP32 * terms
        bound = worst + sums
        bound = bound + HALF_BF16 * (ref.abs() + bound) + 2.0 ** -133
        e = (got.double() - ref).abs()
        assert bool((e <= bound).all()), \
            f"{name} off by {e.max().item()}, {(e / bound).max().item()} of its bound"
        own = torch.linalg.vector_norm(ref.to(torch.bfloat16).double() - ref)
        norm = torch.linalg.vector_norm(e)
        limit = 1.05 * own + 1.75 * square.sum().sqrt() + torch.linalg.vector_norm(fp32 + sums)
        assert ref.numel() < 4000 or norm <= limit, \
            f"{name} off by {norm.item()} in all, {limit.item()} allowed, {own.item()} its own rounding"
