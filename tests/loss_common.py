"""The loss and its gradient in 64 bits, from their definition, and how far
fp32 accumulation and bf16 rounding may put a result from them.

  z = x w, lse = log sum exp z, loss = lse - z[target] (0 where target < 0)
  dz = (softmax(z) - onehot) * dloss (0 where target < 0)
  dx = dz w^T, dw = x^T dz

The bounds are worst cases: a sum of n products in fp32 is off by at most
(n + 8) 2^-24 times the sum of their magnitudes, a value rounded to bf16 by at
most 2^-8 of itself, and the exponential of an argument a by (|a| + 4) 2^-23 of
itself (the argument's product with log2 e is rounded once, the instruction is
good to an ulp).
"""
import torch

HALF_BF16 = 2.0 ** -8
HALF_FP32 = 2.0 ** -24


def reference(x, w, targets):
    """z, lse and loss in 64 bits."""
    z = x.double() @ w.double()
    lse = torch.logsumexp(z, 1)
    kept = targets >= 0
    at = targets.long().clamp(min=0)[:, None]
    loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
    return z, lse, loss


def reference_grad(x, w, targets, dloss, lse):
    """dz, dx and dw in 64 bits; lse is the one the gradient is given."""
    x, w = x.double(), w.double()
    kept = targets >= 0
    rows = torch.nonzero(kept)[:, 0]
    dz = torch.exp(x @ w - lse.double()[:, None])
    dz[rows, targets[rows].long()] -= 1
    dz = torch.where(kept[:, None], dz * dloss.double()[:, None], 0.0)
    return dz, dz @ w.t(), torch.where(kept[:, None], x, 0.0).t() @ dz


def logit_bound(x, w):
    """Per row: how far any fp32 logit may be off."""
    H = x.shape[1]
    return (H + 8) * HALF_FP32 * (x.double().abs() @ w.double().abs()).amax(1)


def loss_bounds(x, w, z, lse, loss):
    """Per row: (lse, loss) bounds.  lse moves by at most what the logits do,
    plus the relative error of its sum of V exponentials and of the logarithm."""
    zb = logit_bound(x, w)
    spread = z.amax(1) - z.amin(1)
    blocks = z.shape[1] // 256 + 80
    sums = (blocks + 64) * HALF_FP32 + (spread.clamp(max=104) + 4) * 2 * HALF_FP32
    lb = zb + sums + (lse.abs() + 1) * 2.0 ** -22
    return lb, lb + zb + (lse.abs() + z.abs().amax(1)) * 2 * HALF_FP32


def check_loss(got_loss, got_lse, x, w, targets):
    z, lse, loss = reference(x, w, targets)
    lb, ob = loss_bounds(x, w, z, lse, loss)
    e = (got_lse.double() - lse).abs()
    assert bool((e <= lb).all()), f"lse off by {e.max().item()}, bound {lb.min().item()}"
    e = (got_loss.double() - loss).abs()
    assert bool((e <= ob).all()), f"loss off by {e.max().item()}, bound {ob.min().item()}"
    assert bool((got_loss[targets < 0] == 0).all())


def check_grad(dx, dw, x, w, targets, dloss, lse):
    """Elementwise worst-case bounds, and the 2-norm against the spread of
    independent roundings: each is off by at most sqrt(3) times its root mean
    square, which 1.75 covers however few terms there are."""
    dz, rx, rw = reference_grad(x, w, targets, dloss, lse)
    kept = (targets >= 0)[:, None]
    zb = logit_bound(x, w)[:, None]
    p = torch.where(kept, torch.exp(x.double() @ w.double() - lse.double()[:, None]), 0.0)
    # exp(z - lse): the logit's error, the subtraction's and the exponential's
    arg = (x.double() @ w.double() - lse.double()[:, None]).abs()
    ferr = p * dloss.double().abs()[:, None] * (zb + (arg.clamp(max=104) + 8) * 2 * HALF_FP32)
    ferr = ferr + 4 * HALF_FP32 * dz.abs()
    err = ferr + HALF_BF16 * (dz.abs() + ferr)
    xa = torch.where(kept, x.double(), 0.0).abs()
    for name, got, ref, worst, terms, squares in (
            ("dx", dx, rx, err @ w.double().abs().t(), dz.abs() @ w.double().abs().t(),
             (dz ** 2) @ (w.double() ** 2).t()),
            ("dw", dw, rw, xa.t() @ err, xa.t() @ dz.abs(), (xa ** 2).t() @ (dz ** 2))):
        if got is None:
            continue
        n = w.shape[1] if name == "dx" else x.shape[0]
        bound = worst + (n + 40) * HALF_FP32 * terms
        # bf16 keeps 2^-8 of a value down to 2^-126; below that its step is 2^-133
        bound = bound + HALF_BF16 * (ref.abs() + bound) + 2.0 ** -133
        e = (got.double() - ref).abs()
        assert bool((e <= bound).all()), \
            f"{name} off by {e.max().item()}, {(e / bound).max().item()} of its bound"
        spread = (HALF_BF16 ** 2 / 3 * (squares.sum() + (ref ** 2).sum())).sqrt()
        fp32 = torch.linalg.vector_norm(bound - HALF_BF16 * ref.abs() - worst) + \
            torch.linalg.vector_norm(ferr) * torch.linalg.vector_norm(w.double() if name == "dx" else x.double().nan_to_num(0, 0, 0))
        norm = torch.linalg.vector_norm(got.double() - ref)
        assert norm <= 1.75 * spread + fp32, f"{name} off by {norm.item()} in all, {spread.item()} expected"
