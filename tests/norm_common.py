"""Layer norm and its gradient in 64 bits, from their definition, and how far
fp32 sums and one rounding of every result may put them from it.

u = 2^-24 is half a step of fp32.  A sum whose longest chain has d additions is
off by at most d u times the sum of its magnitudes; the kernels deal a row to 64
threads or more, so d is at most H / 64 + 32 (eight values of a unit, the
units of a thread, and fewer than 20 levels over threads).  Sums over rows may be
in any order: d is at most B + 16.
"""
import torch

U = 2.0 ** -24
EPS = 1e-5


def half(dtype):
    return torch.finfo(dtype).eps / 2


def forward(x, weight, bias, eps=EPS):
    x = x.double()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / ((d * d).mean(1) + eps).sqrt()
    y = d * rstd[:, None]
    if weight is not None:
        y = y * weight.double()
    if bias is not None:
        y = y + bias.double()
    return y, mean, rstd


def check_forward(y, mean, rstd, x, weight, bias, eps=EPS):
    H = x.shape[1]
    chain = H / 64 + 32
    ry, rm, rr = forward(x, weight, bias, eps)
    xa = x.double().abs()
    em = (chain + 2) * U * xa.mean(1) + 2.0 ** -149
    # the differences from the mean found: their squares sum to the variance plus em^2,
    # each off by a rounding of the difference and one of the square
    d = x.double() - rm[:, None]
    var = (d * d).mean(1)
    ev = em ** 2 + (chain + 6) * U * (var + em ** 2) + 2 * U * (d.abs().mean(1) * em)
    er = rr * (0.5 * ev / (var + eps) * 1.01 + 6 * U)
    assert bool(((mean.double() - rm).abs() <= em).all()), "mean"
    assert bool(((rstd.double() - rr).abs() <= er).all()), "rstd"
    w = 1.0 if weight is None else weight.double().abs()
    b = 0.0 if bias is None else bias.double().abs()
    scaled = d.abs() * rr[:, None] * w
    e = w * ((em * rr)[:, None] + d.abs() * er[:, None]) * 1.01 + 4 * U * scaled + U * b
    bound = e + half(y.dtype) * (ry.abs() + e) + 2.0 ** -133
    off = (y.double() - ry).abs()
    assert bool((off <= bound).all()), f"y off by {(off / bound).max().item()} of its bound"


def gradient(x, weight, dy, mean, rstd):
    """dx, dweight and dbias in 64 bits; mean and rstd are the ones that the gradient is given."""
    r = rstd.double()[:, None]
    xh = (x.double() - mean.double()[:, None]) * r
    dy = dy.double()
    g = dy if weight is None else dy * weight.double()
    dx = r * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def check_gradient(dx, dweight, dbias, x, weight, dy, mean, rstd):
    B, H = x.shape
    chain = H / 64 + 32
    rx, rw, rb = gradient(x, weight, dy, mean, rstd)
    r = rstd.double()[:, None]
    xh = ((x.double() - mean.double()[:, None]) * r).abs()  # off by 2 u of itself
    dya = dy.double().abs()
    g = dya if weight is None else dya * weight.double().abs()
    if dx is not None:
        sg, sk = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
        eg, ek = (chain + 3) * U * sg, (chain + 6) * U * sk
        e = r * (eg + xh * ek + 8 * U * (g + sg + xh * sk))
        bound = e + half(dx.dtype) * (rx.abs() + e) + 2.0 ** -133
        off = (dx.double() - rx).abs()
        assert bool((off <= bound).all()), f"dx off by {(off / bound).max().item()} of its bound"
    for name, got, ref, terms in (("dweight", dweight, rw, (dya * xh).sum(0)), ("dbias", dbias, rb, dya.sum(0))):
        if got is None:
            continue
        e = (B + 16) * U * terms
        bound = e + half(got.dtype) * (ref.abs() + e) + 2.0 ** -133
        off = (got.double() - ref).abs()
        assert bool((off <= bound).all()), f"{name} off by {(off / bound).max().item()} of its bound"
