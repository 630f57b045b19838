"""Layer norm and its gradient on the GPU against their definition in 64 bits
(norm_common), at sizes around units, threads and kernels, with every pair of types."""
import pytest
import torch

from logit_source_projection_amd import sb
from tests import norm_common as ref

pytestmark = pytest.mark.gpu

F, H16 = torch.float32, torch.bfloat16
TYPES = [(F, F, F), (H16, H16, H16), (F, H16, F), (H16, F, F), (F, F, H16), (H16, H16, F)]
SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (4, 9), (7, 63), (17, 64), (9, 511), (6, 512), (33, 520), (5, 1024),
         (257, 1111), (3, 2048), (2, 2056), (19, 4096), (16, 5120), (1, 5120), (3, 6144), (2, 8192), (5, 8200),
         (2, 16384), (3, 16385), (2, 17408), (2, 32768), (2, 40001), (1100, 72), (4099, 24),
         # a gradient of few rows and of one more
         (255, 333), (256, 5120), (257, 5120), (256, 8192), (257, 8192), (256, 8193), (257, 36),
         # every kind of team through several rows each
         (40000, 40), (20000, 104), (10000, 200), (9000, 333), (5000, 520), (3000, 1200), (1600, 5120), (601, 12001)]


def matrix(B, H, dtype, fill, extra=8):
    """A matrix whose padding columns hold `fill`."""
    t = torch.full((B, -(-H // 8) * 8 + extra), fill, dtype=dtype, device="cuda")
    return t, t[:, :H]


def make(B, H, tx, ty, tp, seed, offset=0.5):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    _, x = matrix(B, H, tx, float("nan"))
    x.copy_(normal(B, H) * (0.5 + torch.rand(B, 1, device="cuda", generator=g)) + offset * normal(B, 1))
    _, dy = matrix(B, H, ty, float("nan"))
    dy.copy_(normal(B, H))
    return x, dy, (1 + 0.2 * normal(H)).to(tp), (0.3 * normal(H)).to(tp)


def run(x, dy, w, b, eps=ref.EPS, tp=None):
    """Every output, with the padding of each checked to be left as it was."""
    B, H = x.shape
    n = sb.Norm(x, w, b, eps=eps)
    whole_y, y = matrix(B, H, dy.dtype, -7.0)
    whole_dx, dx = matrix(B, H, x.dtype, -7.0)
    mean, rstd = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    sb.sb_layer_norm(n, y, mean, rstd)
    dw, db = torch.empty(H, dtype=n.param_dtype, device="cuda"), torch.empty(H, dtype=n.param_dtype, device="cuda")
    ws = torch.full((sb.sb_layer_norm_grad_workspace_bytes(n) + 64,), 255, dtype=torch.uint8, device="cuda")
    ws_end = ws[-64:]
    sb.sb_layer_norm_grad(n, dy, mean, rstd, dx, dw, db, ws=ws[:-64])
    assert bool((whole_y[:, H:] == -7).all()) and bool((whole_dx[:, H:] == -7).all()), "padding"
    assert bool((ws_end == 255).all()), "workspace"
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("tx,ty,tp", TYPES)
@pytest.mark.parametrize("B,H", SIZES)
def test_against_definition(require_gpu, B, H, tx, ty, tp):
    print(f"layer norm B={B} H={H} {tx} {ty} {tp}", flush=True)
    x, dy, w, b = make(B, H, tx, ty, tp, 17 * B + H)
    y, mean, rstd, dx, dw, db = run(x, dy, w, b)
    ref.check_forward(y, mean, rstd, x, w, b)
    ref.check_gradient(dx, dw, db, x, w, dy, mean, rstd)


@pytest.mark.parametrize("B,H", [(3, 40), (40, 1111), (2, 5120), (2, 20000)])
def test_without_parameters(require_gpu, B, H):
    x, dy, w, b = make(B, H, H16, H16, F, 5)
    for wt, bs in ((None, None), (w, None), (None, b)):
        y, mean, rstd, dx, dw, db = run(x, dy, wt, bs)
        ref.check_forward(y, mean, rstd, x, wt, bs)
        ref.check_gradient(dx, dw, db, x, wt, dy, mean, rstd)


@pytest.mark.parametrize("B,H", [(5, 264), (300, 1111), (2, 20000)])
def test_any_of_the_outputs(require_gpu, B, H):
    x, dy, w, b = make(B, H, H16, F, F, 6)
    y, mean, rstd, dx, dw, db = run(x, dy, w, b)
    n = sb.Norm(x, w, b)
    only_y = matrix(B, H, F, 0.0)[1]
    assert torch.equal(sb.sb_layer_norm(n, only_y), y)
    for keep in range(1, 7):
        got = sb.sb_layer_norm_grad(n, dy, mean, rstd, matrix(B, H, H16, 0.0)[1] if keep & 1 else None,
                                    torch.empty_like(w) if keep & 2 else None, torch.empty_like(b) if keep & 4 else None)
        for t, want in zip(got, (dx, dw, db)):
            assert t is None or torch.equal(t, want), keep


@pytest.mark.parametrize("B,H", [(1, 64), (255, 40), (256, 40), (2049, 136), (700, 5120)])
def test_sums_of_whole_numbers(require_gpu, B, H):
    """dbias of small whole numbers is exact: no row is lost or taken twice."""
    g = torch.Generator(device="cuda").manual_seed(B)
    dy = torch.randint(-8, 9, (B, H), device="cuda", generator=g).float()
    x = torch.randn(B, H, device="cuda", generator=g)
    *_, dw, db = run(x, dy, None, None)
    assert torch.equal(db, dy.double().sum(0).float())
    # xh of two values is +-1 exactly for eps = 0: dweight is exact too
    x = torch.randint(0, 2, (B, H // 2), device="cuda", generator=g).float()
    x = torch.cat([x, 1 - x], 1) * 2 - 1
    *_, dw, db = run(x, dy, None, None, eps=0.0)
    assert torch.equal(dw, (dy.double() * x.double()).sum(0).float())


def test_gradient_against_differences(require_gpu):
    """Central differences of the definition in 64 bits, in random directions."""
    x, dy, w, b = make(6, 45, F, F, F, 9)
    _, mean, rstd, dx, dw, db = run(x, dy, w, b)
    g = torch.Generator(device="cuda").manual_seed(1)
    for t, grad in ((x, dx), (w, dw), (b, db)):
        for _ in range(4):
            v = torch.randn(t.shape, dtype=torch.float64, device="cuda", generator=g)
            h = 1e-6
            ends = []
            for sign in (h, -h):
                args = [a.double() + sign * v if a is t else a.double() for a in (x, w, b)]
                ends.append((ref.forward(*args)[0] * dy.double()).sum())
            slope, got = (ends[0] - ends[1]) / (2 * h), (grad.double() * v).sum()
            # differences are good to h^2 and 1e-16 / h; the gradient to 2^-24 of about 60 terms each
            assert abs(slope - got) <= 1e-5 * (grad.double().abs() * v.abs()).sum(), (slope, got)


@pytest.mark.parametrize("H", [64, 1111, 5120, 20000])
def test_values_that_are_not_finite_stay_in_their_row(require_gpu, H):
    x, dy, w, b = make(40, H, F, F, F, 11)
    clean = run(x, dy, w, b)
    bad = x.clone()
    bad[3, H // 2], bad[17, 0], bad[39, H - 1] = float("nan"), float("inf"), -float("inf")
    got = run(matrix(40, H, F, 0.0)[1].copy_(bad), dy, w, b)
    rows = torch.ones(40, dtype=torch.bool, device="cuda")
    rows[[3, 17, 39]] = False
    for a, c in zip(got[:4], clean[:4]):
        assert torch.equal(a[rows], c[rows])
    for t in (got[0], got[3]):
        assert bool(t[~rows].isnan().all())
    assert torch.equal(got[5], clean[5])  # dbias takes dy alone


@pytest.mark.parametrize("H", [8, 100, 5120, 20000])
def test_rows_of_one_value(require_gpu, H):
    """A whole number's mean is exact: y is the bias."""
    x = torch.full((5, H), 3.0, device="cuda")
    dy, w, b = torch.ones(5, H, device="cuda"), torch.randn(H, device="cuda"), torch.randn(H, device="cuda")
    y, mean, rstd, dx, *_ = run(x, dy, w, b)
    assert bool((mean == 3).all()) and torch.equal(y, b.expand(5, H))
    assert bool(run(x, dy, w, b, eps=0.0)[0].isnan().all())


def test_far_from_zero(require_gpu):
    """A mean a thousand times the deviation: the variance keeps its digits."""
    x, dy, w, b = make(9, 2000, F, F, F, 13, offset=1000.0)
    y, mean, rstd, dx, dw, db = run(x, dy, w, b)
    ref.check_forward(y, mean, rstd, x, w, b)
    ref.check_gradient(dx, dw, db, x, w, dy, mean, rstd)


@pytest.mark.parametrize("B,H", [(70000, 16), (1 << 21, 8)])
def test_many_rows(require_gpu, B, H):
    x, dy, w, b = make(B, H, H16, H16, F, 15)
    y, mean, rstd, dx, dw, db = run(x, dy, w, b)
    ref.check_forward(y, mean, rstd, x, w, b)
    ref.check_gradient(dx, dw, db, x, w, dy, mean, rstd)


@pytest.mark.parametrize("B,H,ld", [(3, 520, 1 << 30), (300, 520, 1 << 23), (3, 20000, 1 << 30)])
def test_rows_far_apart(require_gpu, B, H, ld):
    """Offsets past 32 bits give what the same rows give side by side."""
    x, dy, w, b = make(B, H, H16, H16, F, 18)
    want = run(x, dy, w, b)

    def far():
        return torch.empty((B - 1) * ld + H, dtype=H16, device="cuda").as_strided((B, H), (ld, 1))

    n, g, y, dx = sb.Norm(far().copy_(x), w, b), far().copy_(dy), far(), far()
    mean, rstd, dw, db = (torch.empty_like(t) for t in (*want[1:3], *want[4:]))
    sb.sb_layer_norm(n, y, mean, rstd)
    sb.sb_layer_norm_grad(n, g, mean, rstd, dx, dw, db)
    for got, ref_ in zip((y, mean, rstd, dx, dw, db), want):
        assert torch.equal(got, ref_)


def test_no_rows(require_gpu):
    w, b = torch.randn(24, device="cuda"), torch.randn(24, device="cuda")
    n = sb.Norm(torch.empty(0, 24, device="cuda"), w, b)
    e, v = torch.empty(0, 24, device="cuda"), torch.empty(0, device="cuda")
    sb.sb_layer_norm(n, e, v, v)
    dw, db = torch.ones(24, device="cuda"), torch.ones(24, device="cuda")
    sb.sb_layer_norm_grad(n, e, v, v, None, dw, db)
    assert not dw.any() and not db.any()


def test_same_bits_again(require_gpu):
    x, dy, w, b = make(1500, 1111, H16, H16, H16, 21)
    one, two = run(x, dy, w, b), run(x, dy, w, b)
    assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_refusals_of_the_binding(require_gpu):
    x, dy, w, b = make(4, 16, F, F, F, 1)
    v = torch.empty(4, device="cuda")
    n = sb.Norm(x, w, b)
    y = torch.empty(4, 16, device="cuda")
    for call, error in (
            (lambda: sb.sb_layer_norm(sb.Norm(x.half(), w, b), y), TypeError),
            (lambda: sb.sb_layer_norm(sb.Norm(x, w, b.bfloat16()), y), TypeError),
            (lambda: sb.sb_layer_norm(sb.Norm(x, w[:8], b), y), ValueError),
            (lambda: sb.sb_layer_norm(sb.Norm(x, w, b, B=5), y), ValueError),
            (lambda: sb.sb_layer_norm(n, y.half()), TypeError),
            (lambda: sb.sb_layer_norm(n, y[:3]), ValueError),
            (lambda: sb.sb_layer_norm(n, y.t()), ValueError),
            (lambda: sb.sb_layer_norm(n, y, v[:3]), ValueError),
            (lambda: sb.sb_layer_norm(n, y, v.double()), TypeError),
            (lambda: sb.sb_layer_norm_grad(n, dy, v, v, dx=y.bfloat16()), TypeError),
            (lambda: sb.sb_layer_norm_grad(n, dy, None, v, dx=y), sb.SbError),
            (lambda: sb.sb_layer_norm_grad(n, dy, v, v), sb.SbError),
            (lambda: sb.sb_layer_norm_grad(n, dy, v, v, dweight=w.bfloat16()), TypeError),
            (lambda: sb.sb_layer_norm_grad(n, dy.expand(4, 16)[:1].expand(4, 16), v, v, dx=y), sb.SbError)):
        with pytest.raises(error):
            call()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("B,H", [(40, 64), (40, 1111), (300, 1111), (300, 5120), (40, 20000)])
def test_where_values_that_are_not_finite_go_in_the_gradient(require_gpu, B, H, bad):
    x, dy, w, b = make(B, H, F, F, F, 12)
    clean = run(x, dy, w, b)
    rows = torch.arange(B, device="cuda") != 17
    columns = torch.arange(H, device="cuda") != H // 2
    # one in x: its rows of y, rstd and dx, and all of dweight
    hit = matrix(B, H, F, 0.0)[1].copy_(x)
    hit[17, H // 2] = bad
    y, mean, rstd, dx, dw, db = run(hit, dy, w, b)
    for t, c in ((y, clean[0]), (rstd, clean[2]), (dx, clean[3])):
        assert bool(t[17].isnan().all()) and torch.equal(t[rows], c[rows])
    assert bool(dw.isnan().all()) and torch.equal(db, clean[5])
    # one in dy: its row of dx, and its column of dweight and dbias
    hit = matrix(B, H, F, 0.0)[1].copy_(dy)
    hit[17, H // 2] = bad
    _, _, _, dx, dw, db = run(x, hit, w, b)
    assert not dx[17].isfinite().any() and torch.equal(dx[rows], clean[3][rows])
    for t, c in ((dw, clean[4]), (db, clean[5])):
        assert not t[H // 2].isfinite() and torch.equal(t[columns], c[columns])
