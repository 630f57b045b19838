"""Embedding lookup and its gradient on the GPU.

A lookup is one fp32 product, rounded to the output's type: compared for equality.
Gradients of small whole numbers are exact in fp32 sums whatever their order, so
those are compared for equality too (a lost, doubled or misplaced position shows at
once).  Of other values a sum of n terms is off by at most (n + 16) 2^-24 of the
sum of their magnitudes, and the result by one rounding."""
import math

import pytest
import torch

from logit_source_projection_amd import sb

pytestmark = pytest.mark.gpu

F, H16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def matrix(B, H, dtype, fill, extra=8):
    t = torch.full((B, -(-H // 8) * 8 + extra), fill, dtype=dtype, device="cuda")
    return t, t[:, :H]


def lanes(V, k):
    return [V * i // k for i in range(k)] + [V]


def split(t, off):
    """Each lane in an allocation of its own, with one row stride."""
    out = []
    for i in range(len(off) - 1):
        whole, part = matrix(off[i + 1] - off[i], t.shape[1], t.dtype, float("nan"))
        part.copy_(t[off[i]:off[i + 1]])
        out.append(part)
    return out


def make_ids(kind, B, V, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    i = torch.arange(B, device="cuda")
    if kind == "uniform":
        ids = torch.randint(0, V, (B,), device="cuda", generator=g)
    elif kind == "one":
        ids = torch.full((B,), V - 1, device="cuda")
    elif kind == "ranks":
        ids = (torch.rand(B, device="cuda", generator=g) * math.log(V + 1)).exp().long().clamp(1, V) - 1
    elif kind == "bytes":
        ids = torch.randint(0, min(V, 100), (B,), device="cuda", generator=g) + max(0, V // 2 - 100)
    elif kind == "falling":
        ids = (V - 1 - i % V)
    elif kind == "padded":  # padding, IDs past the table and the largest and smallest numbers among them
        ids = torch.randint(0, V, (B,), device="cuda", generator=g)
        ids[i % 3 == 1] = -1
        ids[i % 7 == 2] = V
        ids[i % 11 == 3] = -2 ** 31
        ids[i % 13 == 4] = 2 ** 31 - 1
    elif kind == "none":
        ids = torch.full((B,), -100, device="cuda")
    elif kind == "pairs":  # segments that end where runs do
        ids = torch.sort(torch.randint(0, V, (B // 64 + 1,), device="cuda", generator=g))[0].repeat_interleave(64)[:B]
    return ids.to(torch.int32)


def reference_grad(ids, dout, V, scale):
    keep = (ids >= 0) & (ids < V)
    at = ids[keep].long()
    out = torch.zeros(V, dout.shape[1], dtype=torch.float64, device="cuda")
    return out.index_add_(0, at, dout[keep].double()) * scale


LOOKUPS = [(1, 1, 1, 1), (3, 7, 5, 2), (16, 1000, 64, 3), (5, 4096, 2056, 4), (257, 50257, 111, 5), (64, 300, 5120, 1),
           (2000, 999, 72, 64), (3, 17, 8192, 17), (70000, 50, 8, 7)]


@pytest.mark.parametrize("tt,to", [(F, F), (F, H16), (H16, F), (H16, H16)])
@pytest.mark.parametrize("B,V,H,k", LOOKUPS)
def test_lookup(require_gpu, B, V, H, k, tt, to):
    print(f"embed B={B} V={V} H={H} k={k} {tt} {to}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(B + V)
    _, w = matrix(V, H, tt, float("nan"))
    w.copy_(torch.randn(V, H, device="cuda", generator=g))
    ids = make_ids("padded", B, V, 3)
    want = w.float()[ids.long().clamp(0, V - 1)] * 2.7
    want = torch.where((ids < 0)[:, None], 0.0, torch.where((ids >= V)[:, None], float("nan"), want)).to(to)
    off = lanes(V, k)
    for table in (sb.Table(w, off), sb.Table(split(w, off), off)):
        whole, out = matrix(B, H, to, -7.0)
        sb.sb_embed(table, ids, out, scale=2.7)
        assert torch.equal(out.nan_to_num(123.0), want.nan_to_num(123.0)) and torch.equal(out.isnan(), want.isnan())
        assert bool((whole[:, H:] == -7).all()), "padding"


KINDS = ["uniform", "one", "ranks", "bytes", "falling", "padded", "none", "pairs"]
GRADS = [(1, 1, 1, 1), (1, 1000, 8, 3), (63, 300, 40, 2), (64, 7, 16, 1), (65, 7, 16, 4), (128, 2, 2056, 2),
         (129, 50257, 24, 1), (1000, 4096, 100, 3), (4095, 20, 8, 20), (4097, 151936, 8, 4), (10000, 50257, 37, 5),
         (33333, 5000, 16, 64), (70001, 200064, 8, 3)]


@pytest.mark.parametrize("add", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,V,H,k", GRADS)
def test_gradient_of_whole_numbers(require_gpu, B, V, H, k, kind, add):
    print(f"embed gradient B={B} V={V} H={H} k={k} {kind} add={add}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(B + V)
    ids = make_ids(kind, B, V, 5)
    to = (F, H16)[B % 2]
    _, dout = matrix(B, H, to, float("nan"))
    dout.copy_(torch.randint(-8, 9, (B, H), device="cuda", generator=g))
    keep = (ids >= 0) & (ids < V)
    dout[~keep] = float("nan")  # padding may hold anything
    want = reference_grad(ids, dout, V, 0.5)
    off = lanes(V, k)
    whole, dw = matrix(V, H, F, 3.0)
    table = sb.Table(dw, off)
    n = sb.sb_embed_grad_workspace_bytes(table, B, add)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    sb.sb_embed_grad(table, ids, dout, scale=0.5, accumulate=add, ws=ws[:n])
    assert torch.equal(dw, (want + 3 if add else want).float())
    assert bool((whole[:, H:] == 3).all()), "padding"
    assert bool((ws[n:] == 255).all()), "workspace"


@pytest.mark.parametrize("B", [3000, 16384, 16385, 50000])
@pytest.mark.parametrize("tokens", [[5, 261, 517], [5, 6, 261, 40000], list(range(3, 256 * 40, 256)), [0, 50256]])
def test_tokens_that_fill_the_batch(require_gpu, tokens, B):
    """A few tokens, some of them of one group of the sort, make most of the batch."""
    V, H = 50257, 24
    g = torch.Generator(device="cuda").manual_seed(B)
    ids = torch.tensor(tokens, dtype=torch.int32, device="cuda")[torch.randint(0, len(tokens), (B,), device="cuda", generator=g)]
    rare = torch.rand(B, device="cuda", generator=g) < 0.1
    ids = torch.where(rare, make_ids("uniform", B, V, 1), ids)
    dout = torch.randint(-8, 9, (B, H), device="cuda", generator=g).float()
    dw = torch.empty(V, H, device="cuda")
    sb.sb_embed_grad(sb.Table(dw, lanes(V, 5)), ids, dout)
    assert torch.equal(dw, reference_grad(ids, dout, V, 1.0).float())


@pytest.mark.parametrize("V", [256 * 4096, 256 * 4096 + 1, 3000017])
def test_large_vocabularies(require_gpu, V):
    ids = torch.cat([make_ids("uniform", 3000, V, 1), make_ids("padded", 500, V, 2), make_ids("one", 100, V, 3)])
    dout = torch.randint(-8, 9, (len(ids), 16), device="cuda").float()
    dw = torch.empty(V, 16, device="cuda")
    sb.sb_embed_grad(sb.Table(dw, lanes(V, 3)), ids, dout)
    assert torch.equal(dw, reference_grad(ids, dout, V, 1.0).float())


def test_a_table_that_is_zeroed_in_turns(require_gpu):
    """More than 2^31 16-byte chunks of zeros: a table of 33 GiB."""
    V, H = 1 << 24, 528
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of memory")
    dw = torch.empty(V, H, device="cuda")
    dw.fill_(1.0)
    ids = torch.tensor([V - 1, 0, V - 2, V // 2, V - 1], dtype=torch.int32, device="cuda")
    sb.sb_embed_grad(sb.Table(dw, [0, 5000000, V]), ids, torch.ones(5, H, device="cuda"))
    rows = torch.cat([part.any(1) for part in dw.split(1 << 20)]).nonzero()[:, 0]
    assert torch.equal(rows, ids.long().unique())
    assert bool((dw[V - 1] == 2).all()) and bool((dw[[0, V - 2, V // 2]] == 1).all())
    del dw
    torch.cuda.empty_cache()


@pytest.mark.parametrize("tt", [F, H16])
@pytest.mark.parametrize("to", [F, H16])
@pytest.mark.parametrize("B,V,H,k", [(700, 300, 264, 3), (5000, 20000, 40, 4), (300, 10, 5120, 2), (64, 4096, 8192, 1)])
def test_gradient_of_any_numbers(require_gpu, B, V, H, k, tt, to):
    g = torch.Generator(device="cuda").manual_seed(B)
    ids = make_ids("ranks", B, V, 7)
    _, dout = matrix(B, H, to, float("nan"))
    dout.copy_(torch.randn(B, H, device="cuda", generator=g))
    want, terms = reference_grad(ids, dout, V, 11.3), reference_grad(ids, dout.abs(), V, 11.3)
    count = torch.bincount(ids.long(), minlength=V)[:, None]
    # the scale as fp32 is off by 2^-24, the product by as much, the sum by its additions
    e = (count + 18) * U * terms
    half = torch.finfo(tt).eps / 2
    off = lanes(V, k)
    for separate in (False, True):
        dw = torch.full((V, H), 9.0, dtype=tt, device="cuda")
        parts = split(dw, off) if separate else dw
        sb.sb_embed_grad(sb.Table(parts, off), ids, dout, scale=11.3)
        got = torch.cat(parts) if separate else parts
        bound = e + half * (want.abs() + e)
        assert bool(((got.double() - want).abs() <= bound).all())
        assert bool((got[count[:, 0] == 0] == 0).all())
        # added to what is there: one rounding more of the sum
        before = torch.randn(V, H, device="cuda", generator=g).to(tt)
        parts = split(before, off) if separate else before.clone()
        sb.sb_embed_grad(sb.Table(parts, off), ids, dout, scale=11.3, accumulate=True)
        got = torch.cat(parts) if separate else parts
        both = want + before.double()
        bound = e + U * both.abs() + half * (both.abs() + e)
        assert bool(((got.double() - both).abs() <= bound).all())
        same = count[:, 0] == 0
        assert torch.equal(got[same], before[same])


def test_gradient_against_differences(require_gpu):
    """The lookup is linear: a step along any direction changes sum(dout * out) by
    the gradient's product with it, exactly in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(3)
    V, H, B = 50, 24, 300
    w, dout = torch.randn(V, H, device="cuda", generator=g), torch.randn(B, H, device="cuda", generator=g)
    ids = make_ids("padded", B, V, 1)
    keep = (ids >= 0) & (ids < V)
    dw = torch.empty(V, H, device="cuda")
    sb.sb_embed_grad(sb.Table(dw), ids, dout, scale=3.0)

    def value(t):
        return (3.0 * t[ids[keep].long()] * dout[keep].double()).sum()

    for _ in range(4):
        v = torch.randn(V, H, dtype=torch.float64, device="cuda", generator=g)
        slope = (value(w.double() + v) - value(w.double() - v)) / 2
        assert abs(slope - (dw.double() * v).sum()) <= 30 * U * (dw.double().abs() * v.abs()).sum() + 1e-9


def test_values_that_are_not_finite_stay_with_their_token(require_gpu):
    ids = make_ids("ranks", 2000, 400, 2)
    dout = torch.randint(-8, 9, (2000, 40), device="cuda").float()
    want = reference_grad(ids, dout, 400, 1.0).float()
    at = int(ids[1234])
    dout[1234, 17] = float("inf")
    dw = torch.empty(400, 40, device="cuda")
    sb.sb_embed_grad(sb.Table(dw), ids, dout)
    assert dw[at, 17] == float("inf")
    dw[at, 17] = want[at, 17]
    assert torch.equal(dw, want)


def test_same_bits_again(require_gpu):
    ids = make_ids("ranks", 20000, 5000, 4)
    dout = torch.randn(20000, 72, device="cuda")
    one, two = torch.empty(5000, 72, device="cuda"), torch.empty(5000, 72, device="cuda")
    sb.sb_embed_grad(sb.Table(one), ids, dout)
    sb.sb_embed_grad(sb.Table(two), ids, dout)
    assert torch.equal(one, two)


def test_no_rows(require_gpu):
    dw = torch.ones(100, 24, device="cuda")
    ids, none = torch.empty(0, dtype=torch.int32, device="cuda"), torch.empty(0, 24, device="cuda")
    sb.sb_embed(sb.Table(dw), ids, none)
    sb.sb_embed_grad(sb.Table(dw), ids, none, accumulate=True)
    assert bool((dw == 1).all())
    sb.sb_embed_grad(sb.Table(dw), ids, none)
    assert not dw.any()


def test_far_rows_of_a_large_table(require_gpu):
    """Offsets past 32 bits: a table of 5 GiB."""
    V, H = 262144, 10240
    w = torch.empty(V, H, dtype=H16, device="cuda")
    w.copy_(torch.arange(V, device="cuda").remainder(251)[:, None])
    ids = torch.tensor([V - 1, 0, V - 2, 131072, V // 2 + 1, V - 1], dtype=torch.int32, device="cuda")
    out = torch.empty(6, H, device="cuda")
    sb.sb_embed(sb.Table(w, [0, 200000, V]), ids, out)
    assert torch.equal(out, (ids.long() % 251).float()[:, None].expand(6, H))
    sb.sb_embed_grad(sb.Table(w, [0, 200000, V]), ids, torch.ones(6, H, device="cuda"))
    assert torch.equal(w[:, 0].float().nonzero()[:, 0], ids.long().unique())
    assert bool((w[V - 1] == 2).all()) and bool((w[V - 2] == 1).all()) and float(w.float().sum()) == 6 * H


def test_rows_far_apart(require_gpu):
    """Rows of out and dout whose offsets pass 32 bits."""
    w = torch.randn(50, 264, device="cuda").to(H16)
    ids = torch.tensor([7, 49, 7], dtype=torch.int32, device="cuda")
    ld = 1 << 30
    far = torch.empty(2 * ld + 264, dtype=H16, device="cuda").as_strided((3, 264), (ld, 1))
    sb.sb_embed(sb.Table(w), ids, far)
    assert torch.equal(far, w[ids.long()])
    dw = torch.empty(50, 264, device="cuda")
    sb.sb_embed_grad(sb.Table(dw), ids, far)
    want = torch.zeros(50, 264, device="cuda")
    want[7], want[49] = 2 * w[7].float(), w[49].float()
    assert torch.equal(dw, want)


def test_refusals_of_the_binding(require_gpu):
    w, ids = torch.zeros(16, 8, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    t, out = sb.Table(w), torch.empty(4, 8, device="cuda")
    for call, error in (
            (lambda: sb.sb_embed(sb.Table(w.half()), ids, out), TypeError),
            (lambda: sb.sb_embed(sb.Table(w.t()), ids, out), ValueError),
            (lambda: sb.sb_embed(sb.Table(w, [0, 17]), ids, out), ValueError),
            (lambda: sb.sb_embed(sb.Table([w, w.bfloat16()]), ids, out), TypeError),
            (lambda: sb.sb_embed(sb.Table([w, torch.zeros(3, 16, device="cuda")[:, :8]]), ids, out), ValueError),
            (lambda: sb.sb_embed(t, ids.long(), out), TypeError),
            (lambda: sb.sb_embed(t, ids[::2], out), ValueError),
            (lambda: sb.sb_embed(t, ids, out[:3]), ValueError),
            (lambda: sb.sb_embed(t, ids, out.half()), TypeError),
            (lambda: sb.sb_embed(t, ids.cpu(), out), ValueError),
            (lambda: sb.sb_embed_grad(t, ids, out[:, :4]), ValueError),
            (lambda: sb.sb_embed_grad(t, ids, out, ws=torch.empty(16, dtype=torch.uint8, device="cuda")), sb.SbError)):
        with pytest.raises(error):
            call()
