"""GPU tests of the 8-bit head.  Integer sums are exact and the three fp32
roundings of a logit are defined, so everything is compared for equality: the
sums in 64 bits, rounded to fp32, times the two scales in fp32."""
import pytest
import torch

from logit_source_projection_amd import inputs, sb

pytestmark = pytest.mark.gpu


def up(n, m):
    return (n + m - 1) // m * m


def padded(rows, cols, dtype, fill, pad):
    """[rows, cols] inside a wider buffer whose other elements hold `fill`."""
    unit = 16 if dtype == torch.int8 else 8
    buf = torch.full((rows, up(cols, unit) + pad), fill, device="cuda", dtype=dtype)
    return buf, buf[:, :cols]


class Case:
    def __init__(self, B, H, V, lanes, seed=0, separate=False, pad=16, extreme=False):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.V, self.lanes = B, H, V, list(lanes)
        lo, hi = (-128, -126) if extreme else (-128, 128)

        def codes(n):
            return torch.randint(lo, hi, (n, H), device="cuda", generator=g, dtype=torch.int8)

        # the padding holds 113: a product with it would show
        _, self.x = padded(B, H, torch.int8, 113, pad)
        self.x.copy_(codes(B))
        self.xs = torch.rand(B, device="cuda", generator=g) + 0.01
        _, self.w = padded(V, H, torch.int8, 113, pad)
        self.w.copy_(codes(V))
        self.ws = torch.rand(V, device="cuda", generator=g) + 0.01
        w, ws = self.w, self.ws
        if separate:
            w, ws = [], []
            for a, b in zip(lanes, lanes[1:]):
                t = padded(b - a, H, torch.int8, 113, pad)[1]
                t.copy_(self.w[a:b])
                w.append(t)
                ws.append(self.ws[a:b].clone())
        self.head = sb.Int8Head(self.x, self.xs, w, ws, self.lanes)

    def reference(self):
        sums = self.x.double() @ self.w.double().t()
        return (sums.float() * self.xs[:, None]) * self.ws

    def logits(self, dtype=torch.float32, **kw):
        buf = torch.full((self.B, up(self.V, 8) + 8), 7.0, device="cuda", dtype=dtype)
        sb.sb_int8_logits(self.head, buf[:, :self.V], **kw)
        torch.cuda.synchronize()
        assert bool((buf[:, self.V:] == 7).all()), "padding of the output"
        return buf[:, :self.V]

    def tokens(self, **kw):
        ids = torch.full((self.B,), -1, device="cuda", dtype=torch.int32)
        sb.sb_int8_project_tokens(self.head, ids, **kw)
        return ids


SHAPES = [
    # B, H, V, lanes
    (1, 1, 1, (0, 1)),
    (1, 16, 64, (0, 64)),
    (2, 63, 65, (0, 65)),
    (3, 64, 300, (0, 100, 300)),
    (7, 65, 1001, (0, 7, 64, 1001)),
    (16, 2000, 500, (0, 500)),
    (17, 129, 130, (0, 130)),
    (32, 4100, 257, (0, 128, 257)),
    (33, 1024, 1030, (0, 1030)),
    (48, 5120, 320, (0, 320)),
    (64, 300, 40000, (0, 13000, 40000)),
    (5, 192, 70001, (0, 70001)),
    (65, 1, 3, (0, 3)),
    (100, 127, 255, (0, 255)),
    (255, 128, 256, (0, 256)),
    (257, 1000, 513, (0, 250, 513)),
    (300, 259, 2500, (0, 256, 512, 2500)),
    (800, 640, 1100, (0, 300, 1100)),
]


@pytest.mark.parametrize("B,H,V,lanes", SHAPES)
def test_product_and_tokens(require_gpu, B, H, V, lanes):
    print(f"int8 B={B} H={H} V={V} lanes={lanes}", flush=True)
    c = Case(B, H, V, lanes, seed=B + H)
    z = c.reference()
    assert torch.equal(c.logits(), z)
    assert torch.equal(c.logits(torch.bfloat16), z.to(torch.bfloat16))
    assert torch.equal(c.tokens(), z.argmax(1).to(torch.int32))


@pytest.mark.parametrize("B", [32, 33, 64])
@pytest.mark.parametrize("V", [16383, 16384])
def test_both_sides_of_the_few_row_rule(require_gpu, B, V):
    print(f"int8 B={B} V={V}", flush=True)
    c = Case(B, 300, V, (0, 5001, V), seed=B)
    z = c.reference()
    assert torch.equal(c.logits(), z)
    assert torch.equal(c.logits(torch.bfloat16), z.to(torch.bfloat16))
    assert torch.equal(c.tokens(), z.argmax(1).to(torch.int32))


@pytest.mark.parametrize("B,H,V,lanes", [(65, 17408, 5120, (0, 5120)), (100, 3601, 333, (0, 100, 333)),
                                         (129, 5000, 1003, (0, 130, 600, 1003)),
                                         (300, 4111, 2100, (0, 2100)), (1000, 3600, 515, (0, 3, 515))])
def test_tiles_split_along_k(require_gpu, B, H, V, lanes):
    print(f"int8 split tiles B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=H)
    z = c.reference()
    n = max(sb.sb_int8_workspace_bytes(c.head, s) for s in (sb.SB_SURF_TOKENS, sb.SB_SURF_FULL_LOGITS))
    assert n >= 2 * 4 * B * V                       # two slices' sums at least
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):
        assert torch.equal(c.logits(ws=ws), z)
        assert torch.equal(c.tokens(ws=ws), z.argmax(1).to(torch.int32))
    assert torch.equal(c.logits(torch.bfloat16), z.to(torch.bfloat16))


@pytest.mark.parametrize("B,H,V,k", [(9, 100, 1003, 5), (70, 264, 2003, 3), (4, 48, 1601, 64),
                                     (90, 48, 1601, 64)])
def test_lanes_in_their_own_allocations(require_gpu, B, H, V, k):
    print(f"int8 lanes B={B} H={H} V={V} k={k}", flush=True)
    c = Case(B, H, V, inputs.equal_lanes(V, k), seed=k, separate=True)
    z = c.reference()
    assert torch.equal(c.logits(), z)
    assert torch.equal(c.logits(torch.bfloat16), z.to(torch.bfloat16))
    assert torch.equal(c.tokens(), z.argmax(1).to(torch.int32))


@pytest.mark.parametrize("B", [3, 80])
def test_longest_sums_do_not_overflow(require_gpu, B):
    """-128 * -128 over the largest H: 2,147,467,264, just below 2^31."""
    print(f"longest sums B={B}", flush=True)
    c = Case(B, 131071, 70, (0, 70), seed=1, extreme=True)
    c.x[0], c.w[0] = -128, -128
    c.x[1], c.w[1] = 127, -128
    z = c.reference()
    assert (c.x[0].double() @ c.w[0].double()).item() == 16384.0 * 131071
    assert torch.equal(c.logits(), z)


@pytest.mark.parametrize("B,V", [(4, 3000), (4, 50000), (100, 3000)])
def test_ties_go_to_the_lowest_index(require_gpu, B, V):
    c = Case(B, 200, V, (0, 1000, V), seed=3)
    top = torch.full((200,), 127, dtype=torch.int8, device="cuda")
    c.x[:, :] = top
    c.ws.fill_(0.5)
    for cols in ([V - 1], [2999, 1001], [1001, 999], [999, 70, 64], [70, 3, 2]):
        c.w[cols] = top
        assert bool((c.tokens() == min(cols)).all()), cols
    c.w.zero_()
    assert bool((c.tokens() == 0).all())


@pytest.mark.parametrize("B", [3, 70])
@pytest.mark.parametrize("V", [400, 40000])
def test_scales_that_are_not_finite(require_gpu, B, V):
    c = Case(B, 64, V, (0, 200, V), seed=4)
    c.x[:, 0], c.w[:, 0] = 1, 1
    c.x[:, 1:], c.w[:, 1:] = 0, 0
    c.xs.fill_(1.0), c.ws.fill_(1.0)
    c.ws[300], c.ws[250] = float("nan"), float("inf")
    assert bool((c.tokens() == 300).all())           # NaN ranks above infinity
    c.ws[300] = 1
    assert bool((c.tokens() == 250).all())
    c.xs[1] = float("nan")
    ids = c.tokens()
    assert ids[1].item() == 0 and ids[0].item() == 250 and ids[2].item() == 250
    assert torch.equal(c.logits().isnan(), c.reference().isnan())


def quantised(v):
    """Codes and scales of the rows of v (bf16) by their definition."""
    f = v.float()
    scale = (v.double().abs().amax(1) / 127).float()
    q = torch.round(f / scale[:, None]).clamp(-127, 127)
    bad = (scale == 0) | ~scale.isfinite()
    return torch.where(bad[:, None], 0.0, q).to(torch.int8), scale


@pytest.mark.parametrize("B,H", [(1, 1), (3, 7), (5, 8), (2, 100), (16, 5120), (9, 2047), (4, 16384),
                                 (3, 16391), (2, 40009), (700, 256)])
def test_row_codes(require_gpu, B, H):
    print(f"rows B={B} H={H}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(H)
    buf, x = padded(B, H, torch.bfloat16, float("nan"), 8)
    x.copy_(torch.randn(B, H, device="cuda", generator=g) *
            torch.logspace(-30, 30, B, device="cuda")[:, None])
    qb, q = padded(B, H, torch.int8, 99, 16)
    scale = torch.full((B,), float("nan"), device="cuda")
    sb.sb_int8_quantize_rows(x, q, scale)
    rq, rs = quantised(x)
    assert torch.equal(scale, rs) and torch.equal(q, rq)
    assert bool((qb[:, H:] == 99).all())
    assert int(q.int().abs().amax(1).min()) == 127


def test_rows_of_zeros_and_of_non_finite_values(require_gpu):
    x = torch.randn(6, 520, device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[1, 519], x[2, 3], x[3, 7] = float("nan"), float("inf"), -float("inf")
    x[4] = 0
    x[4, 100] = 9.2e-41                          # the smallest bf16
    x[5] = 3.38e38
    q = torch.full((6, 528), 99, dtype=torch.int8, device="cuda")[:, :520]
    scale = torch.empty(6, device="cuda")
    sb.sb_int8_quantize_rows(x, q, scale)
    rq, rs = quantised(x)
    assert torch.equal(q, rq) and torch.equal(scale.isnan(), rs.isnan())
    assert torch.equal(scale.nan_to_num(0), rs.nan_to_num(0))
    assert scale[0].item() == 0 and bool((q[:4] == 0).all()) and q[4, 100].item() == 127
    # the rows' logits: 0, NaN, NaN, NaN
    w = torch.ones(40, 528, dtype=torch.int8, device="cuda")[:, :520]
    head = sb.Int8Head(q, scale, w, torch.ones(40, device="cuda"), [0, 40])
    out = sb.sb_int8_logits(head, torch.empty(6, 40, device="cuda"))
    assert bool((out[0] == 0).all()) and bool(out[1:4].isnan().all()) and bool(out[4].isfinite().all())
    # 520 times 3.38e38 is 1.76e41, past fp32's largest value of 3.4e38
    assert bool((out[5] == float("inf")).all())


@pytest.mark.parametrize("H,V,lanes", [(1, 1, (0, 1)), (64, 64, (0, 64)), (65, 130, (0, 130)),
                                       (300, 1003, (0, 400, 1003)), (1000, 72, (0, 8, 72)),
                                       (2050, 333, (0, 333))])
@pytest.mark.parametrize("separate", [False, True])
def test_head_codes(require_gpu, H, V, lanes, separate):
    print(f"head H={H} V={V} separate={separate}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(V)
    values = (torch.randn(H, V, device="cuda", generator=g) *
              torch.logspace(-20, 20, V, device="cuda")).to(torch.bfloat16)
    if V > 20:
        values[:, 3] = 0
        values[H - 1, 5], values[0, 7] = float("nan"), float("inf")
    if not separate and any(o % 8 for o in lanes[:-1]):
        pytest.skip("lanes of one allocation start at multiples of 8")
    if separate:
        widest = max(b - a for a, b in zip(lanes, lanes[1:]))
        w = [padded(H, widest, torch.bfloat16, float("nan"), 8)[1][:, :b - a]
             for a, b in zip(lanes, lanes[1:])]
        for t, a, b in zip(w, lanes, lanes[1:]):
            t.copy_(values[:, a:b])
        bufs = [padded(b - a, H, torch.int8, 99, 16) for a, b in zip(lanes, lanes[1:])]
        q, scale = [t for _, t in bufs], [torch.empty(b - a, device="cuda") for a, b in zip(lanes, lanes[1:])]
    else:
        w = padded(H, V, torch.bfloat16, float("nan"), 8)[1]
        w.copy_(values)
        bufs = [padded(V, H, torch.int8, 99, 16)]
        q, scale = bufs[0][1], torch.empty(V, device="cuda")
    x = torch.zeros(1, up(H, 8), device="cuda", dtype=torch.bfloat16)[:, :H]
    sb.sb_int8_quantize_head(sb.Head(x, w, lanes), q, scale)
    rq, rs = quantised(values.t())
    gq, gs = (torch.cat(q), torch.cat(scale)) if separate else (q, scale)
    assert torch.equal(gs.isnan(), rs.isnan()) and torch.equal(gs.nan_to_num(0), rs.nan_to_num(0))
    assert torch.equal(gq, rq)
    for buf, _ in bufs:
        assert bool((buf[:, H:] == 99).all())


def test_empty_sizes(require_gpu):
    c = Case(0, 32, 100, (0, 100))
    assert c.tokens().numel() == 0 and c.logits().numel() == 0
    for B in (2, 70):                            # no hidden values: every logit is 0
        x = torch.empty(B, 0, dtype=torch.int8, device="cuda")
        w = torch.empty(100, 0, dtype=torch.int8, device="cuda")
        head = sb.Int8Head(x, torch.ones(B, device="cuda"), w, torch.ones(100, device="cuda"), [0, 100],
                           ldx=0, ldw=0)
        out = torch.full((B, 100), 7.0, device="cuda")
        assert bool((sb.sb_int8_logits(head, out) == 0).all())
        ids = torch.full((B,), -1, dtype=torch.int32, device="cuda")
        assert bool((sb.sb_int8_project_tokens(head, ids) == 0).all())


@pytest.mark.parametrize("B,H,V", [(6, 2048, 900), (40, 200, 50000), (150, 200, 900)])
def test_streams_graphs_and_garbage_workspaces(require_gpu, B, H, V):
    print(f"int8 graph B={B}", flush=True)
    c = Case(B, H, V, (0, V), seed=B)
    z = c.reference()
    want = z.argmax(1).to(torch.int32)
    n = max(16, *(sb.sb_int8_workspace_bytes(c.head, s) for s in
                  (sb.SB_SURF_TOKENS, sb.SB_SURF_FULL_LOGITS)))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.tokens(ws=ws), want) and torch.equal(c.logits(ws=ws), z)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids = torch.empty(B, dtype=torch.int32, device="cuda")
    sb.sb_int8_project_tokens(c.head, ids, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(ids, want)
    # quantise and project, captured once, replayed on new rows
    x = torch.zeros(B, up(H, 8), device="cuda", dtype=torch.bfloat16)[:, :H]
    out = torch.empty(B, up(V, 4), device="cuda")[:, :V]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sb.sb_int8_quantize_rows(x, c.x, c.xs)
        sb.sb_int8_project_tokens(c.head, ids, ws=ws)
        sb.sb_int8_logits(c.head, out, ws=ws)
    for turn in range(4):
        x.copy_(torch.randn(B, H, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        q, scale = quantised(x)
        assert torch.equal(c.x, q) and torch.equal(c.xs, scale)
        z = c.reference()
        assert torch.equal(out, z) and torch.equal(ids, z.argmax(1).to(torch.int32)), turn
        assert torch.equal(c.tokens(ws=ws), ids)


def test_refusals_leave_outputs_alone(require_gpu):
    c = Case(4, 64, 100, (0, 100))
    ids = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="ids must be torch.int32"):
        sb.sb_int8_project_tokens(c.head, ids.long())
    with pytest.raises(TypeError, match="out must be torch.float32"):
        sb.sb_int8_logits(c.head, torch.empty(4, 100, device="cuda", dtype=torch.float16))
    with pytest.raises(ValueError, match="out must be a"):
        sb.sb_int8_logits(c.head, torch.empty(4, 99, device="cuda"))
    with pytest.raises(TypeError, match="q must be torch.int8"):
        sb.sb_int8_quantize_rows(torch.zeros(4, 64, device="cuda", dtype=torch.bfloat16),
                                 torch.zeros(4, 64, device="cuda"), c.xs)
    with pytest.raises(sb.SbError) as e:
        sb.sb_int8_project_tokens(c.head, ids, ws=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == sb.SB_ERR_WORKSPACE
    torch.cuda.synchronize()
    assert bool((ids == -7).all())


def test_a_head_is_trained_and_then_served(require_gpu):
    """Loss, gradient and one step on the bf16 head, then the stepped head in
    8 bits: each call on what the one before it made."""
    B, H, V, lanes = 96, 256, 3000, [0, 1504, 3000]
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(B, H, device="cuda", generator=g).to(torch.bfloat16)
    w = (0.05 * torch.randn(H, V, device="cuda", generator=g)).to(torch.bfloat16)
    t = torch.randint(0, V, (B,), device="cuda", generator=g, dtype=torch.int32)
    t[5] = -100
    head = sb.Head(x, w, lanes)
    loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    sb.sb_cross_entropy(head, t, loss, lse)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    sb.sb_cross_entropy_grad(head, t, lse, torch.full((B,), 1.0 / 95, device="cuda"), dx, dw)
    from tests.loss_common import check_grad, check_loss
    check_loss(loss, lse, x, w, t)
    check_grad(dx, dw, x, w, t, torch.full((B,), 1.0 / 95, device="cuda"), lse)
    w -= 0.5 * dw                              # the descriptor sees the stepped weight
    q, qs = torch.empty(V, H, dtype=torch.int8, device="cuda"), torch.empty(V, device="cuda")
    sb.sb_int8_quantize_head(head, q, qs)
    rq, rs = quantised(w.t())
    assert torch.equal(q, rq) and torch.equal(qs, rs)
    xq, xs = torch.empty(B, H, dtype=torch.int8, device="cuda"), torch.empty(B, device="cuda")
    sb.sb_int8_quantize_rows(x, xq, xs)
    head8 = sb.Int8Head(xq, xs, q, qs, lanes)
    ids = sb.sb_int8_project_tokens(head8, torch.empty(B, dtype=torch.int32, device="cuda"))
    z = sb.sb_int8_logits(head8, torch.empty(B, V, device="cuda"))
    assert torch.equal(ids, z.argmax(1).to(torch.int32))
    # a code is off by half a step at most: with steps s, t of a row and a
    # column, each product by (|x| t + |w| s) / 2 + s t / 4
    f = x.double() @ w.double()
    bound = (x.double().abs().sum(1)[:, None] * qs.double() + xs.double()[:, None] *
             w.double().abs().sum(0)) / 2 + H * xs.double()[:, None] * qs.double() / 4
    assert bool(((z.double() - f).abs() <= bound * (1 + 2.0 ** -20)).all())
