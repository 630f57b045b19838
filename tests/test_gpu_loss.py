"""GPU tests of the loss and its gradient against their definition in 64 bits:
odd sizes around the 256-row and 256-column tiles and the 64-deep K stages,
ignored rows, strided operands whose padding must not be read or written,
streams, graphs and shared workspaces."""
import pytest
import torch

from logit_source_projection_amd import inputs, sb
from tests.loss_common import HALF_FP32, check_grad, check_loss, reference, reference_grad

pytestmark = pytest.mark.gpu


class Case:
    """Inputs with NaN in every padding element and outputs in padded buffers."""

    def __init__(self, B, H, V, lanes, seed=0, ignored=0.15, separate=False, pad=8, scale=0.1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H, self.V, self.lanes = B, H, V, list(lanes)

        def padded(rows, cols, values):
            buf = torch.full((rows, (cols + 7) // 8 * 8 + pad), float("nan"), device="cuda",
                             dtype=torch.bfloat16)
            buf[:, :cols] = values
            return buf[:, :cols]

        self.w = (scale * torch.randn(H, V, device="cuda", generator=g)).to(torch.bfloat16)
        x = torch.randn(B, H, device="cuda", generator=g)
        self.targets = torch.randint(0, V, (B,), device="cuda", generator=g, dtype=torch.int32)
        self.targets[torch.rand(B, device="cuda", generator=g) < ignored] = -100
        self.dloss = torch.randn(B, device="cuda", generator=g)
        self.x = padded(B, H, x)
        if separate:
            widest = max(b - a for a, b in zip(lanes, lanes[1:]))
            self.wt = [padded(H, widest, 0)[:, :b - a] for a, b in zip(lanes, lanes[1:])]
            for t, a, b in zip(self.wt, lanes, lanes[1:]):
                t.copy_(self.w[:, a:b])
        else:
            self.wt = padded(H, V, self.w)
        self.head = sb.Head(self.x, self.wt, self.lanes)

    def outputs(self, pad=16):
        dx = torch.full((self.B, (self.H + 7) // 8 * 8 + pad), 7.0, device="cuda", dtype=torch.bfloat16)
        if isinstance(self.wt, list):
            widest = max(t.shape[1] for t in self.wt)
            dw = [torch.full((self.H, (widest + 7) // 8 * 8 + pad), 7.0, device="cuda",
                             dtype=torch.bfloat16) for _ in self.wt]
        else:
            dw = torch.full((self.H, (self.V + 7) // 8 * 8 + pad), 7.0, device="cuda",
                            dtype=torch.bfloat16)
        return dx, dw

    def loss(self, **kw):
        loss = torch.full((self.B,), float("nan"), device="cuda")
        lse = torch.full((self.B,), float("nan"), device="cuda")
        sb.sb_cross_entropy(self.head, self.targets, loss, lse, **kw)
        return loss, lse

    def grad(self, lse, want=("dx", "dw"), **kw):
        """(dx, dw) without padding, after a check that no padding was written."""
        dx, dw = self.outputs()
        widths = [b - a for a, b in zip(self.lanes, self.lanes[1:])]
        dwa = [t[:, :n] for t, n in zip(dw, widths)] if isinstance(dw, list) else dw[:, :self.V]
        sb.sb_cross_entropy_grad(self.head, self.targets, lse, self.dloss,
                                 dx[:, :self.H] if "dx" in want else None,
                                 dwa if "dw" in want else None, **kw)
        torch.cuda.synchronize()
        assert bool((dx[:, self.H:] == 7).all()), "padding of dx"
        for t, n in zip(dw, widths) if isinstance(dw, list) else ((dw, self.V),):
            assert bool((t[:, n:] == 7).all()), "padding of dw"
        if "dx" not in want:
            assert bool((dx == 7).all())
        if "dw" not in want:
            assert all(bool((t == 7).all()) for t in (dw if isinstance(dw, list) else [dw]))
        dwr = torch.cat(dwa, 1) if isinstance(dwa, list) else dwa
        return (dx[:, :self.H] if "dx" in want else None), (dwr if "dw" in want else None)


SHAPES = [
    # B, H, V, lanes
    (1, 1, 1, (0, 1)),
    (1, 8, 300, (0, 300)),
    (2, 64, 256, (0, 256)),
    (5, 65, 257, (0, 257)),
    (3, 300, 4096, (0, 2048, 4096)),
    (16, 512, 1000, (0, 8, 16, 1000)),
    (17, 72, 3001, (0, 1000, 3001)),
    (33, 1000, 2600, (0, 2600)),
    (64, 256, 5000, (0, 2504, 5000)),
    (65, 129, 777, (0, 777)),
    (128, 640, 1500, (0, 504, 1008, 1500)),
    (129, 31, 2049, (0, 2049)),
    (255, 200, 900, (0, 256, 512, 900)),
    (256, 256, 512, (0, 512)),
    (257, 1111, 1300, (0, 1300)),
    (600, 520, 2000, (0, 640, 1280, 2000)),
    (1030, 96, 700, (0, 700)),
]


@pytest.mark.parametrize("B,H,V,lanes", SHAPES)
def test_loss_and_gradient(require_gpu, B, H, V, lanes):
    print(f"loss B={B} H={H} V={V} lanes={lanes}", flush=True)
    c = Case(B, H, V, lanes, seed=B + H)
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B,H,V,lanes", [(65, 2049, 333, (0, 104, 333)), (100, 4100, 1003, (0, 136, 600, 1003)),
                                         (300, 2100, 2100, (0, 2100)), (1000, 2056, 515, (0, 8, 515))])
def test_tiles_split_along_k(require_gpu, B, H, V, lanes):
    """Few tiles and a long H: slices' logits are stored and added up."""
    print(f"split tiles B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, lanes, seed=H)
    n = sb.sb_cross_entropy_workspace_bytes(c.head, True)
    assert sb.sb_cross_entropy_workspace_bytes(c.head, False) >= 2 * 4 * B * V  # two slices at least
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    c.targets[0], c.targets[B - 1] = V - 1, -1
    loss, lse = c.loss(ws=ws)
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse, ws=ws)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)
    # ignored rows hold anything; a target past the vocabulary is NaN
    c.x[B - 1] = float("nan")
    c.targets[1] = V
    loss, lse = c.loss(ws=ws)
    assert loss[B - 1].item() == 0 and bool(loss[1].isnan()) and bool(loss[:1].isfinite().all())
    dx2, _ = c.grad(lse, ws=ws, want=("dx",))
    rest = torch.arange(B, device="cuda") != 1
    assert bool(dx2[1].isnan().all()) and torch.equal(dx2[rest], dx[rest])


@pytest.mark.parametrize("B,H,V,k", [(4, 100, 1003, 5), (70, 264, 2003, 3), (300, 64, 1601, 64)])
def test_lanes_in_their_own_allocations(require_gpu, B, H, V, k):
    """Lane widths that are no multiple of 8 (or of anything)."""
    print(f"separate lanes B={B} H={H} V={V} k={k}", flush=True)
    c = Case(B, H, V, inputs.equal_lanes(V, k), seed=k, separate=True)
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B", [3, 40, 200])
def test_one_gradient_alone(require_gpu, B):
    print(f"one gradient B={B}", flush=True)
    c = Case(B, 320, 1500, (0, 760, 1500), seed=B)
    _, lse = c.loss()
    dx, dw = c.grad(lse)
    dx1, none = c.grad(lse, want=("dx",))
    assert none is None and torch.equal(dx1, dx)
    none, dw1 = c.grad(lse, want=("dw",))
    assert none is None and torch.equal(dw1, dw)


def test_pieces_of_the_vocabulary(require_gpu):
    """A batch whose dz does not fit one piece: dx is summed over the pieces."""
    B, H, V = 4100, 72, 40000
    print(f"pieces B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, (0, 16000, 40000), seed=5)
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B", [4, 90, 300])
def test_ignored_rows_hold_anything(require_gpu, B):
    """NaN and infinities in ignored rows reach nothing but their own lse."""
    print(f"ignored rows B={B}", flush=True)
    c = Case(B, 136, 900, (0, 900), seed=B)
    c.targets[0], c.targets[1], c.targets[B - 1] = 3, -1, -(1 << 31)
    ig = c.targets < 0
    clean = c.x.clone()
    _, lse = c.loss()
    ref = c.grad(lse)
    c.x[ig] = torch.tensor([float("nan"), float("inf"), -float("inf"), 3e38],
                           device="cuda").repeat(34).to(torch.bfloat16)
    loss, lse2 = c.loss()
    assert bool((loss[ig] == 0).all()) and torch.equal(lse2[~ig], lse[~ig])
    dx, dw = c.grad(lse2)
    assert bool((dx[ig] == 0).all())
    assert torch.equal(dx, ref[0]) and torch.equal(dw, ref[1])
    c.targets.fill_(-100)
    c.x.copy_(clean)
    loss, lse = c.loss()
    assert bool((loss == 0).all())
    dx, dw = c.grad(lse)
    assert bool((dx == 0).all()) and bool((dw == 0).all())


@pytest.mark.parametrize("B", [4, 80])
def test_target_past_the_vocabulary(require_gpu, B):
    c = Case(B, 64, 500, (0, 200, 500), seed=2, ignored=0)
    c.targets[1], c.targets[2] = 500, (1 << 31) - 1
    loss, lse = c.loss()
    bad = torch.zeros(B, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    assert bool(loss[bad].isnan().all()) and bool(loss[~bad].isfinite().all())
    assert bool(lse.isfinite().all())
    dx, dw = c.grad(lse)
    assert bool(dx[bad].isnan().all()) and bool(dx[~bad].isfinite().all())
    assert bool(dw.isnan().all())


@pytest.mark.parametrize("B", [3, 100])
def test_targets_at_lane_and_block_edges(require_gpu, B):
    V, lanes = 1300, (0, 256, 520, 1300)
    c = Case(B, 48, V, lanes, seed=8, ignored=0)
    edges = [0, 255, 256, 519, 520, 775, 776, 1031, 1032, 1299]
    for i in range(0, len(edges), B):
        part = edges[i:i + B]
        c.targets[:len(part)] = torch.tensor(part, dtype=torch.int32, device="cuda")
        loss, lse = c.loss()
        check_loss(loss, lse, c.x, c.w, c.targets)
        dx, dw = c.grad(lse)
        check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


@pytest.mark.parametrize("B", [2, 70])
def test_masked_and_extreme_logits(require_gpu, B):
    """Columns at -inf and at bf16's lowest value have probability 0; a NaN or
    +inf logit makes its row's lse NaN and no other's."""
    H, V = 8, 600
    c = Case(B, H, V, (0, V), seed=4, ignored=0)
    c.x.fill_(0)
    c.x[:, 0] = 1
    w = torch.zeros(H, V, device="cuda")
    w[0] = torch.linspace(-3, 3, V, device="cuda")
    w[0, 100:500] = float("-inf")
    w[0, 0] = -3.0e38
    w[1:, 100:500] = 0
    c.w = w.to(torch.bfloat16)
    c.wt.copy_(c.w)
    # 0 * finite only: -inf stands where x is 1
    c.targets.fill_(50)
    loss, lse = c.loss()
    z = c.w[0].double().expand(B, V)
    ref = torch.logsumexp(z, 1)
    assert bool(((lse.double() - ref).abs() <= 64 * HALF_FP32 * 8).all())
    c.targets[1] = 100                     # an impossible target: infinite loss
    loss, lse = c.loss()
    assert loss[1].item() == float("inf") and bool(loss[0].isfinite())
    c.x[1, 0] = float("nan")
    loss, lse = c.loss()
    assert bool(lse[1].isnan()) and bool(lse[0].isfinite()) and bool(loss[1].isnan())
    c.x[1, 0] = -1                         # the masked columns become +inf
    _, lse = c.loss()
    assert bool(lse[1].isnan()) and bool(lse[0].isfinite())
    # large logits: no overflow in the exponentials
    c.x.zero_()
    c.x[:, 0] = 1
    c.wt.zero_()
    c.wt[0] = torch.linspace(-1e4, 1e4, V, device="cuda").to(torch.bfloat16)
    c.w = c.wt.clone()
    c.targets.fill_(V - 1)
    loss, lse = c.loss()
    check_loss(loss, lse, c.x, c.w, c.targets)
    dx, dw = c.grad(lse)
    check_grad(dx, dw, c.x, c.w, c.targets, c.dloss, lse)


def test_empty_sizes(require_gpu):
    # no rows: the loss does nothing, dw is zeroed
    c = Case(0, 40, 300, (0, 300))
    loss, lse = c.loss()
    assert loss.numel() == 0
    dx, dw = c.grad(lse)
    assert bool((dw == 0).all())
    # no hidden values: every logit is 0
    x = torch.empty(3, 0, device="cuda", dtype=torch.bfloat16)
    w = torch.empty(0, 304, device="cuda", dtype=torch.bfloat16)
    head = sb.Head(x, w, [0, 304], ldx=0, ldw=304)
    t = torch.tensor([0, -1, 303], dtype=torch.int32, device="cuda")
    loss, lse = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    sb.sb_cross_entropy(head, t, loss, lse)
    log = torch.log(torch.tensor(304.0))
    assert torch.allclose(lse.cpu(), log.expand(3), rtol=4 * HALF_FP32, atol=0)
    assert loss[1].item() == 0 and torch.equal(loss[[0, 2]], lse[[0, 2]])


def test_gradient_against_differences(require_gpu):
    """Central differences of the GPU's own losses along random directions.  x
    and w sit on a grid of 1/8, so that a step of 2^-5 is exact in bf16; the
    third-order term is at most eps^2 / 6 times the cube of the logits' range."""
    B, H, V, eps = 6, 40, 500, 2.0 ** -5
    g = torch.Generator(device="cuda").manual_seed(1)
    c = Case(B, H, V, (0, V), seed=1, ignored=0)
    c.dloss.fill_(1.0)

    def grid(*shape, top):
        return torch.randint(-top, top + 1, shape, device="cuda", generator=g) / 8.0

    x0, w0 = grid(B, H, top=7), grid(H, V, top=3)
    c.x.copy_(x0), c.wt.copy_(w0)
    _, lse = c.loss()
    dx, dw = c.grad(lse)
    for trial in range(4):
        sx = torch.randint(0, 2, (B, H), device="cuda", generator=g) * 2.0 - 1
        sw = (torch.rand(H, V, device="cuda", generator=g) < 0.1) * 1.0
        for which, d, grad in (("x", sx, dx), ("w", sw, dw)):
            total = []
            for sign in (1, -1):
                c.x.copy_(x0 + (sign * eps * d if which == "x" else 0))
                c.wt.copy_(w0 + (sign * eps * d if which == "w" else 0))
                loss, _ = c.loss()
                total.append(loss.double().sum())
            slope = ((total[0] - total[1]) / (2 * eps)).item()
            said = (grad.double() * d.double()).sum().item()
            dirz = (d.double() @ w0.double()) if which == "x" else (x0.double() @ d.double())
            span = (dirz.amax(1) - dirz.amin(1))
            third = (span ** 3).sum().item() * eps ** 2 / 6
            # each loss to 1e-5 (fp32 sums of 40 products of this size); the
            # gradient's two roundings, as independent errors of its elements
            noise = 2 * B * 1e-5 / (2 * eps)
            spread = 4 * 2.0 ** -8 * (grad.double() * d.double()).norm().item()
            assert abs(slope - said) <= third + noise + spread, (which, slope, said, third, noise, spread)
    c.x.copy_(x0), c.wt.copy_(w0)


def _all(c, **kw):
    loss, lse = c.loss(**kw)
    return (loss, lse) + tuple(c.grad(lse, **kw))


@pytest.mark.parametrize("B,H,V", [(3, 256, 3000), (50, 130, 1000), (200, 300, 2000)])
def test_repeats_streams_and_garbage_workspaces(require_gpu, B, H, V):
    print(f"repeat B={B} H={H} V={V}", flush=True)
    c = Case(B, H, V, (0, 504, V), seed=B)
    first = _all(c)
    n = max(sb.sb_cross_entropy_workspace_bytes(c.head, g) for g in (False, True))
    for fill in (0xFF, 0x5A):
        ws = torch.full((n,), fill, dtype=torch.uint8, device="cuda")
        for a, b in zip(first, _all(c, ws=ws)):
            assert torch.equal(a, b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _all(c)
    explicit = _all(c, stream=s)
    torch.cuda.synchronize()
    for a, b, d in zip(first, other, explicit):
        assert torch.equal(a, b) and torch.equal(a, d)


@pytest.mark.parametrize("B", [5, 150])
def test_two_graphs_share_a_workspace(require_gpu, B):
    """Loss and gradient captured for two batches on one workspace, replayed in
    turn with eager work between."""
    print(f"graphs B={B}", flush=True)
    cases = [Case(B, 200, 1700, (0, 800, 1700), seed=s) for s in (1, 2)]
    n = max(sb.sb_cross_entropy_workspace_bytes(c.head, g) for c in cases for g in (False, True))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    refs = [_all(c) for c in cases]
    graphs, outs = [], []
    for c in cases:
        loss, lse = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
        dx = torch.empty(B, 200, device="cuda", dtype=torch.bfloat16)
        dw = torch.empty(200, 1704, device="cuda", dtype=torch.bfloat16)[:, :1700]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sb.sb_cross_entropy(c.head, c.targets, loss, lse, ws=ws)
            sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss, dx, dw, ws=ws)
        graphs.append(g)
        outs.append((loss, lse, dx, dw))
    for turn in range(4):
        for g, out, ref, c in zip(graphs, outs, refs, cases):
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, ref):
                assert torch.equal(a, b), turn
            for a, b in zip(_all(c, ws=ws), ref):
                assert torch.equal(a, b)
    # the replay reads the inputs it finds
    cases[0].targets.fill_(-100)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert bool((outs[0][0] == 0).all()) and bool((outs[0][3] == 0).all())


def test_two_streams_at_once(require_gpu):
    """Two calls in flight, each with its own workspace."""
    cases = [Case(60 + 200 * i, 256, 4000, (0, 4000), seed=i) for i in range(2)]
    refs = [_all(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        got = []
        for c, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            loss, lse = torch.empty(c.B, device="cuda"), torch.empty(c.B, device="cuda")
            dx, dw = torch.empty_like(c.x), torch.empty(256, 4000, device="cuda", dtype=torch.bfloat16)
            dx = torch.empty(c.B, 256, device="cuda", dtype=torch.bfloat16)
            sb.sb_cross_entropy(c.head, c.targets, loss, lse, stream=s)
            sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss, dx, dw, stream=s)
            got.append((loss, lse, dx, dw))
        torch.cuda.synchronize()
        for a, b in zip(got, refs):
            for t, u in zip(a, b):
                assert torch.equal(t, u)


def test_refusals_leave_outputs_alone(require_gpu):
    c = Case(4, 64, 300, (0, 300))
    loss, lse = torch.full((4,), -7.0, device="cuda"), torch.full((4,), -7.0, device="cuda")
    with pytest.raises(TypeError, match="targets must be torch.int32"):
        sb.sb_cross_entropy(c.head, c.targets.long(), loss, lse)
    with pytest.raises(ValueError, match="lse must be contiguous with at least 4"):
        sb.sb_cross_entropy(c.head, c.targets, loss, lse[:3])
    with pytest.raises(ValueError, match="different devices"):
        sb._one_device([lse, torch.empty(1)])
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(sb.SbError) as e:
        sb.sb_cross_entropy(c.head, c.targets, loss, lse, ws=small)
    assert e.value.status == sb.SB_ERR_WORKSPACE
    dx = torch.empty(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="dx must be torch.bfloat16"):
        sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss, dx.float())
    with pytest.raises(ValueError, match="one tensor per lane"):
        sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss, None, [dx, dx])
    with pytest.raises(sb.SbError) as e:
        sb.sb_cross_entropy_grad(c.head, c.targets, lse, c.dloss)
    assert e.value.status == sb.SB_ERR_NULL
    torch.cuda.synchronize()
    assert bool((loss == -7).all()) and bool((lse == -7).all())
