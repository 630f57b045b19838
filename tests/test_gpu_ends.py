"""The operators around the head run together: a training step from token IDs to the
gradient of the embedding, a decoding step from drafted tokens to verified ones;
then each of them captured into a graph, on another stream, and several at once."""
import numpy as np
import pytest
import torch

from logit_source_projection_amd import sb
from tests import loss_common, norm_common, test_gpu_verify
from tests.test_gpu_embed import make_ids, reference_grad

pytestmark = pytest.mark.gpu

F, H16 = torch.float32, torch.bfloat16
HALF = 2.0 ** -8  # half a step of bf16


def randn(*shape, seed=0):
    return torch.randn(*shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))


@pytest.mark.parametrize("B,V,H", [(48, 1000, 64), (300, 4096, 200)])
def test_a_training_step(require_gpu, B, V, H):
    """ids -> embedding -> layer norm -> loss, and back to every parameter."""
    table, weight, bias = randn(V, H, seed=1), 1 + 0.1 * randn(H, seed=2), 0.1 * randn(H, seed=3)
    head_w = (randn(H, V, seed=4) * 0.1).to(H16)
    ids, targets = make_ids("ranks", B, V, 5), make_ids("uniform", B, V, 6)
    ids[3], targets[5] = -1, -1
    scale = H ** 0.5
    off = [0, V // 4 // 8 * 8, V]
    # forward
    x = sb.sb_embed(sb.Table(table, off), ids, torch.empty(B, H, device="cuda"), scale=scale)
    norm, y = sb.Norm(x, weight, bias), torch.empty(B, H, dtype=H16, device="cuda")
    mean, rstd, loss, lse = (torch.empty(B, device="cuda") for _ in range(4))
    sb.sb_layer_norm(norm, y, mean, rstd)
    head = sb.Head(y, head_w, off)
    sb.sb_cross_entropy(head, targets, loss, lse)
    # backward of the mean over the kept rows
    dloss = torch.full((B,), 1 / int((targets >= 0).sum()), device="cuda")
    dy, dw = torch.empty_like(y), torch.empty_like(head_w)
    sb.sb_cross_entropy_grad(head, targets, lse, dloss, dy, dw)
    dx, dweight, dbias = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(bias)
    sb.sb_layer_norm_grad(norm, dy, mean, rstd, dx, dweight, dbias)
    dtable = torch.empty_like(table)
    sb.sb_embed_grad(sb.Table(dtable, off), ids, dx, scale=scale)
    # each step against its definition on what it was given
    norm_common.check_forward(y, mean, rstd, x, weight, bias)
    loss_common.check_loss(loss, lse, y, head_w, targets)
    loss_common.check_grad(dy, dw, y, head_w, targets, dloss, lse)
    norm_common.check_gradient(dx, dweight, dbias, x, weight, dy, mean, rstd)
    want = reference_grad(ids, dx, V, scale)
    terms = reference_grad(ids, dx.abs(), V, scale)
    assert bool(((dtable.double() - want).abs() <= (B + 18) * 2.0 ** -24 * terms).all())
    # and all of it against 64 bits: y, dz and dy are rounded to bf16 on the way, and dW at
    # its end, each by at most half a step
    t, w, b, hw = (p.double().clone().requires_grad_() for p in (table, weight, bias, head_w))
    rows = torch.where((ids >= 0)[:, None], t[ids.long().clamp(min=0)] * scale, 0.0)
    z = torch.nn.functional.layer_norm(rows, (H,), w, b, 1e-5) @ hw
    keep = targets >= 0
    torch.nn.functional.cross_entropy(z[keep], targets[keep].long()).backward()
    for name, got, ref in (("table", dtable, t.grad), ("weight", dweight, w.grad), ("bias", dbias, b.grad),
                           ("head", dw, hw.grad)):
        off_by = torch.linalg.vector_norm(got.double() - ref)
        assert off_by <= 4 * HALF * torch.linalg.vector_norm(ref), (name, float(off_by / ref.norm()))


@pytest.mark.parametrize("greedy", [True, False])
@pytest.mark.parametrize("drawn", [True, False])
def test_a_decoding_step(require_gpu, drawn, greedy):
    """Drafted IDs -> embedding -> layer norm -> logits -> verified IDs."""
    N, K, V, H = 9, 3, 3000, 128
    counts = [3, 0, 1, 2, 3, 3, 0, 2, 1]
    T = sum(counts)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    table, head_w = randn(V, H, seed=1).to(H16), (randn(H, V, seed=2) * 0.2).to(H16)
    last, drafted = make_ids("uniform", N, V, 3), make_ids("uniform", T, V, 4)
    # the batch: every sequence's last token, then its drafts
    ids = torch.cat([torch.cat([last[i:i + 1], drafted[offsets[i]:offsets[i + 1]]]) for i in range(N)])
    x = sb.sb_embed(sb.Table(table), ids, torch.empty(T + N, H, dtype=H16, device="cuda"))
    y = sb.sb_layer_norm(sb.Norm(x), torch.empty_like(x))
    logits, best = torch.empty(T + N, V, device="cuda"), torch.empty(T + N, dtype=torch.int32, device="cuda")
    sb.sb_full_logits(sb.Head(y, head_w, [0, 1024, V]), logits, best)
    if greedy:  # some drafts that are right
        first = offsets[:-1].long() + torch.arange(N, device="cuda")
        for i in (0, 3, 4):
            drafted[offsets[i]] = best[first[i]]
    s = dict(counts=counts, K=K, V=V, target=logits, off=offsets, tokens=drafted, u=torch.rand(T, device="cuda"),
             u_next=torch.rand(N, device="cuda"), draft=logits[:T] + 0.5 * randn(T, V, seed=7) if drawn else None,
             temperature=torch.zeros(N, device="cuda") if greedy else None)
    out, accepted = test_gpu_verify.check(s)
    if greedy:
        assert accepted[0] >= 1
        for i in range(N):
            assert out[i, accepted[i]] == best[int(first[i]) + accepted[i]]


def operators():
    """name -> (inputs that may change, call(stream, ws), outputs)."""
    B, H, V = 40, 264, 5000
    cases = {}
    x, dy = randn(B, H, seed=1), randn(B, H, seed=2).to(H16)
    w, b = randn(H, seed=3), randn(H, seed=4)
    n = sb.Norm(x, w, b)
    y, mean, rstd = torch.empty(B, H, dtype=H16, device="cuda"), torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
    cases["layer norm"] = ([x], lambda stream, ws: sb.sb_layer_norm(n, y, mean, rstd, stream=stream), [y, mean, rstd], None)
    m2, r2 = x.mean(1), 1 / x.std(1)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    cases["layer norm gradient"] = (
        [x, dy], lambda stream, ws: sb.sb_layer_norm_grad(n, dy, m2, r2, dx, dw, db, ws=ws, stream=stream), [dx, dw, db],
        lambda: sb.layer_norm_grad_workspace(n))
    # the same of more rows than one launch takes
    x5, dy5 = randn(500, H, seed=9), randn(500, H, seed=10)
    n5, m5, r5 = sb.Norm(x5, w, b), x5.mean(1), 1 / x5.std(1)
    dx5, dw5, db5 = torch.empty_like(x5), torch.empty_like(w), torch.empty_like(b)
    cases["layer norm gradient, more rows"] = (
        [x5, dy5], lambda stream, ws: sb.sb_layer_norm_grad(n5, dy5, m5, r5, dx5, dw5, db5, ws=ws, stream=stream),
        [dx5, dw5, db5], lambda: sb.layer_norm_grad_workspace(n5))
    table, ids = randn(V, H, seed=5), make_ids("ranks", 300, V, 6)
    t, out = sb.Table(table, [0, 1000, V]), torch.empty(300, H, device="cuda")
    cases["embedding"] = ([table, ids], lambda stream, ws: sb.sb_embed(t, ids, out, scale=2.0, stream=stream), [out], None)
    dout, dtable = randn(300, H, seed=7), torch.empty(V, H, device="cuda")
    dt = sb.Table(dtable, [0, 1000, V])
    cases["embedding gradient"] = (
        [dout, ids], lambda stream, ws: sb.sb_embed_grad(dt, ids, dout, scale=2.0, ws=ws, stream=stream), [dtable],
        lambda: sb.embed_grad_workspace(dt, 300))
    s = test_gpu_verify.make([3, 0, 2, 3, 1] * 4, 3, 9001, F, True, 8)
    d = sb.Drafts(s["target"], s["tokens"], s["off"], 3, s["draft"], s["temperature"])
    tokens, accepted = torch.empty(20, 4, dtype=torch.int32, device="cuda"), torch.empty(20, dtype=torch.int32, device="cuda")
    cases["verification"] = (
        [s["target"], s["u"], s["u_next"]],
        lambda stream, ws: sb.sb_verify_drafts(d, s["u"], s["u_next"], tokens, accepted, ws=ws, stream=stream),
        [tokens, accepted], lambda: sb.verify_workspace(d))
    return cases


NAMES = ["layer norm", "layer norm gradient", "layer norm gradient, more rows", "embedding", "embedding gradient",
         "verification"]


def change(inputs, seed):
    """Other values in the same tensors."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for t in inputs:
        if t.dtype == torch.int32:
            t.copy_(t[torch.randperm(t.numel(), device="cuda", generator=g)])
        elif t.dim() == 1:
            t.uniform_(generator=g)
        else:
            t.copy_(torch.randn(t.shape, device="cuda", generator=g))


@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(require_gpu, name):
    inputs, call, outputs, workspace = operators()[name]
    ws = workspace() if workspace else None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call(None, ws)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(None, ws)
    for replay in range(5):
        change(inputs, replay)
        if ws is not None:
            ws.fill_(255 if replay % 2 else 90)
        for t in outputs:
            t.fill_(-7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(-5)
        call(None, ws)
        torch.cuda.synchronize()
        for a, b in zip(got, outputs):
            assert torch.equal(a, b), (name, replay)


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(require_gpu, name):
    """A stream object, its handle and the current stream; the workspace given or not,
    and what is in it."""
    inputs, call, outputs, workspace = operators()[name]
    call(None, None)
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        for fill in (None, 0, 255, 0x5A):
            ws = workspace() if workspace and fill is not None else None
            if ws is not None:
                ws.fill_(fill)
            for t in outputs:
                t.fill_(-7)
            side.wait_stream(torch.cuda.current_stream())
            if stream is None:
                with torch.cuda.stream(side):
                    call(None, ws)
            else:
                call(stream, ws)
            side.synchronize()
            for a, b in zip(want, outputs):
                assert torch.equal(a, b), (name, fill)


def test_all_at_once(require_gpu):
    """Each operator on a stream of its own, many times over, beside the others."""
    cases = operators()
    want = {}
    for name, (_, call, outputs, _) in cases.items():
        call(None, None)
        torch.cuda.synchronize()
        want[name] = [t.clone() for t in outputs]
        for t in outputs:
            t.fill_(-7)
    streams = {name: torch.cuda.Stream() for name in cases}
    spaces = {name: case[3]() if case[3] else None for name, case in cases.items()}
    torch.cuda.synchronize()
    for _ in range(20):
        for name, (_, call, _, _) in cases.items():
            call(streams[name], spaces[name])
    torch.cuda.synchronize()
    for name, (_, _, outputs, _) in cases.items():
        for a, b in zip(want[name], outputs):
            assert torch.equal(a, b), name


def test_tensors_of_several_devices_are_refused(require_gpu):
    cases = operators()
    for name in ("layer norm", "embedding"):
        with pytest.raises(ValueError):
            other = torch.empty(40, 264)
            if name == "layer norm":
                sb.sb_layer_norm(sb.Norm(other.cuda(), other[0]), other.cuda())
            else:
                sb.sb_embed(sb.Table(other.cuda()), torch.zeros(40, dtype=torch.int32), other.cuda())
    assert cases


def test_all_at_once_every_round(require_gpu):
    """As above, but every round has other inputs, and its outputs are kept: copied on the
    operator's own stream before the next round writes them, they equal those of the same
    inputs alone."""
    rounds = 12
    cases = {name: operators()[name] for name in NAMES}  # (of one set, two read the same rows)
    fresh = {name: [[t.clone() for t in inputs]] for name, (inputs, _, _, _) in cases.items()}
    want = {name: [] for name in cases}
    for name, (inputs, call, outputs, _) in cases.items():
        for r in range(rounds):
            if r:
                change(inputs, 100 + r)
                fresh[name].append([t.clone() for t in inputs])
            for t in outputs:
                t.fill_(-7)
            call(None, None)
            torch.cuda.synchronize()
            want[name].append([t.clone() for t in outputs])
        assert any(not torch.equal(a, b) for a, b in zip(want[name][0], want[name][1])), name
    streams = {name: torch.cuda.Stream() for name in cases}
    spaces = {name: case[3]() if case[3] else None for name, case in cases.items()}
    got = {name: [] for name in cases}
    torch.cuda.synchronize()
    for r in range(rounds):
        for name, (inputs, call, outputs, _) in cases.items():
            with torch.cuda.stream(streams[name]):
                for t, value in zip(inputs, fresh[name][r]):
                    t.copy_(value)
                for t in outputs:
                    t.fill_(-5)
                call(None, spaces[name])
                got[name].append([t.clone() for t in outputs])
    torch.cuda.synchronize()
    for name in cases:
        for r in range(rounds):
            for a, b in zip(want[name][r], got[name][r]):
                assert torch.equal(a, b), (name, r)
