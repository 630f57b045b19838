"""The loss, gradient and eight-bit operators of the output head as measured cases.

Each case is one pass through an operator on inputs that live on the GPU:

* ``loss``: softmax cross entropy of hidden rows against the vocabulary, with
  its logsumexp; rows whose target is negative are padding and cost nothing.
* ``grad``: the gradient of that loss with respect to the hidden rows and the
  head weight, given the forward's logsumexp and one weight per row.
* ``int8_logits`` / ``int8_tokens``: hidden rows quantised to 8 bits per row,
  times a head (or projection) weight held in 8 bits per channel: the scaled
  product itself, or its greedy token IDs.

With ``own`` false, ``run`` computes them with elementary torch operations;
with ``own`` true, through the package's entry points.
"""
import math

import torch

own = False

# Largest product B * H * V of any case.
MOST = 4096 * 5120 * 151936


def listed():
    return [
        # a unit-test-sized head: latency
        dict(name="loss_tiny", op="loss", B=4, H=256, V=4096, k=2),
        # scoring one position on one GPU's lane of the dense head
        dict(name="loss_one_row", op="loss", B=1, H=5120, V=37984, k=1),
        # a short evaluation batch, one row over whole blocks, odd width and vocabulary
        dict(name="loss_odd", op="loss", B=257, H=1111, V=50257, k=3),
        # a training or evaluation batch of the dense head
        dict(name="loss_prefill", op="loss", B=2048, H=5120, V=151936, k=4),
        # one optimiser step of a unit-test-sized head: latency
        dict(name="grad_tiny", op="grad", B=4, H=256, V=4096, k=2),
        # a few rows on one GPU's lane: bound by the weight and its gradient
        dict(name="grad_few_rows", op="grad", B=16, H=5120, V=37984, k=1),
        # a ragged training batch, odd in every size
        dict(name="grad_odd", op="grad", B=333, H=1111, V=50257, k=3),
        # a training step's batch on the dense head
        dict(name="grad_train", op="grad", B=4096, H=5120, V=151936, k=4),
        # decoding one row: latency and the weight's bytes
        dict(name="int8_one_row", op="int8_tokens", B=1, H=5120, V=37984, k=1),
        # dense decode with the head in 8 bits
        dict(name="int8_decode", op="int8_tokens", B=16, H=5120, V=151936, k=4),
        # the MLP's down projection as an 8-bit product
        dict(name="int8_down", op="int8_logits", B=64, H=17408, V=5120, k=1, out="bf16"),
        # prompt logits of the dense head in 8 bits
        dict(name="int8_prefill", op="int8_logits", B=2048, H=5120, V=151936, k=4, out="fp32"),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["loss", "grad", "int8_tokens", "int8_logits"])
    while True:
        B = _between(rng, 1, 4096)
        H = _between(rng, 128, 17408 if op.startswith("int8") else 8192)
        V = _between(rng, 1000, 200064)
        if B * H * V <= MOST:
            break
    case = dict(op=op, B=B, H=H, V=V, k=rng.choice([1, 2, 3, 4, 8]))
    if op == "int8_logits":
        case["out"] = rng.choice(["fp32", "bf16"])
    return case


def _up(n, m):
    return (n + m - 1) // m * m


def _lanes(V, k):
    """k nearly equal vocabulary lanes whose offsets are multiples of 8."""
    return [V * i // k // 8 * 8 for i in range(k)] + [V]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    B, H, V = case["B"], case["H"], case["V"]

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    state = dict(case=dict(case), lanes=_lanes(V, case["k"]))
    if case["op"].startswith("int8"):
        # hidden rows as a norm leaves them: unit variance and a few wide channels
        x = normal(B, _up(H, 8))
        x[:, ::97] *= 8
        state["x"] = x.to(torch.bfloat16)[:, :H]
        # channel weights in 8 bits, zero padding up to whole 16-byte units
        q = torch.zeros(V, _up(H, 16), dtype=torch.int8, device="cuda")
        q[:, :H] = torch.randint(-127, 128, (V, H), device="cuda", generator=g, dtype=torch.int8)
        state["w"] = q[:, :H]
        state["w_scale"] = 0.02 / 73 * (0.5 + uniform(V))
        return state
    w = torch.empty(H, _up(V, 8), dtype=torch.bfloat16, device="cuda")
    w.copy_(normal(H, _up(V, 8)) * 0.02)
    state["w"] = w[:, :V]
    targets = torch.randint(0, V, (B,), device="cuda", generator=g)
    # a model that has learned something: hidden rows lean towards their
    # target's column, some hardly and some enough to be confident
    x = normal(B, _up(H, 8))
    x[:, :H] += (6 * uniform(B))[:, None] * state["w"][:, targets].t().float()
    state["x"] = x.to(torch.bfloat16)[:, :H]
    # one position in ten is padding, but not the first
    pad = uniform(B) < 0.1
    pad[0] = False
    state["targets"] = torch.where(pad, -100, targets).to(torch.int32)
    if case["op"] == "grad":
        state["lse"] = torch.logsumexp(state["x"].float() @ state["w"].float(), 1)
        # the mean over the kept rows, each weighted by its sequence
        state["dloss"] = (0.5 + uniform(B)) / (~pad).sum()
    return state


def _run_own(s):
    from logit_source_projection_amd import sb

    c = s["case"]
    B, H, V, op = c["B"], c["H"], c["V"], c["op"]
    if op.startswith("int8"):
        if "head" not in s:  # the descriptor, quantised rows and workspace that a program keeps
            xq = torch.empty(B, _up(H, 16), dtype=torch.int8, device="cuda")[:, :H]
            xs = torch.empty(B, dtype=torch.float32, device="cuda")
            s["head"] = sb.Int8Head(xq, xs, s["w"], s["w_scale"], s["lanes"])
            s["ws"] = sb.int8_workspace(s["head"], sb.SB_SURF_TOKENS if op == "int8_tokens"
                                        else sb.SB_SURF_FULL_LOGITS)
        head = s["head"]
        sb.sb_int8_quantize_rows(s["x"], head.x, head.x_scale)
        if op == "int8_tokens":
            ids = torch.empty(B, dtype=torch.int32, device="cuda")
            return sb.sb_int8_project_tokens(head, ids, ws=s["ws"])
        out = torch.empty(B, _up(V, 8), device="cuda",
                          dtype=torch.float32 if c["out"] == "fp32" else torch.bfloat16)[:, :V]
        return sb.sb_int8_logits(head, out, ws=s["ws"])
    if "head" not in s:
        s["head"] = sb.Head(s["x"], s["w"], s["lanes"])
        s["ws"] = sb.cross_entropy_workspace(s["head"], grad=op == "grad")
    if op == "loss":
        loss = torch.empty(B, device="cuda")
        lse = torch.empty(B, device="cuda")
        sb.sb_cross_entropy(s["head"], s["targets"], loss, lse, ws=s["ws"])
        return {"loss": loss, "lse": lse}
    dx = torch.empty(B, _up(H, 8), dtype=torch.bfloat16, device="cuda")[:, :H]
    dw = torch.empty(H, _up(V, 8), dtype=torch.bfloat16, device="cuda")[:, :V]
    sb.sb_cross_entropy_grad(s["head"], s["targets"], s["lse"], s["dloss"], dx, dw, ws=s["ws"])
    return {"dx": dx, "dw": dw}


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    x, w = state["x"], state["w"]
    if op.startswith("int8"):
        # symmetric scale per row, quotients rounded to the nearest (ties to even)
        scale = (x.double().abs().amax(1) / 127).float()
        q = (x.float() / scale[:, None]).round()
        # integer sums pass 2^24, where 32-bit floats stop being exact
        sums = (q.double() @ w.double().t()).float()
        z = sums * scale[:, None] * state["w_scale"]
        if op == "int8_tokens":
            return z.argmax(1).to(torch.int32)
        return z if state["case"]["out"] == "fp32" else z.to(torch.bfloat16)
    xf, wf = x.float(), w.float()
    z = xf @ wf
    targets = state["targets"].long()
    kept = targets >= 0
    at = targets.clamp(min=0)[:, None]
    if op == "loss":
        top = z.amax(1)
        lse = top + (z - top[:, None]).exp().sum(1).log()
        loss = torch.where(kept, lse - z.gather(1, at)[:, 0], 0.0)
        return {"loss": loss, "lse": lse}
    dz = (z - state["lse"][:, None]).exp()
    dz.scatter_add_(1, at, torch.full_like(dz[:, :1], -1.0))
    dz *= torch.where(kept, state["dloss"], 0.0)[:, None]
    return {"dx": (dz @ wf.t()).to(torch.bfloat16), "dw": (xf.t() @ dz).to(torch.bfloat16)}


def work(case):
    B, H, V = case["B"], case["H"], case["V"]
    if case["op"].startswith("int8"):
        out = 4 * B if case["op"] == "int8_tokens" else B * V * (4 if case["out"] == "fp32" else 2)
        return {"bytes": 2 * B * H + V * H + 4 * V + out, "flops": 2 * B * H * V}
    if case["op"] == "loss":
        return {"bytes": 2 * B * H + 2 * H * V + 12 * B, "flops": 2 * B * H * V}
    # operands read and their gradients written; logits, dx and dw are one product each
    return {"bytes": 4 * B * H + 4 * H * V + 12 * B, "flops": 6 * B * H * V}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("int8"):
        if op == "int8_tokens":
            return None  # whole numbers: equal to the plain form's
        # the scale is the row maximum over 127 and the quotient a 32-bit
        # number by definition; everything after them is exact
        x64 = s["x"].double()
        scale = (x64.abs().max(dim=1).values / 127).float().double()
        codes = torch.round((x64 / scale.unsqueeze(1)).float()).double()
        return torch.mm(codes * scale.unsqueeze(1),
                        (s["w"].double() * s["w_scale"].double().unsqueeze(1)).t())
    x64, w64 = s["x"].double(), s["w"].double()
    logits = torch.mm(x64, w64)
    rows = torch.nonzero(s["targets"] >= 0)[:, 0]
    cols = s["targets"][rows].long()
    if op == "loss":
        lse = torch.logsumexp(logits, dim=1)
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - logits[rows, cols]
        return {"loss": loss, "lse": lse}
    per_row = torch.zeros_like(logits[:, 0])
    per_row[rows] = s["dloss"][rows].double()
    p = torch.exp(logits - s["lse"].double().unsqueeze(1))
    p[rows, cols] -= 1
    p *= per_row.unsqueeze(1)
    return {"dx": torch.mm(p, w64.t()), "dw": torch.mm(x64.t(), p)}
