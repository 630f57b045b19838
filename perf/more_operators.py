"""The operators around the output head as measured cases.

Each case is one pass through an operator on inputs that live on the GPU:

* ``norm``: layer norm of rows, with the mean and the reciprocal deviation
  that its gradient takes.
* ``norm_grad``: the gradient of layer norm for its rows, weight and bias.
* ``embed``: rows of an embedding table looked up by token IDs and scaled;
  negative IDs are padding and give rows of zeros.
* ``embed_grad``: the gradient of that lookup for the whole table.
* ``verify``: drafted tokens of many sequences verified against the target's
  logits from given random numbers: how many are accepted, and the token that
  follows them.  Temperature 0 is greedy.

With ``own`` false, ``run`` computes them with elementary torch operations;
with ``own`` true, through the package's entry points.
"""
import math

import torch

own = False

# Most values that one drawn case of an operator goes through: those of its
# largest listed case.
MOST_ROWS = 8192 * 5120
MOST_TABLE = 151936 * 5120
MOST_LOGITS = 64 * 15 * 151936


def listed():
    return [
        # decoding one row: latency
        dict(name="norm_one_row", op="norm", B=1, H=5120, x="bf16", y="bf16", params="bf16"),
        # a training batch whose rows stay in 32 bits and enter the head in 16
        dict(name="norm_train", op="norm", B=8192, H=5120, x="fp32", y="bf16", params="fp32"),
        # a few rows: latency, and few workgroups for the weight's gradient
        dict(name="norm_grad_few", op="norm_grad", B=16, H=5120, x="bf16", y="bf16", params="bf16"),
        # a ragged batch, odd in every size, all in 32 bits
        dict(name="norm_grad_odd", op="norm_grad", B=1333, H=1111, x="fp32", y="fp32", params="fp32"),
        # a training step's batch
        dict(name="norm_grad_train", op="norm_grad", B=8192, H=5120, x="bf16", y="bf16", params="fp32"),
        # the tokens of one decoding step
        dict(name="embed_decode", op="embed", B=16, V=151936, H=5120, k=4, table="bf16", out="bf16"),
        # a training batch's tokens
        dict(name="embed_train", op="embed", B=16384, V=151936, H=5120, k=1, table="bf16", out="bf16"),
        # a ragged batch on an odd table in 32 bits
        dict(name="embed_grad_odd", op="embed_grad", B=3333, V=50257, H=1111, k=3, table="fp32", out="bf16"),
        # a training step's tokens on the dense model's table
        dict(name="embed_grad_train", op="embed_grad", B=16384, V=151936, H=5120, k=4, table="bf16", out="bf16"),
        # one sequence with four drafts: latency
        dict(name="verify_one", op="verify", N=1, K=4, V=151936, dtype="fp32", drawn=True, ragged=False),
        # a batch of ragged lookups without a draft model, odd vocabulary
        dict(name="verify_lookup", op="verify", N=17, K=10, V=50257, dtype="fp32", drawn=False, ragged=True),
        # a serving batch with a draft model
        dict(name="verify_batch", op="verify", N=64, K=7, V=151936, dtype="fp32", drawn=True, ragged=False),
    ]


def _between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "embed", "embed_grad", "verify"])
    types = ["bf16", "fp32"]
    if op.startswith("norm"):
        while True:
            case = dict(op=op, B=_between(rng, 1, 16384), H=_between(rng, 64, 17408), x=rng.choice(types),
                        y=rng.choice(types), params=rng.choice(types))
            if case["B"] * case["H"] <= MOST_ROWS:
                return case
    if op.startswith("embed"):
        while True:
            case = dict(op=op, B=_between(rng, 1, 32768), V=_between(rng, 1000, 200064),
                        H=_between(rng, 64, 8192), k=rng.choice([1, 2, 3, 4, 8]), table=rng.choice(types),
                        out=rng.choice(types))
            wide = 2 if "fp32" in (case["table"], case["out"]) else 1
            if (case["V"] + 2 * case["B"]) * case["H"] * wide <= MOST_TABLE:
                return case
    while True:
        case = dict(op=op, N=_between(rng, 1, 128), K=rng.randint(1, 12), V=_between(rng, 1000, 200064),
                    dtype=rng.choice(types), drawn=rng.random() < 0.75, ragged=rng.random() < 0.5)
        if case["N"] * (2 * case["K"] + 1) * case["V"] <= MOST_LOGITS:
            return case


def _up(n, m):
    return (n + m - 1) // m * m


def _lanes(V, k):
    """k nearly equal vocabulary lanes."""
    return [V * i // k for i in range(k)] + [V]


def _type(name):
    return torch.float32 if name == "fp32" else torch.bfloat16


def _counts(case):
    """Drafted tokens of every sequence: K, or spread over 0 .. K."""
    K = case["K"]
    return [(7 * i + 3) % (K + 1) if case["ragged"] else K for i in range(case["N"])]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    state = dict(case=dict(case))
    if case["op"].startswith("norm"):
        B, H = case["B"], case["H"]
        params, ty = _type(case["params"]), _type(case["y"])
        # a residual stream: a mean of its own per row, a few wide channels
        x = normal(B, _up(H, 8)) + 0.3 * normal(B, 1)
        x[:, ::97] *= 8
        state["x"] = x.to(_type(case["x"]))[:, :H]
        state["weight"] = (1 + 0.1 * normal(H)).to(params)
        state["bias"] = (0.1 * normal(H)).to(params)
        if case["op"] == "norm_grad":
            xf = state["x"].float()
            state["mean"] = xf.mean(1)
            state["rstd"] = (xf.var(1, correction=0) + 1e-5).rsqrt()
            # a mean's gradient, with rows of different weight
            state["dy"] = (normal(B, _up(H, 8)) * (0.5 + uniform(B, 1)) / B).to(ty)[:, :H]
        return state
    if case["op"].startswith("embed"):
        B, V, H = case["B"], case["V"], case["H"]
        # frequencies of tokens fall with their rank; ranks lie anywhere in the vocabulary
        rank = (uniform(B) * math.log(V)).exp().long().clamp(1, V) - 1
        ids = torch.randperm(V, device="cuda", generator=g)[rank]
        # one position in fifty is padding, but not the first
        pad = uniform(B) < 0.02
        pad[0] = False
        state["ids"] = torch.where(pad, -1, ids).to(torch.int32)
        state["scale"] = math.sqrt(H)
        state["lanes"] = _lanes(V, case["k"])
        if case["op"] == "embed":
            table = torch.empty(V, _up(H, 8), dtype=_type(case["table"]), device="cuda")
            table.copy_(normal(V, _up(H, 8)) * 0.02)
            state["table"] = table[:, :H]
        else:
            state["dout"] = (normal(B, _up(H, 8)) / B).to(_type(case["out"]))[:, :H]
        return state
    N, K, V = case["N"], case["K"], case["V"]
    counts = _counts(case)
    drafts = sum(counts)
    off = torch.tensor([0] + counts, dtype=torch.int64, device="cuda").cumsum(0)
    # every fourth sequence is greedy, the others sample
    temperature = 0.6 + 0.6 * uniform(N)
    temperature[3::4] = 0
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), off.diff() + 1)
    last = off[1:] + torch.arange(N, device="cuda")  # the row behind a sequence's drafts
    # a tail that holds a part of the mass, and twenty likely tokens
    z = 2 * normal(drafts + N, _up(V, 8))
    likely = torch.randint(0, V, (drafts + N, 20), device="cuda", generator=g)
    z.scatter_(1, likely, math.log(V) + 2 + 4 * uniform(drafts + N, 20))
    target = z.to(_type(case["dtype"]))[:, :V]
    drafted = torch.ones(drafts + N, dtype=torch.bool, device="cuda")
    drafted[last] = False
    t = temperature[seq][drafted][:, None]
    near = z[drafted] + 0.7 * normal(drafts, _up(V, 8))
    draft = near.to(_type(case["dtype"]))[:, :V]
    noise = -(-uniform(drafts, V).clamp(min=1e-30).log()).log()
    score = torch.where(t > 0, draft.float() / t.clamp(min=0.1) + (noise if case["drawn"] else 0), draft.float())
    state.update(target=target, temperature=temperature, off=off.to(torch.int32), rows=drafts + N,
                 tokens=score.argmax(1).to(torch.int32) if drafts else torch.zeros(0, dtype=torch.int32, device="cuda"),
                 u=uniform(drafts), u_next=uniform(N))
    state["draft"] = draft if case["drawn"] else None
    return state


def _run_own(s):
    from logit_source_projection_amd import sb

    c = s["case"]
    op = c["op"]
    if op.startswith("norm"):
        B, H = c["B"], c["H"]
        if "desc" not in s:  # the descriptor and workspace that a program keeps
            s["desc"] = sb.Norm(s["x"], s["weight"], s["bias"], eps=1e-5)
            s["ws"] = sb.layer_norm_grad_workspace(s["desc"]) if op == "norm_grad" else None
        if op == "norm":
            y = torch.empty(B, _up(H, 8), dtype=_type(c["y"]), device="cuda")[:, :H]
            mean, rstd = torch.empty(B, device="cuda"), torch.empty(B, device="cuda")
            sb.sb_layer_norm(s["desc"], y, mean, rstd)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx = torch.empty(B, _up(H, 8), dtype=_type(c["x"]), device="cuda")[:, :H]
        dweight, dbias = torch.empty_like(s["weight"]), torch.empty_like(s["bias"])
        sb.sb_layer_norm_grad(s["desc"], s["dy"], s["mean"], s["rstd"], dx, dweight, dbias, ws=s["ws"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "embed":
        if "desc" not in s:
            s["desc"] = sb.Table(s["table"], s["lanes"])
        out = torch.empty(c["B"], _up(c["H"], 8), dtype=_type(c["out"]), device="cuda")[:, :c["H"]]
        return sb.sb_embed(s["desc"], s["ids"], out, scale=s["scale"])
    if op == "embed_grad":
        if "desc" not in s:
            s["dtable"] = torch.empty(c["V"], _up(c["H"], 8), dtype=_type(c["table"]), device="cuda")[:, :c["H"]]
            s["desc"] = sb.Table(s["dtable"], s["lanes"])
            s["ws"] = sb.embed_grad_workspace(s["desc"], c["B"])
        sb.sb_embed_grad(s["desc"], s["ids"], s["dout"], scale=s["scale"], ws=s["ws"])
        return s["dtable"]
    if "desc" not in s:
        s["desc"] = sb.Drafts(s["target"], s["tokens"], s["off"], c["K"], draft=s["draft"],
                              temperature=s["temperature"])
        s["ws"] = sb.verify_workspace(s["desc"])
    out = torch.empty(c["N"], c["K"] + 1, dtype=torch.int32, device="cuda")
    accepted = torch.empty(c["N"], dtype=torch.int32, device="cuda")
    sb.sb_verify_drafts(s["desc"], s["u"], s["u_next"], out, accepted, ws=s["ws"])
    return {"tokens": out, "accepted": accepted}


def _verify(s):
    # in 64 bits throughout: drawn numbers meet the borders of a cumulative sum
    N, K = s["case"]["N"], s["case"]["K"]
    off, tokens = s["off"].long(), s["tokens"].long()
    z = s["target"]
    seq = torch.repeat_interleave(torch.arange(N, device="cuda"), off.diff() + 1, output_size=s["rows"])
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"].double())[seq][:, None]

    def softmax(v, t):
        e = ((v.double() - v.double().amax(1, keepdim=True)) / t).exp()
        return e / e.sum(1, keepdim=True)

    p, best = softmax(z, t), z.argmax(1)
    # draft j of sequence i, where there is one
    j = torch.arange(K, device="cuda")
    at = off[:-1, None] + j
    there = at < off[1:, None]
    at = torch.where(there, at, 0)
    row = torch.where(there, at + torch.arange(N, device="cuda")[:, None], 0)
    first = off[:-1] + torch.arange(N, device="cuda")  # a sequence's first row
    if not tokens.numel():
        accepted = torch.zeros(N, dtype=torch.int64, device="cuda")
        x = at
        rest = p[first]
    else:
        x = tokens[at]
        px = p[row, x]
        if s["draft"] is not None:
            td = torch.where(greedy, 1.0, s["temperature"].double()).repeat_interleave(off.diff(), output_size=len(tokens))
            q = softmax(s["draft"], td[:, None])
            qx = q[at, x]
        else:
            qx = torch.ones_like(px)
        ok = torch.where(greedy[:, None], best[row] == x, s["u"].double()[at] * qx < px) & there
        accepted = ok.long().cumprod(1).sum(1)
        # what is left where a draft was rejected, or the row behind the last one
        rest = p[first + accepted]
        rejected = accepted < off.diff()
        last = torch.where(rejected, off[:-1] + accepted, 0)
        if s["draft"] is not None:
            less = (rest - q[last]).clamp(min=0)
        else:
            less = rest.scatter(1, tokens[last][:, None], 0.0)
        rest = torch.where(rejected[:, None] & (less.sum(1, keepdim=True) > 0), less, rest)
    sums = rest.cumsum(1)
    drawn = (sums <= s["u_next"].double()[:, None] * sums[:, -1:]).sum(1)
    follows = torch.where(greedy, best[first + accepted], drawn)
    steps = torch.arange(K + 1, device="cuda")
    out = torch.where(steps < accepted[:, None], torch.nn.functional.pad(x, (0, 1)), -1)
    out = torch.where(steps == accepted[:, None], follows[:, None], out)
    return {"tokens": out.to(torch.int32), "accepted": accepted.to(torch.int32)}


def run(state):
    if own:
        return _run_own(state)
    c = state["case"]
    op = c["op"]
    if op == "norm":
        x = state["x"].float()
        mean = x.mean(1)
        d = x - mean[:, None]
        rstd = ((d * d).mean(1) + 1e-5).rsqrt()
        y = d * rstd[:, None] * state["weight"].float() + state["bias"].float()
        return {"y": y.to(_type(c["y"])), "mean": mean, "rstd": rstd}
    if op == "norm_grad":
        dy, rstd = state["dy"].float(), state["rstd"][:, None]
        xh = (state["x"].float() - state["mean"][:, None]) * rstd
        g = dy * state["weight"].float()
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        params = _type(c["params"])
        return {"dx": dx.to(_type(c["x"])), "dweight": (dy * xh).sum(0).to(params), "dbias": dy.sum(0).to(params)}
    if op == "embed":
        ids = state["ids"].long()
        rows = state["table"][ids.clamp(min=0)].float() * state["scale"]
        return torch.where((ids >= 0)[:, None], rows, 0.0).to(_type(c["out"]))
    if op == "embed_grad":
        ids = state["ids"].long()
        rows = torch.where((ids >= 0)[:, None], state["dout"].float(), 0.0)
        sums = torch.zeros(c["V"], c["H"], device="cuda")
        sums.index_add_(0, ids.clamp(min=0), rows)
        return (sums * state["scale"]).to(_type(c["table"]))
    return _verify(state)


def _bytes(name):
    return 4 if name == "fp32" else 2


def work(case):
    op = case["op"]
    if op.startswith("norm"):
        B, H = case["B"], case["H"]
        rows = B * H * (_bytes(case["x"]) + _bytes(case["y"]))
        params = H * _bytes(case["params"])
        if op == "norm":
            return {"bytes": rows + 2 * params + 8 * B, "flops": 8 * B * H}
        return {"bytes": rows + B * H * _bytes(case["x"]) + 3 * params + 8 * B, "flops": 14 * B * H}
    if op.startswith("embed"):
        B, V, H = case["B"], case["V"], case["H"]
        if op == "embed":
            # distinct rows of the table, by the distribution of the tokens
            rows = sum(1 - (1 - math.log1p(1 / (r + 1)) / math.log(V)) ** B for r in range(V))
            return {"bytes": rows * H * _bytes(case["table"]) + B * H * _bytes(case["out"]) + 4 * B, "flops": B * H}
        return {"bytes": V * H * _bytes(case["table"]) + B * H * _bytes(case["out"]) + 4 * B, "flops": 2 * B * H}
    drafts, V = sum(_counts(case)), case["V"]
    rows = drafts + case["N"] + (drafts if case["drawn"] else 0)
    # a difference, an exponential and a sum for every logit
    return {"bytes": rows * V * _bytes(case["dtype"]), "flops": 3 * rows * V}


def exact(case, seed):
    op = case["op"]
    if op == "verify":
        return None  # whole numbers: equal to the plain form's
    s = prepare(case, seed)
    if op.startswith("norm"):
        x = s["x"].double()
        w, H = s["weight"].double(), case["H"]
        if op == "norm":
            var, mean = torch.var_mean(x, dim=1, correction=0)
            rstd = torch.pow(var + 1e-5, -0.5)
            y = torch.addcmul(s["bias"].double(), (x - mean.unsqueeze(1)) * w, rstd.unsqueeze(1))
            return {"y": y, "mean": mean, "rstd": rstd}
        r = s["rstd"].double().unsqueeze(1)
        dy = s["dy"].double()
        xh = torch.sub(x, s["mean"].double().unsqueeze(1)) * r
        a = torch.mv(dy, w) / H
        b = torch.mv(dy * xh, w) / H
        dx = torch.addcmul(dy * w - a.unsqueeze(1), xh, b.unsqueeze(1), value=-1) * r
        one = torch.ones(case["B"], dtype=torch.float64, device="cuda")
        return {"dx": dx, "dweight": torch.mv((dy * xh).t(), one), "dbias": torch.mv(dy.t(), one)}
    ids = s["ids"].long()
    kept = torch.nonzero(ids >= 0)[:, 0]
    if op == "embed":
        out = torch.zeros(case["B"], case["H"], dtype=torch.float64, device="cuda")
        out[kept] = torch.index_select(s["table"], 0, ids[kept]).double() * s["scale"]
        return out
    out = torch.zeros(case["V"], case["H"], dtype=torch.float64, device="cuda")
    return out.index_put_((ids[kept],), s["dout"][kept].double() * s["scale"], accumulate=True)
