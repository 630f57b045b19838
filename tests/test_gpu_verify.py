"""Verification of drafted tokens on the GPU against a plain implementation in 64
bits, one sequence at a time.  Tokens are whole numbers and have to be equal: both
sides sum in 64 bits, and their cumulative sums differ by about 1e-14 of the whole,
so that a random number falls between them once in 1e8 draws."""
import math

import numpy as np
import pytest
import torch

from logit_source_projection_amd import sb

pytestmark = pytest.mark.gpu

F, H16 = torch.float32, torch.bfloat16


def softmax(z, t):
    """None where the row has no distribution."""
    z = z.astype(np.float64)
    if np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return None
    with np.errstate(invalid="ignore"):
        e = np.exp((z - z.max()) / t)
    e[z == -np.inf] = 0
    return e / e.sum()


def draw(weights, u):
    sums = np.cumsum(weights)
    goal = (u if u > 0 else 0.0) * sums[-1]
    there = np.nonzero((sums > goal) & (weights > 0))[0]
    return int(there[0]) if len(there) else int(np.nonzero(weights > 0)[0][-1])


def one_sequence(z, y, x, u, u_next, t):
    """Accepted drafts and the token behind them; y is None without draft logits."""
    n, V = len(x), z.shape[1]
    if not t > 0:
        best = z.argmax(1)  # NaN first, then the lowest index, as numpy's
        for j in range(n):
            if best[j] != x[j]:
                return j, int(best[j])
        return n, int(best[n])
    for j in range(n):
        p = softmax(z[j], t)
        if p is None:
            return j, -1
        q = softmax(y[j], t) if y is not None else None
        inside = 0 <= x[j] < V
        ok = inside and (y is None or q is not None)
        qx = 1.0 if y is None else q[x[j]] if ok else 0.0
        if ok and float(u[j]) * qx < p[x[j]]:
            continue
        rest = p
        if y is not None:
            rest = np.maximum(p - q, 0) if q is not None else p
        elif inside:
            rest = p.copy()
            rest[x[j]] = 0
        return j, draw(rest if rest.sum() > 0 else p, float(u_next))
    p = softmax(z[n], t)
    return n, -1 if p is None else draw(p, float(u_next))


def reference(s):
    N, K = len(s["counts"]), s["K"]
    z = s["target"].float().cpu().numpy()
    y = None if s["draft"] is None else s["draft"].float().cpu().numpy()
    x, u, un = (s[k].cpu().numpy() for k in ("tokens", "u", "u_next"))
    t = np.ones(N) if s["temperature"] is None else s["temperature"].double().cpu().numpy()
    out, acc, at = np.full((N, K + 1), -1), np.zeros(N, dtype=int), 0
    for i, n in enumerate(s["counts"]):
        m = min(n, K)
        a, token = one_sequence(z[at + i:at + i + m + 1], None if y is None else y[at:at + m], x[at:at + m],
                                u[at:at + m], un[i], t[i])
        out[i, :a], out[i, a], acc[i] = x[at:at + a], token, a
        at += n
    return out, acc


def make(counts, K, V, dtype=F, drawn=True, seed=0, spread=2.0, near=0.5, temperature="mixed", extra=8):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N, T = len(counts), sum(counts)

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    def uniform(*shape):
        return torch.rand(*shape, device="cuda", generator=g)

    def rows(n):
        return torch.full((n, -(-V // 8) * 8 + extra), float("nan"), dtype=dtype, device="cuda")[:, :V]

    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    target, draft = rows(T + N), rows(T)
    target.copy_(normal(T + N, V) * spread)
    is_draft = torch.ones(T + N, dtype=torch.bool, device="cuda")
    is_draft[off[1:].long() + torch.arange(N, device="cuda")] = False
    draft.copy_(target[is_draft].float() + near * normal(T, V))
    noise = -(-uniform(T, V).clamp(min=1e-30).log()).log()
    tokens = (draft.float() + noise).argmax(1) if T else torch.zeros(0, device="cuda")
    if not drawn and T:
        tokens = target[is_draft].float().argmax(1)
    t = None
    if temperature == "mixed":
        t = 0.5 + uniform(N)
        t[1::3] = 0
    elif temperature is not None:
        t = torch.full((N,), float(temperature), device="cuda")
    return dict(counts=list(counts), K=K, V=V, target=target, draft=draft if drawn else None, off=off,
                tokens=tokens.to(torch.int32), u=uniform(T), u_next=uniform(N), temperature=t)


def run(s, ws=None):
    N, K = len(s["counts"]), s["K"]
    d = sb.Drafts(s["target"], s["tokens"], s["off"], K, draft=s["draft"], temperature=s["temperature"])
    whole = torch.full((N, K + 4), -7, dtype=torch.int32, device="cuda")
    accepted = torch.full((N + 2,), -7, dtype=torch.int32, device="cuda")
    n = sb.sb_verify_workspace_bytes(d)
    ws = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    sb.sb_verify_drafts(d, s["u"], s["u_next"], whole[:, :K + 1], accepted, ws=ws[:n])
    assert bool((whole[:, K + 1:] == -7).all()) and bool((accepted[N:] == -7).all()), "outside"
    assert bool((ws[n:] == 255).all()), "workspace"
    return whole[:, :K + 1].cpu().numpy(), accepted[:N].cpu().numpy()


def check(s):
    got, want = run(s), reference(s)
    assert np.array_equal(got[1], want[1]), (got[1], want[1])
    assert np.array_equal(got[0], want[0]), np.nonzero((got[0] != want[0]).any(1))
    return got


COUNTS = [[0], [1], [4], [0, 3, 1, 5, 0, 2], [7] * 9, [2, 0, 12, 1] * 4, [1] * 130]


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("dtype", [F, H16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 100, 8191, 8192, 8193, 20000, 50257])
@pytest.mark.parametrize("counts", COUNTS, ids=lambda c: f"{len(c)}x{max(c)}")
def test_against_definition(require_gpu, counts, V, dtype, drawn):
    print(f"verify N={len(counts)} K={max(counts)} V={V} {dtype} drawn={drawn}", flush=True)
    if V * (sum(counts) + len(counts)) > 5_000_000:
        counts = counts[:20]
    check(make(counts, max(counts), V, dtype, drawn, seed=V + len(counts)))


@pytest.mark.parametrize("near", [0.0, 0.05, 3.0])
@pytest.mark.parametrize("spread", [0.0, 0.1, 10.0])
def test_flat_and_peaked_rows(require_gpu, spread, near):
    for t in (None, 0.2, 1.7, "mixed"):
        s = make([3] * 40, 3, 9000, F, True, 31, spread, near, t)
        accepted = check(s)[1]
        if near == 0.0 and t is not None and t != "mixed":
            assert (accepted == 3).all()  # p = q: u < 1 accepts
    check(make([5, 5], 5, 151936, F, True, 32, spread, near, None))


@pytest.mark.parametrize("dtype", [F, H16])
def test_large_vocabularies_and_many_drafts(require_gpu, dtype):
    """More chunks of a row than a wave has lanes, more rows than a verdict has waves."""
    check(make([2, 0, 1], 2, 1000003, dtype, True, 51, temperature="mixed"))
    check(make([1, 2], 2, 600000, dtype, False, 52, spread=0.0, temperature=None))
    for near in (0.05, 0.5):
        check(make([40, 33, 0, 17, 16, 15], 40, 3000, dtype, True, 53, near=near, temperature=0.9))
    s = make([40, 33, 0, 17], 40, 9000, dtype, False, 54, temperature=0.0)
    s["tokens"][60] = 5
    assert check(s)[1][0] == 40


def test_more_chunks_than_workgroups(require_gpu):
    check(make([4] * 150, 4, 20000, H16, True, 55))
    check(make([0] * 700, 0, 17000, F, False, 56))


def test_rows_far_apart(require_gpu):
    """Offsets past 32 bits."""
    s = make([2, 1], 2, 9001, H16, True, 57)
    for name in ("target", "draft"):
        t, ld = s[name], 1 << 30
        far = torch.empty((len(t) - 1) * ld + 9001, dtype=H16, device="cuda").as_strided(t.shape, (ld, 1))
        s[name] = far.copy_(t)
    check(s)


def test_more_drafts_than_allowed(require_gpu):
    check(make([6, 1, 9, 0], 4, 500, seed=3))
    check(make([3, 2], 0, 500, seed=4))


def test_borders_of_a_flat_row(require_gpu):
    """All logits equal: a multiple k / V of the whole draws exactly token k, across
    units, threads and chunks."""
    for V in (8, 4096, 16384):
        N = 512
        s = make([0] * N, 0, V, F, False, 1, 0.0, 0.0, None)
        k = torch.linspace(0, V - 1, N, device="cuda").round()
        s["u_next"] = k / V
        k = k.long().cpu().numpy()
        off = np.nonzero(run(s)[0][:, 0] != k)[0]
        assert not len(off), (V, off[:5])
        # just below a border: the token before (below 0 counts as 0)
        s["u_next"] = torch.nextafter(s["u_next"], torch.tensor(-1.0, device="cuda"))
        off = np.nonzero(run(s)[0][:, 0] != np.maximum(k - 1, 0))[0]
        assert not len(off), (V, off[:5])


def test_masked_rows(require_gpu):
    """Logits of -inf are never drawn, in masks that end inside units, threads and
    chunks and leave one token, or none."""
    V = 17000
    s = make([1] * 60, 1, V, F, True, 5, temperature="mixed")
    z = s["target"]
    for r in range(120):
        keep = [slice(r * 100, r * 100 + 1), slice(8190, 8194), slice(V - 1, V), slice(0, 1), slice(8192, V)][r % 5]
        row = z[r].clone()
        z[r] = -float("inf")
        z[r, keep] = row[keep]
    z[10] = -float("inf")  # nothing left of sequence 5's draft row
    z[21] = -float("inf")  # nor behind sequence 10's draft
    s["draft"][7] = -float("inf")
    out, accepted = check(s)
    if s["temperature"][5] > 0:
        assert out[5, 0] == -1 and accepted[5] == 0
    # the type's lowest number is a number: alone it makes a flat row
    s["target"][:] = torch.finfo(F).min
    check(s)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("nan")])
@pytest.mark.parametrize("V", [5, 9000])
def test_rows_without_a_distribution(require_gpu, V, bad):
    for seed in range(3):
        s = make([2] * 30, 2, V, F, True, 40 + seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = torch.randint(0, 90, (12,), device="cuda", generator=g)
        s["target"][rows, torch.randint(0, V, (12,), device="cuda", generator=g)] = bad
        rows = torch.randint(0, 60, (8,), device="cuda", generator=g)
        s["draft"][rows, torch.randint(0, V, (8,), device="cuda", generator=g)] = bad
        check(s)


def test_random_numbers_at_their_ends(require_gpu):
    for V in (6, 9000):
        for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan")):
            for drawn in (True, False):
                s = make([2] * 12, 2, V, F, drawn, 6, temperature=0.8)
                s["u"].fill_(u)
                s["u_next"].fill_(u)
                s["target"][:, -1] = -float("inf")
                check(s)


def test_nothing_left_of_a_row(require_gpu):
    """The draft model equals the target and u is 1: rejected, and drawn from p."""
    s = make([2] * 20, 2, 10000, F, True, 8, near=0.0, temperature=1.0)
    s["u"].fill_(1.0)
    out, accepted = check(s)
    assert (accepted == 0).all() and (out[:, 0] >= 0).all()


def test_tokens_outside_the_vocabulary(require_gpu):
    for drawn in (True, False):
        s = make([3] * 12, 3, 700, F, drawn, 9)
        s["tokens"][::5] = torch.tensor([-1, 700, -2 ** 31, 2 ** 31 - 1, -100, 701, 5000, -1],
                                        dtype=torch.int32, device="cuda")
        check(s)


@pytest.mark.parametrize("t", [0.0, -1.0, float("nan"), float("inf"), 1e-30, 1e-45, 1e30, 3e38])
def test_temperatures(require_gpu, t):
    for dtype in (F, H16):
        s = make([3] * 20, 3, 9001, dtype, True, 10, temperature=t)
        s["target"][:, 3:50] = -float("inf")
        check(s)


def test_ties_go_to_the_lowest_index(require_gpu):
    s = make([2] * 20, 2, 30000, H16, False, 11, temperature=0.0)
    s["target"].clamp_(max=4.0)
    check(s)


def test_offsets_that_do_not_fit(require_gpu):
    """Nothing is read out of range (the rows are the whole of their tensors), and
    sequences whose own offsets are right are not touched by the others'."""
    s = make([3, 3, 3, 3], 3, 640, F, True, 12, extra=0)
    want = run(s)
    s["off"] = torch.tensor([0, 3, -5, 2 ** 31 - 1, 12], dtype=torch.int32, device="cuda")
    got = run(s)
    assert np.array_equal(got[0][0], want[0][0]) and got[1][0] == want[1][0]
    s["off"] = torch.tensor([2 ** 31 - 1, -2 ** 31, 9, 4, 12], dtype=torch.int32, device="cuda")
    out, accepted = run(s)
    assert ((accepted >= 0) & (accepted <= 3)).all() and ((out >= -1) & (out < 640)).all()


def test_alone_as_in_a_batch(require_gpu):
    s = make([4, 0, 2, 4, 1], 4, 20001, F, True, 13)
    out, accepted = run(s)
    at = 0
    for i, n in enumerate(s["counts"]):
        one = dict(s, counts=[n], target=s["target"][at + i:at + i + n + 1], draft=s["draft"][at:at + n],
                   tokens=s["tokens"][at:at + n], u=s["u"][at:at + n], u_next=s["u_next"][i:i + 1],
                   off=torch.tensor([0, n], dtype=torch.int32, device="cuda"), temperature=s["temperature"][i:i + 1])
        o, a = run(one)
        assert np.array_equal(o[0], out[i]) and a[0] == accepted[i]
        at += n


def test_tokens_follow_the_target(require_gpu):
    """Drafts drawn from q and verified: the first token's frequencies are p's, within
    five standard deviations."""
    N, V = 40000, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    z, y = torch.randn(8, device="cuda", generator=g), torch.randn(8, device="cuda", generator=g)
    p = torch.softmax(z[:V].double(), 0)
    for drawn in (True, False):
        noise = -(-torch.rand(N, V, device="cuda", generator=g).log()).log()
        x = (y[:V] + noise).argmax(1) if drawn else torch.full((N,), 2, device="cuda")
        s = dict(counts=[1] * N, K=1, target=z.expand(2 * N, 8).contiguous()[:, :V],
                 draft=y.expand(N, 8).contiguous()[:, :V] if drawn else None, tokens=x.to(torch.int32),
                 off=torch.arange(N + 1, dtype=torch.int32, device="cuda"), temperature=None,
                 u=torch.rand(N, device="cuda", generator=g), u_next=torch.rand(N, device="cuda", generator=g))
        share = np.bincount(run(s)[0][:, 0], minlength=V) / N
        pn = p.cpu().numpy()
        assert (np.abs(share - pn) <= 5 * np.sqrt(pn * (1 - pn) / N)).all(), (share, pn)


def test_refusals_of_the_binding(require_gpu):
    s = make([2, 2], 2, 64)
    u, un, off, tok = s["u"], s["u_next"], s["off"], s["tokens"]
    out = torch.empty(2, 3, dtype=torch.int32, device="cuda")
    acc = torch.empty(2, dtype=torch.int32, device="cuda")

    def call(target=s["target"], tokens=tok, offsets=off, K=2, draft=s["draft"], t=None, u=u, un=un, out=out, acc=acc, ws=None):
        return lambda: sb.sb_verify_drafts(sb.Drafts(target, tokens, offsets, K, draft, t), u, un, out, acc, ws=ws)

    for f, error in (
            (call(target=s["target"].half()), TypeError), (call(target=s["target"][:5]), ValueError),
            (call(target=s["target"].t()), ValueError), (call(tokens=tok.long()), TypeError),
            (call(tokens=tok[::2]), ValueError), (call(offsets=off.long()), TypeError), (call(offsets=off[:0]), ValueError),
            (call(draft=s["draft"].bfloat16()), TypeError), (call(draft=s["draft"][:3]), ValueError),
            (call(t=un.double()), TypeError), (call(t=un[:1]), ValueError), (call(u=u[:3]), ValueError),
            (call(u=None), sb.SbError), (call(un=un[:1]), ValueError), (call(out=out[:, :2]), ValueError),
            (call(out=out.long()), TypeError), (call(out=out[:1].expand(2, 3)), sb.SbError), (call(acc=acc[:1]), ValueError),
            (call(K=-1), sb.SbError), (call(acc=acc.cpu()), ValueError),
            (call(ws=torch.empty(16, dtype=torch.uint8, device="cuda")), sb.SbError)):
        with pytest.raises(error):
            f()


@pytest.mark.parametrize("dtype", [F, H16])
@pytest.mark.parametrize("V", [1500, 40965, 151936])
@pytest.mark.parametrize("u", [1.0, 1.0 + 2.0 ** -23, 7.0, float("inf")])
def test_numbers_from_one_up_draw_the_last_token(require_gpu, u, V, dtype):
    """The last columns have shares of about e^-60 of the whole, which no sum of it
    shows: still the last of them that can be drawn is, not the one where a
    cumulative sum first reaches the whole."""
    N = 48
    for how in ("row", "without", "less"):
        n = 0 if how == "row" else 1
        s = make([n] * N, n, V, dtype, how == "less", 61, near=0.5, temperature=None)
        s["u"].fill_(float("nan"))  # accepts no draft
        s["u_next"].fill_(u)
        s["target"][:, -300:] -= 60
        last = V - 1
        if n:
            s["tokens"].fill_(0)
        if how == "less":
            # q is below p in the tail by e^-19 or less, but for its last two columns
            s["draft"][:, -300:] = s["target"][::2, -300:] - 20
            s["draft"][:, -2:] += 40
            last = V - 3
        out, accepted = run(s)
        off = np.nonzero(out[:, 0] != last)[0]
        assert not len(off) and not accepted.any(), (how, off, out[off, 0])


@pytest.mark.parametrize("dtype", [F, H16])
@pytest.mark.parametrize("t", [None, 0.7, 1e-12])
def test_shares_of_equal_logits_are_exact(require_gpu, t, dtype):
    """2^k equal logits and nothing else have shares of 2^-k exactly, whatever the logits
    are: u q < p is false where both sides are equal, and true where u is the next lower
    number."""
    N, V = 240, 20000
    z = torch.linspace(-40, 40, N, device="cuda").to(dtype)
    g = torch.Generator(device="cuda").manual_seed(3)
    for k, kq in ((0, None), (1, None), (2, None), (5, None), (9, None), (3, 1), (6, 2)):
        s = make([1] * N, 1, V, dtype, kq is not None, 71, temperature=t)
        s["target"].fill_(-float("inf"))
        # (from chunk to chunk, the drafted token among them)
        at = torch.randperm(V, device="cuda", generator=g)[:2 ** k]
        s["target"][::2, at] = z[:, None]
        s["target"][1::2, 0] = 0
        s["tokens"].fill_(int(at[0]))
        border = 2.0 ** -k
        if kq is not None:
            s["draft"].fill_(-float("inf"))
            s["draft"][:, at[:2 ** kq]] = -z[:, None]
            border = 2.0 ** (kq - k)
        for u, want in ((border, 0), (float(np.nextafter(np.float32(border), np.float32(0))), 1)):
            s["u"].fill_(u)
            accepted = run(s)[1]
            assert (accepted == want).all(), (k, kq, u, np.nonzero(accepted != want)[0])


@pytest.mark.parametrize("z", [-17.3, 0.1, 1e6])
def test_borders_of_a_flat_row_of_any_logit(require_gpu, z):
    """Shares of 2^-14 exactly: a multiple k / V of the whole draws token k, the number
    below it the one before."""
    N, V = 512, 16384
    s = make([0] * N, 0, V, F, False, 1, 0.0, 0.0, None)
    s["target"].fill_(z)
    k = torch.linspace(0, V - 1, N, device="cuda").round()
    for u, token in ((k / V, k), (torch.nextafter(k / V, torch.tensor(-1.0, device="cuda")), (k - 1).clamp(min=0))):
        s["u_next"] = u
        assert np.array_equal(run(s)[0][:, 0], token.long().cpu().numpy())
