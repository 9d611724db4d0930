"""Preference and policy losses with their gradients against the formulas in 64
bits.  Tolerances, with e = 2^-24 and u = 2^-53: sums are 64-bit (n u of the sum
of magnitudes, below 2^-30 of it here) and outputs rounded once, e.  A policy's
token terms are fp32: r = exp(x) is off by (|x| + 4) e, r A by 2 e more; the KL
estimate by 16 e of itself, |k| e times its slope for k's rounding and, past |k| =
1, 4 e of exp(k) - 1; the weighted sum and kl's rounding 3 e."""
import ctypes
import math

import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b

E = 2.0 ** -24
F = torch.float32
NAN, INF = float("nan"), float("inf")
gpu = pytest.mark.gpu


def close(got, ref, tol, what):
    got = got.double().cpu()
    ref, tol = torch.as_tensor(ref).double(), torch.as_tensor(tol).double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    bad = ~((got - ref).abs() <= tol + 1e-38) & ~torch.isnan(ref) & (got != ref)
    if bad.any():
        i = bad.nonzero()[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {i}: "
                             f"got {got[tuple(i)]} ref {ref[tuple(i)]} tol {tol[tuple(i)]}")


def batch(S, T, seed=0, outside=False, empty=False):
    """Inputs on the GPU; outside: tokens before the first sequence and after the last."""
    g = torch.Generator().manual_seed(seed)
    lo, hi = (T // 8, T - T // 5) if outside else (0, T)
    cuts = torch.randint(lo, hi + 1, (max(S - 1, 0),), generator=g).sort().values
    if empty and S > 3:
        cuts[1] = cuts[0]
    starts = torch.cat([torch.tensor([lo]), cuts, torch.tensor([hi])])[:S + 1].int()
    lp = -torch.rand(T, generator=g) * 3
    d = dict(starts=starts, logps=lp, ref=lp + torch.randn(T, generator=g) * 0.5,
             old=lp + torch.randn(T, generator=g) * 0.3,
             mask=torch.rand(T, generator=g) < 0.7)
    d["adv_s"], d["adv_t"] = torch.randn(S, generator=g), torch.randn(T, generator=g)
    return {k: v.cuda() for k, v in d.items()}


def runs(starts):
    s = starts.tolist()
    return list(zip(s[:-1], s[1:]))


def preference(d, beta, eps, form, average, ref, mask, up=1.0):
    """(loss, rewards, gradient, magnitude of the sums) in 64 bits."""
    lp = d["logps"].double().cpu()
    x = lp - d["ref"].double().cpu() if ref else lp
    m = d["mask"].cpu() if mask else torch.ones_like(lp, dtype=torch.bool)
    r, S = runs(d["starts"]), d["starts"].numel() - 1
    g, rewards, loss, size = torch.zeros_like(lp), [], 0.0, 0.0
    n = [max(1, int(m[a:c].sum())) if average else 1 for a, c in r]
    sums = [float(x[a:c][m[a:c]].sum()) / k for (a, c), k in zip(r, n)]
    for p in range(S // 2):
        h = sums[2 * p] - sums[2 * p + 1]
        z = beta * h
        if form == "sigmoid":
            up_ = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
            f = (1 - eps) * up_(-z) + (eps * up_(z) if eps else 0.0)
            s = 1 / (1 + math.exp(-z)) if z > -700 else 0.0
            t = 1 / (1 + math.exp(z)) if z < 700 else 0.0
            dh = beta * (eps * s - (1 - eps) * t)
        elif form == "hinge":
            f, dh = max(0.0, 1 - z), -beta if z < 1 else 0.0
        else:
            f, dh = (h - 0.5 / beta) ** 2, 2 * (h - 0.5 / beta)
        loss += f
        rewards.append([beta * sums[2 * p], beta * sums[2 * p + 1]])
        for q, sign in ((2 * p, 1), (2 * p + 1, -1)):
            a, c = r[q]
            g[a:c] = torch.where(m[a:c], sign * dh / n[q] * 2 / S * up, 0.0)
            size = max(size, float(x[a:c].abs().sum()))
    return loss * 2 / max(S, 1), torch.tensor(rewards, dtype=torch.float64).view(-1, 2), g, size


BATCHES = [(2, 0), (2, 1), (2, 7), (4, 64), (6, 1000), (16, 4097), (256, 8192), (258, 8192),
           (20, 8193), (2, 30000), (514, 100003), (3000, 9000), (9000, 30011)]


@gpu
@pytest.mark.parametrize("form,eps,average", [("sigmoid", 0.0, False), ("sigmoid", 0.2, True),
                                              ("hinge", 0.0, False), ("squared", 0.0, True)])
@pytest.mark.parametrize("S,T", BATCHES)
def test_preference(S, T, form, eps, average):
    beta = 0.3
    for k, (ref, mask) in enumerate(((True, True), (False, False), (True, False))):
        d = batch(S, T, S + T + k, outside=k == 1, empty=k == 0)
        loss, rewards, g, size = preference(d, beta, eps, form, average, ref, mask, -2.5)
        args = dict(ref=d["ref"] if ref else None, mask=d["mask"] if mask else None, beta=beta,
                    smoothing=eps, form=form, average=average)
        got = snk.preference_grads(d["logps"], d["starts"], **args,
                                   dloss=torch.tensor(-2.5, device="cuda"))
        off = 2.0 ** -30 * (1 + size)  # of d's sums
        slope = beta if form != "squared" else 2 * (size + 1 / beta)
        close(got[0], loss, 1.01 * E * abs(loss) + slope * 2 * off, "loss")
        close(got[1], rewards, 1.01 * E * rewards.abs() + beta * off, "rewards")
        close(got[2], g, 1.01 * E * g.abs() + 2.5 * 4 * off / max(S // 2, 1), "gradient")
        alone = snk.preference_grads(d["logps"], d["starts"], **args, want=(True, False))
        assert alone[2] is None and torch.equal(alone[0], got[0]) and torch.equal(alone[1], got[1])
        only = snk.preference_grads(d["logps"], d["starts"], **args, want=(False, True),
                                    dloss=torch.tensor(-2.5, device="cuda"))
        assert only[0] is None and only[1] is None and torch.equal(only[2], got[2])


def policy(d, low, high, kl, average, by, old, ref, mask, up=1.0):
    """(loss, stats, gradient) and their tolerances in 64 bits."""
    lp = d["logps"].double().cpu()
    T, S = lp.numel(), d["starts"].numel() - 1
    w, a = torch.zeros(T, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    inside = torch.zeros(T, dtype=torch.bool)
    m = d["mask"].cpu() if mask else torch.ones(T, dtype=torch.bool)
    for i, (x, y) in enumerate(runs(d["starts"])):
        inside[x:y] = m[x:y]
        w[x:y] = 1 / (S * max(1, int(m[x:y].sum())))
        a[x:y] = float(d["adv_s"][i])
    n = max(1, int(inside.sum()))
    if average == "tokens":
        w[:] = 1 / n
    if by == "tokens":
        a = d["adv_t"].double().cpu()
    w = torch.where(inside, w, 0.0)
    move = lp - d["old"].double().cpu() if old else torch.zeros_like(lp)
    r = move.exp()
    held = r.clamp(1 - low, 1 + high)
    cut = ((a > 0) & (move > math.log1p(high))) | ((a < 0) & (move < math.log1p(-low)
                                                              if low < 1 else False))
    f = -torch.minimum(r * a, held * a)
    df = torch.where(cut, 0.0, -r * a)
    tf = (move.abs() + 6) * E * (held * a).abs().maximum((r * a).abs())
    tdf = (move.abs() + 6) * E * df.abs()
    k3 = torch.zeros_like(lp)
    if ref:
        k = d["ref"].double().cpu() - lp
        em1 = torch.expm1(k)
        k3 = em1 - k
        tk = 16 * E * k3 + E * k.abs() * em1.abs() + torch.where(k.abs() < 1, 0.0, 4 * E * em1.abs())
        f, df = f + kl * k3, df - kl * em1
        tf, tdf = tf + kl * tk + E * kl * k3, tdf + kl * (tk + E * k.abs() + 6 * E * em1.abs())
        ts = (tk * inside).sum() / n
    else:
        ts = 0.0
    f, df, k3 = (torch.where(inside, v, 0.0) for v in (f, df, k3))
    loss = float((f * w).sum())
    stats = torch.stack([(k3 * inside).sum() / n, (cut & inside).double().sum() / n])
    tl = float((torch.where(inside, tf + 3 * E * f.abs(), 0.0) * w).sum()) + 2 * E * abs(loss) + 1e-12
    g = df * w * up
    tg = (torch.where(inside, tdf, 0.0) * w * abs(up)) + 3 * E * g.abs()
    return loss, stats, g, tl, torch.stack([torch.as_tensor(ts + 0.0).double(), torch.zeros(()).double()]) + 2 * E * stats, tg


@gpu
@pytest.mark.parametrize("average", ["tokens", "sequences"])
@pytest.mark.parametrize("by", ["tokens", "sequences"])
@pytest.mark.parametrize("S,T", [(1, 1), (3, 5)] + BATCHES)
def test_policy(S, T, by, average):
    for k, (old, ref, mask) in enumerate(((True, True, True), (True, False, False),
                                          (False, True, False), (True, True, False))):
        d = batch(S, T, S + T + k, outside=k == 1, empty=k == 0)
        adv = d["adv_t"] if by == "tokens" else d["adv_s"]
        adv[::5] = 0
        want = policy(d, 0.2, 0.3, 0.05, average, by, old, ref, mask, 1.5)
        args = (d["logps"], d["old"] if old else None, adv, d["starts"])
        more = dict(ref=d["ref"] if ref else None, mask=d["mask"] if mask else None,
                    clip=(0.2, 0.3), kl=0.05, average=average, by=by)
        up = torch.tensor(1.5, device="cuda")
        loss, stats, g = snk.policy_grads(*args, **more, dloss=up)
        close(loss, want[0], want[3], "loss")
        close(stats, want[1], want[4], "stats")
        close(g, want[2], want[5], "gradient")
        again = snk.policy_grads(*args, **more, want=(True, False))
        assert again[2] is None and torch.equal(again[0], loss) and torch.equal(again[1], stats)
        only = snk.policy_grads(*args, **more, dloss=up, want=(False, True))
        assert only[0] is None and only[1] is None and torch.equal(only[2], g)


@gpu
@pytest.mark.parametrize("S,T", [(4, 40), (400, 40000)])
def test_rows_of_a_matrix(S, T):
    d = batch(S, T, 3)
    lp, starts = d["logps"].view(S, -1), torch.arange(0, T + 1, T // S, dtype=torch.int32).cuda()
    a = snk.preference_grads(lp, ref=d["ref"].view(S, -1), mask=d["mask"].view(S, -1))
    c = snk.preference_grads(d["logps"], starts, ref=d["ref"], mask=d["mask"])
    assert torch.equal(a[0], c[0]) and torch.equal(a[2], c[2].view(S, -1))
    u8 = snk.preference_grads(lp, ref=d["ref"].view(S, -1), mask=d["mask"].view(S, -1).byte())
    assert torch.equal(u8[2], a[2])
    a = snk.policy_grads(lp, d["old"].view(S, -1), d["adv_s"], mask=d["mask"].view(S, -1))
    c = snk.policy_grads(d["logps"], d["old"], d["adv_s"], starts, mask=d["mask"])
    assert torch.equal(a[0], c[0]) and torch.equal(a[2], c[2].view(S, -1))
    one = snk.policy_grads(d["logps"], d["old"], d["adv_s"][:1])  # a vector: one sequence
    two = snk.policy_grads(d["logps"], d["old"], d["adv_s"][:1],
                           torch.tensor([0, T], dtype=torch.int32, device="cuda"))
    assert torch.equal(one[2], two[2])
    t = lp.t().contiguous().t()  # another order in memory
    assert torch.equal(snk.policy_grads(t, d["old"].view(S, -1), d["adv_s"])[2],
                       snk.policy_grads(lp, d["old"].view(S, -1), d["adv_s"])[2])


@gpu
@pytest.mark.parametrize("S,T", [(8, 400), (8, 30000)])
def test_masked_tokens_hold_anything(S, T):
    d = batch(S, T, 6)
    args = dict(ref=d["ref"], mask=d["mask"])
    want = snk.preference_grads(d["logps"], d["starts"], **args)
    pol = snk.policy_grads(d["logps"], d["old"], d["adv_t"], d["starts"], by="tokens", kl=0.1,
                           average="sequences", **args)
    for k, v in enumerate((NAN, INF, -INF)):
        for name in ("logps", "ref", "old", "adv_t"):
            d[name][~d["mask"]] = v
        for a, c in zip(want, snk.preference_grads(d["logps"], d["starts"], **args)):
            assert torch.equal(a, c)
        for a, c in zip(pol, snk.policy_grads(d["logps"], d["old"], d["adv_t"], d["starts"],
                                              by="tokens", kl=0.1, average="sequences", **args)):
            assert torch.equal(a, c)
    none = torch.zeros_like(d["mask"])
    loss, stats, g = snk.policy_grads(d["logps"], d["old"], d["adv_s"], d["starts"], mask=none)
    assert float(loss) == 0 and (stats == 0).all() and (g == 0).all()
    loss, rewards, g = snk.preference_grads(d["logps"], d["starts"], mask=none, average=True)
    assert abs(float(loss) - math.log(2)) <= E and (rewards == 0).all() and (g == 0).all()


@gpu
@pytest.mark.parametrize("pad", [0, 9000])
def test_values_by_the_formula(pad):
    """Infinities and borders; pad: the same on the path of large batches."""
    def seqs(*values):
        lp = torch.zeros(len(values) + pad, device="cuda")
        lp[:len(values)] = torch.tensor(values)
        starts = list(range(len(values))) + [len(values) + pad]
        return lp, torch.tensor(starts, dtype=torch.int32, device="cuda")
    lp, st = seqs(-INF, 0.0)
    loss, _, g = snk.preference_grads(lp, st, beta=1.0)
    assert float(loss) == INF and float(g[0]) == -1.0
    lp, st = seqs(0.0, -INF)
    loss, _, g = snk.preference_grads(lp, st, beta=1.0)
    assert float(loss) == 0.0 and float(g[0]) == 0.0
    assert float(snk.preference_grads(lp, st, beta=1.0, smoothing=0.5)[0]) == INF
    assert float(snk.preference_grads(lp, st, beta=1.0, form="hinge")[0]) == 0.0
    lp, st = seqs(-INF, -INF)
    for form in ("sigmoid", "hinge", "squared"):
        loss, _, g = snk.preference_grads(lp, st, form=form)
        assert math.isnan(float(loss)) and math.isnan(float(g[0]))
    lp, st = seqs(1000.0, -1000.0)
    loss, _, g = snk.preference_grads(-lp, st, beta=1.0)
    assert float(loss) == 2000.0 and float(g[1]) == 1.0
    # exactly on a border: the ratio is 1, and the clip of 0 does not decide
    lp, st = seqs(-1.0, -1.0)
    adv = torch.tensor([1.0, -1.0], device="cuda")
    loss, stats, g = snk.policy_grads(lp, lp, adv, st, clip=(0.0, 0.0), average="sequences")
    assert float(stats[1]) == 0.0 and float(g[0]) == -0.5
    # a ratio past every float is clipped where that is the smaller, and only there
    old = lp - 200.0
    _, _, g = snk.policy_grads(lp, old, adv, st, average="sequences")
    assert float(g[0]) == 0.0 and float(g[-1]) == INF
    _, _, g = snk.policy_grads(lp, lp + 200.0, adv, st, clip=(1.0, 0.2), average="sequences")
    assert float(g[0]) <= 0.0 and abs(float(g[0])) < 1e-38


@gpu
def test_gradients_are_the_differences():
    S, T, h = 6, 60, 1e-4
    d = batch(S, T, 9)
    g = torch.Generator().manual_seed(2)
    v = torch.randn(T, generator=g).double().cuda()

    def moved(s):
        e = dict(d)
        e["logps"] = d["logps"].double() + s * h * v
        return e

    for form in ("sigmoid", "squared"):
        up, down = (preference(moved(s), 0.3, 0.0, form, False, True, True)[0] for s in (1, -1))
        got = snk.preference_grads(d["logps"], d["starts"], ref=d["ref"], mask=d["mask"], beta=0.3,
                                   form=form)[2]
        got = float((got.double() * v).sum())
        assert abs(got - (up - down) / (2 * h)) <= 1e-5 * (1 + abs(got))
    up, down = (policy(moved(s), 0.9, 9.0, 0.1, "tokens", "sequences", True, True, True)[0]
                for s in (1, -1))
    got = snk.policy_grads(d["logps"], d["old"], d["adv_s"], d["starts"], ref=d["ref"],
                           mask=d["mask"], clip=(0.9, 9.0), kl=0.1)[2]
    got = float((got.double() * v).sum())
    # third derivatives times h^2 / 6 and the roundings of 60 terms
    assert abs(got - (up - down) / (2 * h)) <= 1e-5 * (1 + abs(got))


@gpu
def test_autograd():
    d = batch(8, 500, 12)
    lp = d["logps"].clone().requires_grad_(True)
    loss, rewards = snk.preference_loss(lp, d["starts"], d["ref"], d["mask"], beta=0.2)
    assert not rewards.requires_grad and loss.shape == () and rewards.shape == (4, 2)
    (3 * loss).backward()
    three = torch.tensor(3.0, device="cuda")
    assert torch.equal(lp.grad, snk.preference_grads(d["logps"], d["starts"], d["ref"], d["mask"],
                                                     0.2, dloss=three)[2])
    lp.grad = None
    loss, stats = snk.policy_loss(lp, d["old"], d["adv_s"], d["starts"], d["ref"], d["mask"],
                                  kl=0.1)
    assert not stats.requires_grad
    (3 * loss).backward()
    assert torch.equal(lp.grad, snk.policy_grads(d["logps"], d["old"], d["adv_s"], d["starts"],
                                                 d["ref"], d["mask"], kl=0.1, dloss=three)[2])
    with torch.no_grad():
        assert torch.equal(snk.policy_loss(lp, d["old"], d["adv_s"], d["starts"])[0],
                           snk.policy_grads(d["logps"], d["old"], d["adv_s"], d["starts"])[0])


@gpu
@pytest.mark.parametrize("S,T", [(8, 300), (40, 20000)])
def test_streams_graphs_and_the_binding(S, T):
    d = batch(S, T, 13)

    def both():
        return [*snk.preference_grads(d["logps"], d["starts"], d["ref"], d["mask"]),
                *snk.policy_grads(d["logps"], d["old"], d["adv_s"], d["starts"], d["ref"],
                                  d["mask"], kl=0.1)]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = both()
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, other))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    for gr in graphs:
        with torch.cuda.graph(gr):
            outs.append(both())
    for k in range(3):
        d["logps"].copy_(-torch.rand(T, device="cuda"))
        d["mask"].copy_(torch.rand(T, device="cuda") < 0.5)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        want = both()
        for o in outs:
            assert all(torch.equal(a, c) for a, c in zip(want, o)), k
    q = snk.snack_seqs(S, T, d["starts"], d["mask"])
    ws = torch.empty(max(1, snk.snack_seqs_workspace(S, T)), dtype=torch.uint8, device="cuda")
    got = [torch.empty_like(w) for w in want]
    snk.snack_preference(q, b.SnackPref(0.1, 0.0, b.PREF_SIGMOID, 0), d["logps"], d["ref"], None,
                         *got[:3], ws)
    snk.snack_policy_loss(q, b.SnackPolicy(0.2, 0.2, 0.1, 0, 0), d["logps"], d["old"], d["ref"],
                          d["adv_s"], None, *got[3:], ws)
    assert all(torch.equal(a, c) for a, c in zip(want, got))


@gpu
@pytest.mark.parametrize("T", [100, 20000])
def test_starts_that_do_not_fit_stay_inside(T):
    """Not a promise of values: places past the tokens are cut to them."""
    lp = -torch.rand(T, device="cuda")
    for starts in ([-5, T + 1000, 2 ** 31 - 1], [T, 3, -2 ** 31], [2 ** 30, 5, T]):
        st = torch.tensor(starts, dtype=torch.int32, device="cuda")
        loss, rewards, g = snk.preference_grads(lp, st)
        assert g.shape == (T,) and rewards.shape == (1, 2)
        snk.policy_grads(lp, lp, torch.ones(2, device="cuda"), st)
    torch.cuda.synchronize()


SEQS = dict(S=4, T=40, starts=0x1000, mask=0x2000)
PREF = dict(beta=0.1, smoothing=0.0, form=0, average=0)
POLICY = dict(low=0.2, high=0.2, kl=0.1, by_token=0, sequence_mean=0)
PTRS = dict(logps=0x10000, ref=0x11000, dloss=0x12000, loss=0x13000, rewards=0x14000,
            dlogps=0x15000, ws=0x100000, ws_bytes=1 << 20)
POLICY_PTRS = dict(logps=0x10000, old=0x16000, ref=0x11000, adv=0x17000, dloss=0x12000,
                   loss=0x13000, stats=0x14000, dlogps=0x15000, ws=0x100000, ws_bytes=1 << 20)
BAD_SEQS = [(dict(S=-1), -2), (dict(T=-1), -2), (dict(S=(1 << 24) + 2), -10),
            (dict(T=(1 << 30) + 1), -10), (dict(starts=None, T=41), -2),
            (dict(starts=None, S=0), -2)]
BAD_PTRS = [(dict(logps=None), -1), (dict(dlogps=0x10000), -2), (dict(dlogps=0x11008), -2),
            (dict(loss=0x12000), -2), (dict(loss=0x15010), -2), (dict(dlogps=0x1000), -2),
            (dict(dlogps=0x2004), -2)]
LARGE = dict(T=100000, mask=None)
FAR = dict(logps=1 << 32, ref=1 << 33, old=1 << 34, adv=1 << 35, dlogps=1 << 36)


@pytest.mark.parametrize("seqs,ptrs,cfg,status",
                         [(s, {}, {}, st) for s, st in BAD_SEQS]
                         + [({}, p, {}, st) for p, st in BAD_PTRS]
                         + [(dict(S=3), {}, {}, -2), ({}, dict(rewards=0x13000), {}, -2),
                            (LARGE, dict(FAR, ws=None), {}, -1),
                            (LARGE, dict(FAR, ws_bytes=8), {}, -9),
                            (LARGE, dict(FAR, ws=(1 << 36) + 64), {}, -2)]
                         + [({}, {}, c, st) for c, st in (
                             (dict(beta=0.0), -2), (dict(beta=-1.0), -2), (dict(beta=INF), -2),
                             (dict(beta=NAN), -7), (dict(smoothing=NAN), -7),
                             (dict(smoothing=-0.1), -2), (dict(smoothing=1.1), -2),
                             (dict(form=3), -2), (dict(form=-1), -2),
                             (dict(form=1, smoothing=0.1), -2))])
def test_refusals_of_preferences(seqs, ptrs, cfg, status):
    q = b.SnackSeqs(*dict(SEQS, **seqs).values())
    c = b.SnackPref(*dict(PREF, **cfg).values())
    p = {k: v for k, v in dict(PTRS, **ptrs).items() if k in PTRS}
    assert b.raw_status("snack_preference", ctypes.byref(q), ctypes.byref(c), *p.values(),
                        None) == status


@pytest.mark.parametrize("seqs,ptrs,cfg,status",
                         [(s, {}, {}, st) for s, st in BAD_SEQS]
                         + [({}, p, {}, st) for p, st in BAD_PTRS]
                         + [({}, dict(adv=None), {}, -1), ({}, dict(stats=0x13000), {}, -2),
                            ({}, dict(dlogps=0x16000), {}, -2), ({}, dict(dlogps=0x17000), {}, -2),
                            (LARGE, dict(FAR, ws=None), {}, -1),
                            (LARGE, dict(FAR, ws_bytes=8), {}, -9)]
                         + [({}, {}, c, st) for c, st in (
                             (dict(low=-0.1), -2), (dict(low=1.1), -2), (dict(low=NAN), -7),
                             (dict(high=-0.1), -2), (dict(high=NAN), -7), (dict(kl=-1.0), -2),
                             (dict(kl=NAN), -7))])
def test_refusals_of_policies(seqs, ptrs, cfg, status):
    q = b.SnackSeqs(*dict(SEQS, **seqs).values())
    c = b.SnackPolicy(*dict(POLICY, **cfg).values())
    p = dict(POLICY_PTRS, **ptrs)
    assert b.raw_status("snack_policy_loss", ctypes.byref(q), ctypes.byref(c), *p.values(),
                        None) == status


def test_missing_structs():
    q, c, p = b.SnackSeqs(0, 0), b.SnackPref(0.1, 0, 0, 0), b.SnackPolicy(0.2, 0.2, 0, 0, 0)
    none = [None] * 6
    assert b.raw_status("snack_preference", None, ctypes.byref(c), *none, None, 0, None) == -1
    assert b.raw_status("snack_preference", ctypes.byref(q), None, *none, None, 0, None) == -1
    assert b.raw_status("snack_policy_loss", None, ctypes.byref(p), *none, None, None, None, 0,
                        None) == -1
    assert b.raw_status("snack_policy_loss", ctypes.byref(q), None, *none, None, None, None, 0,
                        None) == -1
    assert b.raw_status("snack_seqs_workspace", 1, 1, None) == -1
    assert b.raw_status("snack_seqs_workspace", -1, 1, ctypes.byref(ctypes.c_size_t())) == -2


def test_wrappers_refuse_what_does_not_fit():
    with pytest.raises(TypeError, match="on the GPU"):
        snk.preference_grads(torch.zeros(4))
    with pytest.raises(ValueError, match="form"):
        snk.preference_loss(torch.zeros(4), form="other")
    with pytest.raises(ValueError, match="average"):
        snk.policy_loss(torch.zeros(4), None, torch.zeros(1), average="other")
    with pytest.raises(ValueError, match="by"):
        snk.policy_grads(torch.zeros(4), None, torch.zeros(1), by="other")


@gpu
def test_wrappers_refuse_on_the_gpu():
    c = dict(device="cuda")
    lp, adv = torch.zeros(4, 6, **c), torch.zeros(4, **c)
    st = torch.tensor([0, 12, 24], dtype=torch.int32, **c)
    for kind, call in [
            (TypeError, lambda: snk.preference_grads(lp.double())),
            (ValueError, lambda: snk.preference_grads(lp, st.long())),
            (ValueError, lambda: snk.preference_grads(lp, st.cpu())),
            (ValueError, lambda: snk.preference_grads(lp[None])),
            (ValueError, lambda: snk.preference_grads(lp, ref=lp[:2])),
            (TypeError, lambda: snk.preference_grads(lp, ref=lp.half())),
            (ValueError, lambda: snk.preference_grads(lp, mask=lp)),
            (ValueError, lambda: snk.preference_grads(lp, mask=lp[0] > 0)),
            (TypeError, lambda: snk.preference_grads(lp, dloss=torch.zeros(2, **c))),
            (snk.SnackError, lambda: snk.preference_grads(lp[:3])),
            (snk.SnackError, lambda: snk.preference_grads(lp, beta=0.0)),
            (ValueError, lambda: snk.policy_grads(lp, lp, adv[:3])),
            (ValueError, lambda: snk.policy_grads(lp, lp, adv, by="tokens")),
            (TypeError, lambda: snk.policy_grads(lp, lp, adv.double())),
            (ValueError, lambda: snk.policy_grads(lp, lp[0], adv)),
            (snk.SnackError, lambda: snk.policy_grads(lp, lp, adv, clip=(-1.0, 0.2)))]:
        with pytest.raises(kind):
            call()
