"""Workloads of the two ends of a fine-tuning step, from token numbers to the
first layer and from logits to a loss, for timing and for comparing the
library's kernels with a plain form of the same formulas.

Kinds of case:
  drop    dropout by a counter-based generator, on a sum or not, and its gradient
  embed   rows of a table looked up by token, and the table's gradient
  logp    log-probabilities of target tokens from logits, and the logits' gradient
  pref    a loss over pairs of sequences by their log ratios, with its gradient
  policy  a clipped policy loss with a KL term, with its gradient

``own`` selects the library's kernels (True) or the plain form (False).
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SEED = 20 ** 14  # of the dropout's generator


def listed():
    return [
        # the gradient through the dropout before the adapters of a small fp32 model
        dict(name="drop_grad_odd", kind="drop", T=515, K=1001, p=0.1, step=7, residual=False,
             back=True, strided=False, dtype="f32"),
        # the dropout at the end of a block of a training step, added to the block's input
        dict(name="drop_residual", kind="drop", T=8192, K=4096, p=0.1, step=123456, residual=True,
             back=False, strided=False, dtype="bf16"),
        # a decode step of 37 requests
        dict(name="embed_decode", kind="embed", back=False, T=37, V=32000, D=4096, ids="mixed",
             base=False, wide=True, dtype="bf16"),
        # the table's gradient of a training step of a small model
        dict(name="embed_grad", kind="embed", back=True, T=8192, V=50000, D=768, ids="text",
             base=False, wide=True, dtype="bf16"),
        # the same where the table is the head's weight too, whose gradient is there already
        dict(name="embed_grad_tied", kind="embed", back=True, T=20001, V=32001, D=1000, ids="text",
             base=True, wide=False, dtype="f32"),
        # log-probabilities of a few drafted tokens, a wide vocabulary
        dict(name="logp_few", kind="logp", back=False, T=5, V=128000, ignored=0.0, wide=True,
             dtype="bf16"),
        # all tokens of a training step
        dict(name="logp_8192", kind="logp", back=False, T=8192, V=32000, ignored=0.0, wide=True,
             dtype="bf16"),
        # the logits' gradient of answers after prompts, an odd vocabulary
        dict(name="logp_grad", kind="logp", back=True, T=4099, V=50001, ignored=0.3, wide=True,
             dtype="bf16"),
        # eight pairs of short answers on one GPU
        dict(name="pref_8", kind="pref", S=16, T=1500, form="sigmoid", smoothing=0.0, beta=0.1,
             average=False, ref=True, mask=False),
        # a large batch of long answers, prompts masked
        dict(name="pref_2048", kind="pref", S=4096, T=4000000, form="sigmoid", smoothing=0.1,
             beta=0.1, average=False, ref=True, mask=True),
        # answers to a few prompts, one mean over all tokens
        dict(name="policy_64", kind="policy", S=64, T=12345, kl=0.04, low=0.2, high=0.2,
             average="tokens", by="sequences", ref=True, mask=True),
        # a large batch of long answers, a mean for each sequence
        dict(name="policy_1024", kind="policy", S=1024, T=2000003, kl=0.04, low=0.2, high=0.28,
             average="sequences", by="tokens", ref=True, mask=True),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["drop", "embed", "embed", "logp", "logp", "pref", "policy"])
    dtype, back = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5
    if kind == "drop":
        T, K = _log(rng, 1, 8192), _log(rng, 48, 11008)
        if rng.random() < 0.6:  # widths are mostly multiples of a power of two
            K = max(64, K // 64 * 64)
        T = max(1, min(T, 33000000 // K))
        return dict(kind=kind, T=T, K=K, p=rng.choice([0.05, 0.1, 0.1, 0.5]),
                    step=rng.randint(0, 1 << 20), residual=not back and rng.random() < 0.5,
                    back=back, strided=rng.random() < 0.3, dtype=dtype)
    if kind == "embed":
        T, V, D = _log(rng, 1, 32768), _log(rng, 300, 130000), _log(rng, 48, 8192)
        if rng.random() < 0.6:
            D = max(64, D // 64 * 64)
        D = max(16, min(D, 32000000 // V, 32000000 // T))
        return dict(kind=kind, back=back, T=T, V=V, D=D,
                    ids=rng.choice(["text", "text", "mixed", "one"]),
                    base=back and rng.random() < 0.5, wide=rng.random() < 0.5, dtype=dtype)
    if kind == "logp":
        V = _log(rng, 300, 130000)
        if rng.random() < 0.5:
            V = max(64, V // 64 * 64)
        T = max(1, min(_log(rng, 1, 16384), 130000000 // V))
        return dict(kind=kind, back=back, T=T, V=V, ignored=rng.choice([0.0, 0.3, 0.7]),
                    wide=rng.random() < 0.5, dtype=dtype)
    S = 2 * _log(rng, 1, 2000)
    T = S * _log(rng, 1, max(2, min(8000, 2000000 // S))) + rng.randint(0, 100)
    if kind == "pref":
        form = rng.choice(["sigmoid", "sigmoid", "hinge", "squared"])
        return dict(kind=kind, S=S, T=T, form=form, beta=rng.choice([0.05, 0.1, 0.5]),
                    smoothing=rng.choice([0.0, 0.1]) if form == "sigmoid" else 0.0,
                    average=rng.random() < 0.3, ref=rng.random() < 0.8, mask=rng.random() < 0.5)
    return dict(kind=kind, S=max(1, S - rng.randint(0, 1)), T=T, kl=rng.choice([0.001, 0.04, 0.1]),
                low=0.2, high=rng.choice([0.2, 0.28]), average=rng.choice(["tokens", "sequences"]),
                by=rng.choice(["tokens", "sequences"]), ref=rng.random() < 0.7,
                mask=rng.random() < 0.6)


def _ids(case, gen):
    T, V = case["T"], case["V"]
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
    if case["ids"] == "one":
        ids = torch.full((T,), V // 3, device="cuda")
    elif case["ids"] == "mixed":
        ids = (u * V).long()
    else:  # the r-th most frequent of a text's tokens about 1/r as frequent as the first
        rank = (V + 1.0) ** u - 1
        ids = (rank.long().clamp(max=V - 1) * 7919 + 11) % V
    if T > 40:  # padding
        ids[torch.rand(T, generator=gen, device="cuda") < 0.02] = -1
    return ids if case["wide"] else ids.to(torch.int32)


def _starts(case, gen):
    """Where the sequences start, T tokens in all, in ragged lengths."""
    S, T = case["S"], case["T"]
    cuts = torch.randint(0, T + 1, (S - 1,), generator=gen, device="cuda").sort().values
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind, T = case["kind"], case["T"]

    def normal(*shape, std=1.0, dtype=torch.float32):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)

    s = dict(case=case)
    if kind == "drop":
        dt, K = TYPES[case["dtype"]], case["K"]
        # rows of a wider tensor, as a split of fused projections leaves them
        s["x"] = normal(T, K + 64, dtype=dt)[:, :K] if case["strided"] else normal(T, K, dtype=dt)
        s["residual"] = normal(T, K, dtype=dt) if case["residual"] else None
        return s
    if kind == "embed":
        dt, V, D = TYPES[case["dtype"]], case["V"], case["D"]
        s["ids"] = _ids(case, gen)
        if case["back"]:
            s["dy"] = normal(T, D, std=1e-2, dtype=dt)
            s["base"] = normal(V, D, std=1e-2, dtype=dt) if case["base"] else None
        else:
            s["weight"] = normal(V, D, std=0.02, dtype=dt)
        return s
    if kind == "logp":
        dt, V = TYPES[case["dtype"]], case["V"]
        x = torch.randn(T, V, generator=gen, device="cuda").mul_(2.5)
        t = torch.randint(0, V, (T,), generator=gen, device="cuda")
        # the model has learnt something of its targets
        x[torch.arange(T, device="cuda"), t] += 6 * torch.rand(T, generator=gen, device="cuda")
        x = x.to(dt)
        if case["ignored"] > 0 and T > 8:  # prompts before answers, four to a batch
            at = torch.arange(T, device="cuda") % (T // 4 + 1)
            t = torch.where(at < case["ignored"] * T / 4, -100, t)
        s["logits"], s["targets"] = x, t if case["wide"] else t.to(torch.int32)
        if case["back"]:
            s["norm"] = _norm(x)  # what the forward of the same step has kept
            s["dlogp"] = torch.where(t < 0, 0.0, normal(T, std=1e-3))
        return s
    s["starts"] = _starts(case, gen)
    lp = (1 - torch.rand(T, generator=gen, device="cuda")).log() * 0.8
    s["logps"] = lp
    s["ref"] = (lp + normal(T, std=0.1)).clamp(max=0) if case["ref"] else None
    s["mask"] = torch.rand(T, generator=gen, device="cuda") < 0.8 if case["mask"] else None
    if kind == "policy":
        s["old"] = lp + normal(T, std=0.15)
        s["advantages"] = normal(case["S"] if case["by"] == "sequences" else T)
    return s


# ------------------------------------------------------------- the plain form
def _wrap(z):
    """A whole number modulo 2^64 as int64 holds it."""
    z &= (1 << 64) - 1
    return z - (1 << 64) if z >> 63 else z


def _mix(z):
    """The generator's output function on 64-bit states, kept as int64."""
    def shifted(z, n):  # zeros enter from the left
        return (z >> n) & ((1 << (64 - n)) - 1)
    z = (z ^ shifted(z, 30)) * _wrap(0xBF58476D1CE4E5B9)
    z = (z ^ shifted(z, 27)) * _wrap(0x94D049BB133111EB)
    return z ^ shifted(z, 31)


def _dropped(n, seed, step, level):
    """Which of n elements are dropped: 16 bits of the stream each, below level."""
    gamma = _wrap(0x9E3779B97F4A7C15)
    stream = _mix(torch.tensor(_wrap(seed + (step + 1) * 0x9E3779B97F4A7C15), device="cuda"))
    z = _mix(stream + (torch.arange(-(-n // 4), device="cuda") + 1) * gamma)
    u = (z[:, None] >> torch.tensor([0, 16, 32, 48], device="cuda")) & 0xFFFF
    return (u < level).flatten()[:n]


def _level(p):
    return int(math.floor(p * 65536 + 0.5))


def _norm(x):
    """(T, 2): each row's largest logit, and the logarithm of the sum of exp(x - largest)."""
    x = x.float()
    m = x.amax(1)
    return torch.stack([m, (x - m[:, None]).exp().sum(1).log()], 1)


def _segments(s):
    """The sequence of every token."""
    T = s["case"]["T"]
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    return torch.searchsorted(s["starts"][1:], at, right=True)


def _sums(v, starts):
    """The sum of v over every sequence (in 64 bits: differences of running sums)."""
    c = torch.cat([v.new_zeros(1), v.cumsum(0)])[starts.long()]
    return c[1:] - c[:-1]


def run(s):
    case = s["case"]
    kind = case["kind"]
    if own:
        import unstructured_sparse_nn_amd as snk
        if kind == "drop":
            if case["back"]:
                return {"dx": snk.dropout_bwd(s["x"], case["p"], SEED, case["step"])}
            return {"y": snk.dropout_fwd(s["x"], case["p"], SEED, case["step"],
                                         residual=s["residual"])}
        if kind == "embed":
            if case["back"]:
                return {"dW": snk.embed_bwd(s["dy"], s["ids"], case["V"], scale=0.5,
                                            base=s["base"])}
            return {"y": snk.embed_fwd(s["ids"], s["weight"], scale=8.0)}
        if kind == "logp":
            if case["back"]:
                return {"dx": snk.logp_bwd(s["dlogp"], s["logits"], s["targets"], s["norm"])}
            logp, norm = snk.logp_fwd(s["logits"], s["targets"])
            return {"logp": logp, "norm": norm}
        if kind == "pref":
            loss, rewards, g = snk.preference_grads(
                s["logps"], s["starts"], ref=s["ref"], mask=s["mask"], beta=case["beta"],
                smoothing=case["smoothing"], form=case["form"], average=case["average"])
            return {"loss": loss, "rewards": rewards, "dlogps": g}
        loss, stats, g = snk.policy_grads(
            s["logps"], s["old"], s["advantages"], s["starts"], ref=s["ref"], mask=s["mask"],
            clip=(case["low"], case["high"]), kl=case["kl"], average=case["average"],
            by=case["by"])
        return {"loss": loss, "stats": stats, "dlogps": g}
    if kind == "drop":
        x, level = s["x"], _level(case["p"])
        out = _dropped(x.numel(), SEED, case["step"], level).view(x.shape)
        y = torch.where(out, 0.0, x.float() * (65536 / (65536 - level)))
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return {"dx" if case["back"] else "y": y.to(x.dtype)}
    if kind == "embed":
        ids = s["ids"].long()
        if not case["back"]:
            w = s["weight"]
            y = torch.where((ids >= 0)[:, None], w[ids.clamp(min=0)].float() * 8.0, 0.0)
            return {"y": y.to(w.dtype)}
        dy = torch.where((ids >= 0)[:, None], s["dy"].float(), 0.0)
        dW = torch.zeros(case["V"], case["D"], device="cuda").index_add_(0, ids.clamp(min=0), dy)
        dW = dW * 0.5
        if s["base"] is not None:
            dW = s["base"].float() + dW
        return {"dW": dW.to(s["dy"].dtype)}
    if kind == "logp":
        x, t = s["logits"].float(), s["targets"].long()
        rows, has = torch.arange(case["T"], device="cuda"), t >= 0
        norm = s["norm"] if case["back"] else _norm(x)
        logp = (x - norm[:, :1]) - norm[:, 1:]
        mine = torch.where(has, logp[rows, t.clamp(min=0)], 0.0)
        if not case["back"]:
            return {"logp": mine, "norm": norm}
        g = torch.where(has, s["dlogp"], 0.0)
        dx = logp.exp() * -g[:, None]
        dx[rows, t.clamp(min=0)] = -mine.expm1() * g
        return {"dx": dx.to(s["logits"].dtype)}
    # values next to a border and sums of millions of terms: in 64 bits
    S, of = case["S"], _segments(s)
    lp = s["logps"].double()
    counts = torch.ones_like(lp) if s["mask"] is None else s["mask"].double()
    ratio = lp - s["ref"].double() if s["ref"] is not None else None
    n = _sums(counts, s["starts"])
    if kind == "pref":
        beta, eps = case["beta"], case["smoothing"]
        d = _sums(torch.where(counts > 0, lp if ratio is None else ratio, 0.0), s["starts"])
        per = 1 / n.clamp(min=1) if case["average"] else torch.ones_like(n)
        d = d * per
        z = beta * (d[0::2] - d[1::2])
        if case["form"] == "sigmoid":
            loss = ((1 - eps) * torch.log1p(torch.exp(-z.abs())) + (1 - eps) * (-z).clamp(min=0)
                    + eps * torch.log1p(torch.exp(-z.abs())) + eps * z.clamp(min=0))
            dz = eps / (1 + torch.exp(-z)) - (1 - eps) / (1 + torch.exp(z))
        elif case["form"] == "hinge":
            loss, dz = (1 - z).clamp(min=0), -(z < 1).double()
        else:
            loss = (z / beta - 0.5 / beta) ** 2
            dz = 2 * (z / beta - 0.5 / beta) / beta
        c = torch.stack([dz, -dz], 1).flatten() * beta * per / (S // 2)
        g = torch.where(counts > 0, c[of], 0.0)
        return {"loss": loss.mean().float(), "rewards": (beta * d).view(-1, 2).float(),
                "dlogps": g.float()}
    a = s["advantages"].double()
    if case["by"] == "sequences":
        a = a[of]
    move = lp - s["old"].double()
    cut = (((a > 0) & (move > math.log1p(case["high"])))
           | ((a < 0) & (move < math.log1p(-case["low"]))))
    limit = torch.where(a > 0, 1 + case["high"], 1 - case["low"])
    part = -torch.where(cut, limit, move.exp()) * a
    dpart = torch.where(cut, 0.0, -move.exp() * a)
    kl = torch.zeros_like(lp)
    if ratio is not None:
        kl = torch.expm1(-ratio) + ratio
        part = part + case["kl"] * kl
        dpart = dpart - case["kl"] * torch.expm1(-ratio)
    weight = (1 / (S * n.clamp(min=1)))[of] if case["average"] == "sequences" \
        else 1 / n.sum().clamp(min=1)
    weight = torch.where(counts > 0, weight, 0.0)
    total = n.sum().clamp(min=1)
    stats = torch.stack([(kl * counts).sum() / total, (cut * counts).sum() / total])
    return {"loss": (part * weight).sum().float(), "stats": stats.float(),
            "dlogps": (dpart * weight).float()}


# ---------------------------------------------------------- the exact values
def _kept_exactly(n, step, level):
    """Which of n elements stay, from the generator's definition on unsigned numbers."""
    u64 = np.uint64
    with np.errstate(over="ignore"):
        def out(state):
            state = (state ^ (state >> u64(30))) * u64(0xBF58476D1CE4E5B9)
            state = (state ^ (state >> u64(27))) * u64(0x94D049BB133111EB)
            return state ^ (state >> u64(31))
        gamma = u64(0x9E3779B97F4A7C15)
        first = out(np.array([SEED], dtype=u64) + u64(step + 1) * gamma)
        z = out(first + np.arange(1, -(-n // 4) + 1, dtype=u64) * gamma)
    fields = z.astype("<u8").view("<u2")[:n]
    return torch.from_numpy(fields >= level)


def exact(case, seed):
    """The same outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    kind, T = case["kind"], case["T"]
    if kind == "drop":
        level = _level(case["p"])
        keep = _kept_exactly(T * case["K"], case["step"], level).cuda().view(T, case["K"])
        y = s["x"].double() * 65536 / (65536 - level) * keep
        return {"dx" if case["back"] else "y": y if s["residual"] is None
                else y + s["residual"].double()}
    if kind == "embed":
        real = (s["ids"] >= 0).nonzero()[:, 0]
        if not case["back"]:
            y = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
            y[real] = 8 * s["weight"].double()[s["ids"][real].long()]
            return {"y": y}
        out = torch.zeros(case["V"], case["D"], dtype=torch.float64, device="cuda")
        out.index_put_((s["ids"][real].long(),), s["dy"][real].double() / 2, accumulate=True)
        return {"dW": out if s["base"] is None else out + s["base"].double()}
    if kind == "logp":
        logp, norm, dx = [], [], []
        for rows in torch.arange(T, device="cuda").split(1024):
            x, t = s["logits"][rows].double(), s["targets"][rows].long()
            top, has = x.max(1).values, t >= 0
            lse = torch.logsumexp(x, 1)
            norm.append(torch.stack([top, lse - top], 1))
            own_x = x.gather(1, t.clamp(min=0)[:, None])[:, 0]
            logp.append((own_x - lse) * has)
            if case["back"]:
                g = (s["dlogp"][rows].double() * has)[:, None]
                one = torch.zeros_like(x).scatter_(1, t.clamp(min=0)[:, None], 1.0)
                dx.append(g * (one - (x - lse[:, None]).exp()))
        if case["back"]:
            return {"dx": torch.cat(dx)}
        return {"logp": torch.cat(logp), "norm": torch.cat(norm)}
    # sequence by sequence, on the CPU
    c = {k: v.double().cpu() for k, v in s.items() if isinstance(v, torch.Tensor)}
    cuts, S = [int(v) for v in c["starts"]], case["S"]
    runs = [slice(a, b) for a, b in zip(cuts[:-1], cuts[1:])]
    counts = c.get("mask", torch.ones(T, dtype=torch.float64))
    g = torch.zeros(T, dtype=torch.float64)
    if kind == "pref":
        beta, P, loss, rewards = case["beta"], S // 2, 0.0, []
        for p in range(P):
            d, per = [], []
            for q in runs[2 * p:2 * p + 2]:
                r = c["logps"][q] - c["ref"][q] if "ref" in c else c["logps"][q]
                per.append(1 / max(1.0, float(counts[q].sum())) if case["average"] else 1.0)
                d.append(float((r * counts[q]).sum()) * per[-1])
            h = d[0] - d[1]
            z = beta * h
            if case["form"] == "sigmoid":
                e = case["smoothing"]
                soft = lambda v: max(v, 0) + math.log1p(math.exp(-abs(v)))  # noqa: E731
                sig = lambda v: 0.5 * (1 + math.tanh(v / 2))  # noqa: E731
                loss += (1 - e) * soft(-z) + e * soft(z)
                dh = beta * (e * sig(z) - (1 - e) * sig(-z))
            elif case["form"] == "hinge":
                loss += max(0.0, 1 - z)
                dh = -beta if z < 1 else 0.0
            else:
                loss += (h - 1 / (2 * beta)) ** 2
                dh = 2 * (h - 1 / (2 * beta))
            rewards.append([beta * d[0], beta * d[1]])
            for k, q in enumerate(runs[2 * p:2 * p + 2]):
                g[q] = (1 - 2 * k) * dh * per[k] / P * counts[q]
        return {"loss": loss / P, "rewards": torch.tensor(rewards, dtype=torch.float64),
                "dlogps": g}
    loss = kl_sum = cut_sum = 0.0
    total = max(1.0, float(counts.sum()))
    low, high = math.log1p(-case["low"]), math.log1p(case["high"])
    for i, q in enumerate(runs):
        a = c["advantages"][q] if case["by"] == "tokens" else c["advantages"][i]
        m = counts[q]
        w = m / total if case["average"] == "tokens" else m / (S * max(1.0, float(m.sum())))
        move = c["logps"][q] - c["old"][q]
        r = move.exp()
        up, down = (a > 0) & (move > high), (a < 0) & (move < low)
        held = torch.where(up, 1 + case["high"], torch.where(down, 1 - case["low"], r))
        loss -= float((w * held * a).sum())
        g[q] -= torch.where(up | down, 0.0, w * r * a)
        cut_sum += float(((up | down) * m).sum())
        if "ref" in c:
            d = c["ref"][q] - c["logps"][q]
            k3 = d.expm1() - d
            loss += case["kl"] * float((w * k3).sum())
            g[q] -= case["kl"] * w * d.expm1()
            kl_sum += float((k3 * m).sum())
    return {"loss": loss, "stats": torch.tensor([kl_sum / total, cut_sum / total]).double(),
            "dlogps": g}


def work(case):
    kind, T = case["kind"], case["T"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if kind == "drop":
        n = T * case["K"]
        return {"bytes": e * n * (3 if case["residual"] else 2), "flops": 2 * n}
    if kind == "embed":
        D, V, i = case["D"], case["V"], 8 if case["wide"] else 4
        if not case["back"]:
            return {"bytes": e * D * (T + min(T, V)) + i * T, "flops": T * D}
        return {"bytes": e * D * (T + (2 if case["base"] else 1) * V) + i * T, "flops": T * D}
    if kind == "logp":
        n, i = T * case["V"], 8 if case["wide"] else 4
        if not case["back"]:
            return {"bytes": e * n + (i + 12) * T, "flops": 4 * n}
        read = 1 - case["ignored"] if T > 8 else 1  # rows without a target are written only
        return {"bytes": int(e * n * (1 + read)) + (i + 12) * T, "flops": 4 * n}
    per = 8 + (4 if case["ref"] else 0) + (1 if case["mask"] else 0)
    if kind == "pref":
        return {"bytes": per * T + 12 * case["S"], "flops": 4 * T}
    per += 4 + (4 if case["by"] == "tokens" else 0)
    return {"bytes": per * T + 8 * case["S"], "flops": 40 * T}
