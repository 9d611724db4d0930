"""Workloads of the low-rank adapters and of gradient clipping, for timing and
for comparing the library's kernels with a plain form of the same formulas.

Three kinds of case:
  fwd   y = base + s_a t B_a with t = x A_a^T, a = the adapter of each token
  bwd   dx, dA and dB of the same from dy
  clip  the 2-norm over many gradients, and the gradients scaled by
        min(1, max_norm / (norm + eps))

``own`` selects the library's kernels (True) or the plain form (False).
"""
import math

import torch

own = False

EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one request of one token beside a 4096 x 4096 projection: latency
        dict(name="decode_1", kind="fwd", T=1, K=4096, M=4096, L=8, R=16, ids="mixed", mixed=False,
             base=True, save=False, dtype="bf16"),
        # a decode step of 37 requests, each with its own adapter, ranks 8 to 32
        dict(name="decode_37", kind="fwd", T=37, K=4096, M=11008, L=64, R=32, ids="mixed",
             mixed=True, base=True, save=False, dtype="bf16"),
        # a few drafted tokens each of some dozens of requests
        dict(name="draft_200", kind="fwd", T=200, K=4096, M=4096, L=16, R=64, ids="segments",
             mixed=False, base=True, save=False, dtype="bf16"),
        # prompts of several requests, ragged, one after the other
        dict(name="prompts_4099", kind="fwd", T=4099, K=4096, M=11008, L=12, R=16, ids="segments",
             mixed=False, base=True, save=False, dtype="bf16"),
        # odd sizes in fp32, no shared projection beside it
        dict(name="odd_f32", kind="fwd", T=515, K=1001, M=2047, L=3, R=12, ids="mixed", mixed=True,
             base=False, save=False, dtype="f32"),
        # the forward of a fine-tuning step, which keeps t for its backward
        dict(name="train_fwd_8192", kind="fwd", T=8192, K=4096, M=4096, L=1, R=16, ids="one",
             mixed=False, base=True, save=True, dtype="bf16"),
        # the backward of a small fp32 model with four tasks, t computed again
        dict(name="bwd_f32_1024", kind="bwd", T=1024, K=768, M=2304, L=4, R=8, ids="segments",
             mixed=False, base=True, save=False, dtype="f32"),
        # the backward of a fine-tuning step of one adapter
        dict(name="bwd_8192", kind="bwd", T=8192, K=4096, M=4096, L=1, R=16, ids="one",
             mixed=False, base=True, save=True, dtype="bf16"),
        # 24 adapters trained together on tokens in any order, high ranks
        dict(name="bwd_mixed_6001", kind="bwd", T=6001, K=4096, M=11008, L=24, R=64, ids="mixed",
             mixed=True, base=True, save=True, dtype="bf16"),
        # the adapters of a small model: 48 gradients of a few thousand elements
        dict(name="clip_adapters", kind="clip", n=48, low=768, high=18432, dtype="f32",
             bucket=False, max_norm=1.0),
        # one flat bucket holding 600 gradients of odd sizes, as views
        dict(name="clip_bucket", kind="clip", n=600, low=1, high=400000, dtype="bf16",
             bucket=True, max_norm=1.0),
        # the value gradients of 48 sparse projections at 90% sparsity
        dict(name="clip_values", kind="clip", n=48, low=1677722, high=4508877, dtype="bf16",
             bucket=False, max_norm=1.0),
    ]


def _log(rng, low, high):
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "clip":
        n = _log(rng, 1, 600)
        high = _log(rng, 64, min(4000000, 150000000 // n))
        return dict(kind=kind, n=n, low=max(1, high // rng.randint(1, 200)), high=high, dtype=dtype,
                    bucket=n > 48 or rng.random() < 0.3, max_norm=rng.choice([0.5, 1.0, 1e5]))
    T, K, M = _log(rng, 1, 8192), _log(rng, 48, 11008), _log(rng, 48, 11008)
    if rng.random() < 0.6:  # model widths are mostly multiples of a power of two
        K, M = max(64, K // 64 * 64), max(64, M // 64 * 64)
    L, R = _log(rng, 1, 64), rng.choice([1, 4, 8, 12, 16, 16, 32, 64])
    T = max(1, min(T, 60000000 // (K + M), 90000000000 // ((K + M) * L * R)))
    return dict(kind=kind, T=T, K=K, M=M, L=L, R=R, ids=rng.choice(["one", "segments", "mixed"]),
                mixed=rng.random() < 0.4, base=rng.random() < 0.8, save=rng.random() < 0.5,
                dtype=dtype)


def _ranks(case):
    """Ranks of the adapters: all R, or R, R/2, R/4 in turn."""
    return [max(1, case["R"] >> (l % 3)) if case["mixed"] else case["R"] for l in range(case["L"])]


def _sizes(case):
    """Element counts of the gradients: low to high, evenly over the logarithm, in mixed order."""
    n, a, b = case["n"], math.log(case["low"]), math.log(case["high"])
    return [int(math.exp(a + (b - a) * ((i * 37) % n) / max(1, n - 1))) for i in range(n)]


def _ids(case, gen):
    T, L = case["T"], case["L"]
    if case["ids"] == "one":
        return torch.zeros(T, dtype=torch.int32, device="cuda")
    if case["ids"] == "mixed":  # any order, some tokens without an adapter (where more than one)
        low = -1 if T > 1 else 0
        ids = torch.randint(low, L, (T,), generator=gen, device="cuda")
        return ids.to(torch.int32)
    n = min(T, 2 * L)  # ragged runs of tokens, two to an adapter
    cuts = torch.randint(0, T, (n - 1,), generator=gen, device="cuda").sort().values
    of = torch.randint(0, L, (n,), generator=gen, device="cuda")
    run = torch.searchsorted(cuts, torch.arange(T, device="cuda"), right=True)
    return of[run].to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dt)

    s = dict(case=case)
    if case["kind"] == "clip":
        sizes = _sizes(case)
        if case["bucket"]:
            s["flat"] = normal(sum(sizes), std=1e-2)
            s["flat_out"] = torch.empty_like(s["flat"])
            s["grads"], s["out"] = list(s["flat"].split(sizes)), list(s["flat_out"].split(sizes))
        else:
            s["grads"] = [normal(n, std=1e-2) for n in sizes]
            s["out"] = [torch.empty_like(g) for g in s["grads"]]
        return s
    T, K, M, L, R = (case[k] for k in "TKMLR")
    ranks = _ranks(case)
    s["ids"] = _ids(case, gen)
    s["A"] = normal(L, R, K, std=K ** -0.5)
    s["B"] = normal(L, R, M, std=0.05)
    s["scale"] = torch.tensor([16.0 / r for r in ranks], device="cuda")
    s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda") if case["mixed"] else None
    s["x"] = normal(T, K)
    if case["kind"] == "fwd":
        s["base"] = normal(T, M) if case["base"] else None
        s["out"] = torch.empty(T, M, dtype=dt, device="cuda")
        s["t"] = torch.empty(T, R, device="cuda") if case["save"] else None
    else:
        s["dy"] = normal(T, M, std=0.02)
        s["base"] = normal(T, K, std=0.02) if case["base"] else None
        # what the forward of the same step has kept
        s["t"] = _reduce(s["x"], s["A"], s["ids"], s["ranks"]) if case["save"] else None
    return s


def _mine(ids, ranks, R):
    """(T, R): which ranks each token has."""
    has = (ids >= 0)[:, None].expand(-1, R)
    if ranks is None:
        return has
    of = ranks[ids.long().clamp(min=0)]
    return has & (torch.arange(R, device=ids.device) < of[:, None])


def _reduce(x, F, ids, ranks):
    """t[i, j] = sum_k F[a(i), j, k] x[i, k], (T, R) in fp32."""
    (L, R, K), T = F.shape, x.shape[0]
    a = ids.long().clamp(min=0)
    if T * R * K <= 1 << 26:
        t = (F[a].float() * x.float()[:, None, :]).sum(-1)
    else:
        t = (x.float() @ F.float().view(L * R, K).t()).view(T, L, R)
        t = t[torch.arange(T, device=x.device), a]
    return torch.where(_mine(ids, ranks, R), t, 0.0)


def _wide(t, ids, L):
    """(T, L * R): t in the columns of each token's adapter, zeros elsewhere."""
    T, R = t.shape
    w = torch.zeros(T, L, R, device=t.device)
    w[torch.arange(T, device=t.device), ids.long().clamp(min=0)] = t
    return w.view(T, L * R)


def _expand(t, F, ids):
    """sum_j t[i, j] F[a(i), j, m], (T, M) in fp32."""
    (L, R, M), T = F.shape, t.shape[0]
    if T * R * M <= 1 << 26:
        return (t[:, :, None] * F[ids.long().clamp(min=0)].float()).sum(1)
    return _wide(t, ids, L) @ F.float().view(L * R, M)


def _scaled(t, s):
    return t * s["scale"][s["ids"].long().clamp(min=0)][:, None]


def run(s):
    case = s["case"]
    if own:
        import unstructured_sparse_nn_amd as snk
        if case["kind"] == "clip":
            norm = snk.clip_grads(s["grads"], case["max_norm"], eps=EPS, out=s["out"])
            return {"norm": norm, "grads": s["flat_out"] if case["bucket"] else s["out"]}
        if case["kind"] == "fwd":
            y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], scale=s["scale"], ranks=s["ranks"],
                             base=s["base"], out=s["out"], t=s["t"])
            return {"y": y, "t": s["t"]} if case["save"] else {"y": y}
        dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], scale=s["scale"],
                                  ranks=s["ranks"], t=s["t"], base=s["base"])
        return {"dx": dx, "dA": dA, "dB": dB}
    if case["kind"] == "clip":
        # squares summed in 64 bits: sums of 10^8 terms
        sums = torch.stack([g.double().square().sum() for g in s["grads"]])
        norm = sums.sum().sqrt()
        c = (case["max_norm"] / (norm + EPS)).clamp(max=1.0)
        if case["bucket"]:
            return {"norm": norm.float(), "grads": (s["flat"].float() * c.float()).to(s["flat"].dtype)}
        return {"norm": norm.float(),
                "grads": [(g.float() * c.float()).to(g.dtype) for g in s["grads"]]}
    ids, A, B, ranks = s["ids"], s["A"], s["B"], s["ranks"]
    if case["kind"] == "fwd":
        t = _reduce(s["x"], A, ids, ranks)
        y = _expand(_scaled(t, s), B, ids)
        if s["base"] is not None:
            y = s["base"].float() + y
        y = y.to(s["x"].dtype)
        return {"y": y, "t": t} if case["save"] else {"y": y}
    dt, (L, R, K), M = s["x"].dtype, A.shape, B.shape[2]
    t = s["t"] if case["save"] else _reduce(s["x"], A, ids, ranks)
    u = _scaled(_reduce(s["dy"], B, ids, ranks), s)
    dx = _expand(u, A, ids)
    if s["base"] is not None:
        dx = s["base"].float() + dx
    dA = _wide(u, ids, L).t() @ s["x"].float()
    dB = _wide(_scaled(t, s), ids, L).t() @ s["dy"].float()
    return {"dx": dx.to(dt), "dA": dA.view(L, R, K).to(dt), "dB": dB.view(L, R, M).to(dt)}


def exact(case, seed):
    """The same outputs from the definitions in 64 bits, adapter by adapter."""
    s = prepare(case, seed)
    if case["kind"] == "clip":
        total = sum(float((g.double() ** 2).sum()) for g in s["grads"])
        norm = math.sqrt(total)
        c = min(1.0, case["max_norm"] / (norm + EPS))
        if case["bucket"]:
            return {"norm": norm, "grads": s["flat"].double() * c}
        return {"norm": norm, "grads": [g.double() * c for g in s["grads"]]}
    T, K, M, L, R = (case[k] for k in "TKMLR")
    x, A, B = s["x"].double(), s["A"].double(), s["B"].double()
    f64 = dict(dtype=torch.float64, device=x.device)
    fwd = case["kind"] == "fwd"
    out = torch.zeros(T, M if fwd else K, **f64) if s["base"] is None else s["base"].double()
    t_all = torch.zeros(T, R, **f64)
    dA, dB = torch.zeros(L, R, K, **f64), torch.zeros(L, R, M, **f64)
    for l, r in enumerate(_ranks(case)):
        rows = (s["ids"] == l).nonzero()[:, 0]
        if rows.numel() == 0:
            continue
        xl, Al, Bl, sl = x[rows], A[l, :r], B[l, :r], float(s["scale"][l])
        t = xl @ Al.t()
        t_all[rows, :r] = t
        if fwd:
            out[rows] += sl * (t @ Bl)
            continue
        dyl = s["dy"].double()[rows]
        if case["save"]:
            t = s["t"].double()[rows, :r]
        u = dyl @ Bl.t()
        out[rows] += sl * (u @ Al)
        dA[l, :r] = sl * (u.t() @ xl)
        dB[l, :r] = sl * (t.t() @ dyl)
    if fwd:
        return {"y": out, "t": t_all} if case["save"] else {"y": out}
    return {"dx": out, "dA": dA, "dB": dB}


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * e * n, "flops": 3 * n}
    T, K, M, L, R = (case[k] for k in "TKMLR")
    ranks = _ranks(case)
    used = 1 if case["ids"] == "one" else min(L, T)  # adapters that tokens have
    r = sum(ranks) / L  # a token's rank
    ab = e * used * r * (K + M)
    kept = 4 * T * R if case["save"] else 0
    if case["kind"] == "fwd":
        return {"bytes": e * T * (K + M + (M if case["base"] else 0)) + ab + kept,
                "flops": 2 * T * r * (K + M)}
    return {"bytes": e * T * (2 * K + M + (K if case["base"] else 0)) + ab + kept
            + e * L * R * (K + M),
            "flops": 2 * T * r * (2 * K + 2 * M + (0 if case["save"] else K))}
