"""Adapters where values, tensors or sizes are special: infinities and NaN in
the gradients, outputs that other tensors share, moves of the module between
types, sizes past what a launch holds.  Formulas and tolerances are those of
the adapters' other tests."""
import ctypes
import random

import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b
from test_lora import close, make, reference

gpu = pytest.mark.gpu


def exact_grads(s, t=None):
    """dA and dB by the formulas in 64 bits, term by term, so that infinities
    and NaN come out as the formulas have them."""
    x, dy, A, B = (s[k].double().cpu() for k in ("x", "dy", "A", "B"))
    ids, scale = s["ids"].cpu(), s["scale"].double().cpu()
    dA, dB = torch.zeros_like(A), torch.zeros_like(B)
    for l in range(A.shape[0]):
        rows, r = (ids == l).nonzero()[:, 0], int(s["ranks"][l])
        for j in range(r if rows.numel() else 0):
            u = (dy[rows] * B[l, j]).sum(1)
            tj = (x[rows] * A[l, j]).sum(1) if t is None else t[rows.to(t.device), j].double().cpu()
            dA[l, j] = scale[l] * (u[:, None] * x[rows]).sum(0)
            dB[l, j] = scale[l] * (tj[:, None] * dy[rows]).sum(0)
    return {"dA": dA, "dB": dB}


def same_pattern(got, want, ref, tol, what):
    """Infinities and NaN where the formula has them, and the rest close."""
    g = got.double().cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(want)), what
    inf = torch.isinf(want)
    assert torch.equal(torch.isinf(g), inf) and torch.equal(g[inf], want[inf]), what
    ok = torch.isfinite(want)
    close(g[ok], ref[ok], tol[ok], what)


# One adapter or several, one run of tokens or several that are joined, ranks
# up to and past 16, and none of them a multiple of it.
RANKS = [(90, 1, 16, [5]), (300, 3, 16, [8, 5, 9]), (700, 1, 40, [20]), (2500, 3, 64, [9, 33, 20]),
         (6000, 1, 20, [5]), (6000, 2, 16, [9, 16])]


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["x", "dy"])
@pytest.mark.parametrize("case", RANKS, ids=str)
def test_infinities_in_the_gradients(case, where, dt):
    """An infinity and a NaN in rows that have an adapter: ranks that it does
    not have stay zero, every other entry is the formula's."""
    T, L, R, ranks = case
    s = make(T, 136, 200, L, R, dt, seed=T + R, ids="runs", ranks=False)
    s["ids"][3] = -1
    s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    args = (s["A"], s["B"], s["scale"], s["ranks"])
    t = torch.empty(T, R, device="cuda")
    snk.lora_fwd(s["x"], s["ids"], *args, t=t)
    ref, tol = reference(s, dt, grads=True)  # of the finite columns
    s[where][1, 7], s[where][T - 2, 100] = float("inf"), float("nan")
    for kept in (t, None):
        want = exact_grads(s, kept)
        dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], *args, t=kept)
        for l, r in enumerate(ranks):
            # a NaN counts as nonzero
            assert int(dA[l, r:].count_nonzero()) == 0 == int(dB[l, r:].count_nonzero()), (l, r)
        same_pattern(dA, want["dA"], ref["dA"], tol["dA"], "dA")
        same_pattern(dB, want["dB"], ref["dB"], tol["dB"], "dB")


@gpu
@pytest.mark.parametrize("T", [5, 100])
def test_written_tensors_count_as_changed(T):
    """What a call writes into its caller's tensors moves their version, so that
    a backward that has saved them raises instead of using the new values."""
    s = make(T, 24, 24, 2, 8, "f32", seed=T, ranks=False)
    args = (s["ids"], s["A"], s["B"])

    def saved(n):  # sigmoid's backward uses its output
        return torch.sigmoid(torch.zeros(T, n, device="cuda", requires_grad=True))

    calls = [(24, lambda v: snk.lora_fwd(s["x"], *args, base=v, out=v)),
             (24, lambda v: snk.lora_fwd(s["x"], *args, out=v)),
             (8, lambda v: snk.lora_fwd(s["x"], *args, t=v)),
             (24, lambda v: snk.lora_bwd(s["dy"], s["x"], *args, base=v, out=v)),
             (24, lambda v: snk.lora_bwd(s["dy"], s["x"], *args, out=v, want=(True, False, False)))]
    for n, call in calls:
        v = saved(n)
        version = v._version
        with torch.no_grad():
            call(v)
        assert v._version > version
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            v.sum().backward()
    v = saved(24)  # only read: as before
    with torch.no_grad():
        snk.lora_fwd(s["x"], *args, base=v)
        snk.lora_bwd(s["dy"], s["x"], *args, base=v)
    v.sum().backward()
    with torch.inference_mode():  # has no versions
        v = torch.zeros(T, 24, device="cuda")
        assert snk.lora_fwd(s["x"], *args, out=v) is v


# Addresses far apart: nothing here is read, for every call is refused.
PLACES = dict(X=1 << 30, Y=2 << 30, base=3 << 30, A=4 << 30, B=5 << 30, ids=6 << 30, t=7 << 30,
              scale=8 << 30, rank=9 << 30, ws=10 << 30, dA=11 << 30, dB=12 << 30, dX=13 << 30)
SIZE = dict(T=40, K=64, M=32, L=2, R=8)  # fp32
BYTES = dict(X=40 * 64 * 4, Y=40 * 32 * 4, base=40 * 32 * 4, A=2 * 8 * 64 * 4, B=2 * 8 * 32 * 4,
             ids=40 * 4, t=40 * 8 * 4, scale=8, rank=8)


def raw(which, **places):
    """The status of a call with contiguous tensors at these addresses."""
    p, z = {**PLACES, **places}, SIZE
    bank = ctypes.byref(b.snack_lora(p["A"], p["B"], z["M"], z["K"], z["L"], z["R"], p["scale"],
                                     p["rank"]))
    end = (p["ws"], 1 << 30, None)
    if which == "fwd":
        return b.raw_status("snack_lora_fwd", bank, 0, p["ids"], z["T"], p["X"], z["K"], p["base"],
                            z["M"], p["Y"], z["M"], p["t"], *end)
    return b.raw_status("snack_lora_bwd", bank, 0, p["ids"], p["t"], z["T"], p["X"], z["K"], p["Y"],
                        z["M"], p["base"], z["K"], p["dX"], z["K"], p["dA"], p["dB"], *end)


@pytest.mark.parametrize("name", ["X", "base", "A", "B", "ids", "t", "scale", "rank"])
def test_outputs_over_other_tensors_are_refused(name):
    """The first or the last element of an output on another tensor's."""
    at, n = PLACES[name], BYTES[name]
    for start in (at + n - 4, at - BYTES["Y"] + 4, at + 4 if n > 8 else at):
        assert raw("fwd", Y=start) == -2, (name, start - at)
    if name != "t":
        for start in (at + n - 4, at - BYTES["t"] + 4, at):
            assert raw("fwd", t=start) == -2, (name, start - at)
    n = BYTES["X"] if name == "base" else n  # the backward's base is like X
    for out, size in (("dX", BYTES["X"]), ("dA", BYTES["A"]), ("dB", BYTES["B"])):
        for start in (at + n - 4, at - size + 4):
            assert raw("bwd", **{out: start}) == -2, (name, out, start - at)


def test_outputs_over_outputs_are_refused():
    assert raw("bwd", dA=PLACES["dB"] + BYTES["B"] - 4) == -2
    assert raw("bwd", dA=PLACES["dX"]) == -2 and raw("bwd", dB=PLACES["dX"] + 4) == -2
    assert raw("bwd", dX=PLACES["Y"] + 8) == -2            # over dY
    assert raw("fwd", base=PLACES["Y"] + 32 * 4) == -2     # base a row further on


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("seed", range(4))
def test_rows_beside_each_other_in_one_buffer(seed, dt):
    """Rows of x and y anywhere in one buffer: a call is refused exactly where
    an element belongs to both, and otherwise right."""
    from test_lora import DT
    rng = random.Random(seed)
    T, K, M, L, R = 7, 12, 9, 2, 4
    s = make(T, K, M, L, R, dt, seed=seed, ranks=False)
    lora = b.snack_lora(s["A"], s["B"], M, K, L, R)
    ws = torch.empty(b.snack_lora_workspace(lora, b._dtype(s["x"]), T), dtype=torch.uint8,
                     device="cuda")
    want = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"])
    done = {True: 0, False: 0}
    for _ in range(300):
        ldx, ldy = rng.choice([(24, 24), (24, 24), (25, 25), (48, 24), (24, 31), (12, 9), (60, 60)])
        ox, oy = rng.randrange(0, 300), rng.randrange(0, 300)
        if rng.random() < 0.5:  # next to each other's rows
            oy = ox + rng.choice([-1, 0, 1, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16]) + ldx * rng.randrange(8)
            oy = max(oy, 0)
        over = bool({ox + i * ldx + k for i in range(T) for k in range(K)}
                    & {oy + i * ldy + m for i in range(T) for m in range(M)})
        buf = torch.zeros(1500, dtype=DT[dt], device="cuda")
        x, y = buf[ox:].as_strided((T, K), (ldx, 1)), buf[oy:].as_strided((T, M), (ldy, 1))
        x.copy_(s["x"])
        kept = buf.clone()
        try:
            b.snack_lora_fwd(lora, s["ids"], T, x, ldx, None, M, y, ldy, ws=ws)
        except snk.SnackError as e:
            assert e.status == -2 and over, (ox, oy, ldx, ldy)
            assert torch.equal(buf, kept)
        else:
            assert not over, (ox, oy, ldx, ldy)
            assert torch.equal(y, want) and torch.equal(x, s["x"])
        done[over] += 1
    assert min(done.values()) > 50


@pytest.mark.parametrize("move", [lambda m: m.to(torch.bfloat16), lambda m: m.bfloat16(),
                                  lambda m: m.type(torch.bfloat16),
                                  lambda m: torch.nn.Sequential(m).bfloat16()[0],
                                  lambda m: m.bfloat16().float()], ids=range(5))
def test_scales_and_ranks_keep_their_type(move):
    m = snk.LoraAdapters(24, 16, 3, 8, alpha=5.0, ranks=[3, 7, 8], device="cpu")
    moved = move(m)
    assert moved.scale.dtype == torch.float32 and moved.ranks.dtype == torch.int32
    assert torch.equal(moved.scale, torch.tensor([5 / 3, 5 / 7, 5 / 8]))
    assert moved.ranks.tolist() == [3, 7, 8]
    assert set(dict(moved.named_buffers())) == {"scale", "ranks"}
    meta = moved.to("meta")
    assert meta.scale.is_meta and meta.bfloat16().A.dtype == torch.bfloat16
    assert snk.LoraAdapters(24, 16, 3, 8, device="cpu").bfloat16().ranks is None


@gpu
@pytest.mark.parametrize("default", [torch.float32, torch.bfloat16, torch.float64])
def test_moved_module_and_other_default_types(default):
    """The module cast to bf16 and moved to the GPU, and made under another
    default type, computes what its parameters say."""
    s = make(70, 24, 16, 3, 8, "bf16", seed=6, ranks=False)
    s["ranks"] = torch.tensor([3, 7, 8], dtype=torch.int32, device="cuda")
    before = torch.get_default_dtype()
    torch.set_default_dtype(default)
    try:
        m = torch.nn.Sequential(snk.LoraAdapters(24, 16, 3, 8, alpha=5.0, ranks=[3, 7, 8],
                                                 device="cpu")).bfloat16().cuda()[0]
        with torch.no_grad():
            m.A.copy_(s["A"])
            m.B.copy_(s["B"])
        x = s["x"].clone().requires_grad_()
        y = m(x, s["ids"], s["base"])
        y.backward(s["dy"])
    finally:
        torch.set_default_dtype(before)
    s["scale"], s["gbase"] = torch.tensor([5 / 3, 5 / 7, 5 / 8]), torch.zeros(70, 24)
    ref, tol = reference(s, "bf16", grads=True)
    for k, v in (("y", y.detach()), ("dx", x.grad), ("dA", m.A.grad), ("dB", m.B.grad)):
        close(v, ref[k], tol[k], k)


MOST = {False: 2 ** 28 - 2 ** 20, True: 2 ** 27 - 2 ** 19}  # tokens of a forward and of a backward


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("L,R", [(1, 1), (8192, 256)])
def test_more_tokens_than_a_launch_holds_are_refused(L, R, backward):
    bank = b.snack_lora(PLACES["A"], PLACES["B"], 8, 8, L, R)
    most = MOST[backward]
    assert b.snack_lora_workspace(bank, b.F32, most, backward) > 0
    for T in (most + 1, 2 ** 30):
        with pytest.raises(snk.SnackError) as e:
            b.snack_lora_workspace(bank, b.F32, T, backward)
        assert e.value.status == -10
        args = (PLACES["ws"], 1 << 50, None)
        if backward:
            st = b.raw_status("snack_lora_bwd", ctypes.byref(bank), 0, 1 << 20, None, T, 1 << 40, 8,
                              1 << 42, 8, None, 8, 1 << 44, 8, None, None, *args)
        else:
            st = b.raw_status("snack_lora_fwd", ctypes.byref(bank), 0, 1 << 20, T, 1 << 40, 8, None,
                              8, 1 << 44, 8, None, *args)
        assert st == -10


@gpu
@pytest.mark.parametrize("backward", [False, True])
def test_the_most_tokens(backward):
    """All tokens a launch holds, some rows nonzero: 8 features, rank 2."""
    T, K, M, R = MOST[backward], 8, 8, 2
    rows = torch.tensor([0, 77, T // 2 + 31, T - 2 ** 20, T - 33, T - 1], device="cuda")
    s = make(rows.numel(), K, M, 1, R, "bf16", seed=2, ids="0", ranks=False)
    s["base"], s["gbase"] = torch.zeros_like(s["base"]), torch.zeros_like(s["gbase"])
    ref, tol = reference(s, "bf16", grads=True)

    def spread(v):
        w = torch.zeros(T, v.shape[1], dtype=v.dtype, device="cuda")
        w[rows] = v
        return w

    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    args = (ids, s["A"], s["B"], s["scale"])
    x = spread(s["x"])
    if backward:
        dx, dA, dB = snk.lora_bwd(spread(s["dy"]), x, *args)
        close(dx[rows], ref["dx"], tol["dx"], "dx")
        close(dA, ref["dA"], tol["dA"], "dA")
        close(dB, ref["dB"], tol["dB"], "dB")
        out = dx
    else:
        out = snk.lora_fwd(x, *args)
        close(out[rows], ref["y"], tol["y"], "y")
    out[rows] = 0
    assert int(out.view(-1, 2 ** 20).any(1).sum()) == 0  # all others


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_binding_and_torch_calls_agree(dt):
    """The binding's own calls, bit for bit, with all arguments and with few."""
    T, K, M, L, R = 90, 24, 40, 3, 8
    s = make(T, K, M, L, R, dt, seed=1)
    args = (s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    lora = b.snack_lora(s["A"], s["B"], M, K, L, R, s["scale"], s["ranks"])
    code = b._dtype(s["x"])

    def ws(backward):
        return torch.empty(b.snack_lora_workspace(lora, code, T, backward), dtype=torch.uint8,
                           device="cuda")

    y, t = torch.empty_like(s["base"]), torch.empty(T, R, device="cuda")
    b.snack_lora_fwd(lora, s["ids"], T, s["x"], K, s["base"], M, y, M, t=t, ws=ws(False))
    want_t = torch.empty_like(t)
    assert torch.equal(y, snk.lora_fwd(*args, s["base"], t=want_t)) and torch.equal(t, want_t)
    dx, dA, dB = torch.empty_like(s["x"]), torch.empty_like(s["A"]), torch.empty_like(s["B"])
    b.snack_lora_bwd(lora, s["ids"], t, T, s["x"], K, s["dy"], M, s["gbase"], K, dx, K, dA, dB,
                     ws=ws(True))
    want = snk.lora_bwd(s["dy"], *args, t=t, base=s["gbase"])
    assert all(torch.equal(p, q) for p, q in zip((dx, dA, dB), want))
    b.snack_lora_bwd(lora, s["ids"], None, T, s["x"], K, s["dy"], M, None, K, None, K, dB=dB,
                     ws=ws(True))
    assert torch.equal(dB, snk.lora_bwd(s["dy"], *args, want=(False, False, True))[2])


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,R", [(5, 16), (100, 16), (100, 40), (3000, 16)])
def test_sums_next_to_the_largest_float(T, R, dt):
    """t and u of 2^128 - 2^118, which rounds to infinity in bf16: beside small
    factors the results are finite."""
    K = M = 136
    s = make(T, K, M, 1, R, dt, seed=T + R, ids="0", ranks=False)
    s["scale"] = torch.ones(1, device="cuda")
    s["base"], s["gbase"] = torch.zeros_like(s["base"]), torch.zeros_like(s["gbase"])
    steps = torch.zeros(K, device="cuda")
    steps[:10] = 2.0 ** (63 - torch.arange(10, device="cuda", dtype=torch.float32))
    for a, f in (("x", "A"), ("dy", "B")):  # sum over the features: 2^127 + ... + 2^118
        v = dict(s)
        v[a] = torch.full_like(s[a], 2.0 ** 64)
        v[f] = torch.zeros_like(s[f])
        v[f][0, 3], v[f][0, R - 1] = steps, -steps
        other, small = ("B", "dy") if a == "x" else ("A", "x")
        v[other], v[small] = (s[other] * 2.0 ** -100).to(s[a].dtype), (s[small] * 2.0 ** -120).to(s[a].dtype)
        ref, tol = reference(v, dt, grads=True)
        args = (v["ids"], v["A"], v["B"])
        if a == "x":
            t = torch.empty(T, R, device="cuda")
            close(snk.lora_fwd(v["x"], *args, t=t), ref["y"], tol["y"], "y")
            assert float(t.abs().max()) == 2.0 ** 128 - 2.0 ** 118
            for kept in (t, None):
                dB = snk.lora_bwd(v["dy"], v["x"], *args, t=kept, want=(False, False, True))[2]
                close(dB, ref["dB"], tol["dB"], "dB")
        else:
            dx, dA, _ = snk.lora_bwd(v["dy"], v["x"], *args, want=(True, True, False))
            close(dx, ref["dx"], tol["dx"], "dx")
            close(dA, ref["dA"], tol["dA"], "dA")


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("width", [136, 200, 648])
@pytest.mark.parametrize("case", [(20, 1, 16, [16]), (90, 1, 16, [9]), (300, 3, 16, [16, 5, 11]),
                                  (3000, 2, 16, [13, 16]), (200, 2, 40, [33, 40])], ids=str)
def test_infinities_in_the_factors(case, width, dt):
    """Infinities of both signs and a NaN in factors that tokens use: the
    columns that they lie in are the formula's, all others finite."""
    T, L, R, ranks = case
    s = make(T, width, width, L, R, dt, seed=T + width, ids="runs", ranks=False)
    s["ids"][2] = -1
    s["ranks"] = torch.tensor(ranks, dtype=torch.int32, device="cuda")
    inf, nan = float("inf"), float("nan")
    for f in ("A", "B"):  # the last rank of the first adapter, the first ranks of the last one
        s[f][0, ranks[0] - 1, 7], s[f][0, 1, width - 1] = inf, -inf
        s[f][L - 1, 0, 9], s[f][L - 1, 2, 64], s[f][L - 1, 1, 66] = -inf, inf, nan
        s[f][L - 1, 0, 70], s[f][L - 1, 1, 70] = inf, -inf
    cols = [7, 9, 64, 66, 70, width - 1]

    def formula(v, F, base):
        want = base.double().cpu().clone()
        F, scale, ids = F.double().cpu(), s["scale"].double().cpu(), s["ids"].cpu()
        for l, r in enumerate(ranks):
            rows = ids == l
            want[rows] += scale[l] * (v[rows, :r, None] * F[l, :r]).sum(1)
        return want

    # t of x by the factor without infinities, and so u of dy
    clean = {f: torch.where(torch.isfinite(s[f]), s[f], torch.zeros_like(s[f])) for f in ("A", "B")}
    for name, got, want, v in (
            ("y", snk.lora_fwd(s["x"], s["ids"], clean["A"], s["B"], s["scale"], s["ranks"],
                               s["base"]), "B", "x"),
            ("dx", snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], clean["B"], s["scale"],
                                s["ranks"], base=s["gbase"], want=(True, False, False))[0], "A", "dy")):
        c = dict(s, **clean)
        if name == "dx":
            c = dict(c, x=s["dy"], A=clean["B"], B=clean["A"], base=s["gbase"])
        ref, tol = reference(c, dt)
        full = formula(ref["t"], s[want], c["base"])
        same_pattern(got, full, ref["y"], tol["y"], name)
        assert torch.isfinite(got[:, [k for k in range(width) if k not in cols]]).all()
