"""Low-rank adapters beside a shared projection against their formulas in 64
bits: forward and gradients at odd sizes, ranks, strides and alignments, rows
without an adapter, adapters without a row, and the refusals.

Tolerances, with e = 2^-24 (half a step of fp32 relative to the value), h =
2^-8 (of bf16) and S the sum of the terms' magnitudes:
  t   n e S for chains of at most n = K/4 + 64 additions (the kernels split a
      row at least eightfold);
  y   what the error of t carries, (R + 4) e S for the products and sums of
      the expansion, 2^-16 S where t is fed to the matrix cores as two bf16
      parts, and the output's rounding, e or h of the value;
  gradients alike, with chains of at most T additions."""
import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b

E = 2.0 ** -24
SPLIT = {"f32": 0.0, "bf16": 2.0 ** -16}
ROUND = {"f32": E, "bf16": 2.0 ** -8}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
gpu = pytest.mark.gpu


def make(T, K, M, L, R, dt, seed=0, ids="mixed", ranks=True, dev="cuda"):
    """Inputs on the device; adapters' rows past their rank hold NaN."""
    g = torch.Generator().manual_seed(seed)

    def n(*shape, std=1.0):
        return (torch.randn(*shape, generator=g) * std).to(DT[dt])

    s = dict(x=n(T, K), A=n(L, R, K, std=K ** -0.5), B=n(L, R, M, std=0.3), dy=n(T, M),
             base=n(T, M), gbase=n(T, K), scale=torch.rand(L, generator=g) + 0.5)
    if ids == "mixed":
        s["ids"] = torch.randint(-1, L, (T,), generator=g).int()
    elif ids == "runs":
        s["ids"] = torch.sort(torch.randint(0, L, (T,), generator=g)).values.int().flip(0)
    else:
        s["ids"] = torch.full((T,), int(ids), dtype=torch.int32)
    s["ranks"] = torch.randint(0, R + 1, (L,), generator=g).int() if ranks else None
    if ranks:
        s["ranks"][L // 2] = R
        for l in range(L):
            s["A"][l, s["ranks"][l]:] = float("nan")
            s["B"][l, s["ranks"][l]:] = float("nan")
    return {k: v.to(dev) if v is not None else None for k, v in s.items()}


def reference(s, dt, grads=False):
    """The formulas in 64 bits on the CPU, and each output's tolerance."""
    c = {k: v.double().cpu() if v is not None and v.is_floating_point() else
         (v.cpu() if v is not None else None) for k, v in s.items()}
    x, A, B, ids = c["x"], c["A"], c["B"], c["ids"]
    (T, K), (L, R, M) = x.shape, B.shape
    out = {k: torch.zeros(*v, dtype=torch.float64) for k, v in dict(
        t=(T, R), y=(T, M), dx=(T, K), dA=(L, R, K), dB=(L, R, M)).items()}
    tol = {k: torch.zeros_like(v) for k, v in out.items()}
    out["y"] += c["base"]
    out["dx"] += c["gbase"]
    tol["y"] += (R + 4) * E * c["base"].abs()
    tol["dx"] += (R + 4) * E * c["gbase"].abs()
    nK, nM, sp = K / 4 + 64, M / 4 + 64, SPLIT[dt]
    for l in range(L):
        rows = (ids == l).nonzero()[:, 0]
        r = int(c["ranks"][l]) if c["ranks"] is not None else R
        if rows.numel() == 0 or r == 0:
            continue
        a, bb, sc, xl, g = A[l, :r], B[l, :r], float(c["scale"][l]), x[rows], c["dy"][rows]
        t, u = xl @ a.t(), g @ bb.t()
        et, eu = nK * E * (xl.abs() @ a.abs().t()), nM * E * (g.abs() @ bb.abs().t())
        out["t"][rows, :r], tol["t"][rows, :r] = t, et
        out["y"][rows] += sc * (t @ bb)
        tol["y"][rows] += sc * ((et + ((R + 4) * E + sp) * t.abs()) @ bb.abs())
        if grads:
            out["dx"][rows] += sc * (u @ a)
            tol["dx"][rows] += sc * ((eu + ((R + 4) * E + sp) * u.abs()) @ a.abs())
            out["dA"][l, :r] = sc * (u.t() @ xl)
            out["dB"][l, :r] = sc * (t.t() @ g)
            n = T + 4
            tol["dA"][l, :r] = sc * ((eu + (n * E + sp) * u.abs()).t() @ xl.abs())
            tol["dB"][l, :r] = sc * ((et + (n * E + sp) * t.abs()).t() @ g.abs())
    for k in ("y", "dx", "dA", "dB"):
        tol[k] += ROUND[dt] * (out[k].abs() + tol[k])
    return out, tol


def close(got, ref, tol, what):
    got = got.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol + 1e-37)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"got {got[i]} ref {ref[i]} tol {tol[i]}")


# (T, K, M, L, R): one token, few, tiles that end inside, wide and odd everything
SIZES = [(1, 64, 64, 1, 1), (1, 257, 100, 5, 16), (2, 1, 1, 2, 3), (3, 4096, 520, 4, 16),
         (7, 33, 1001, 3, 17), (17, 512, 129, 70, 8), (40, 136, 2049, 3, 64), (63, 100, 7, 2, 5),
         (64, 128, 128, 1, 16), (65, 129, 136, 1, 33), (130, 1001, 257, 4, 12),
         (200, 264, 640, 16, 64), (300, 72, 200, 70, 100), (515, 48, 1030, 3, 256),
         (1500, 200, 96, 2, 16), (2111, 40, 72, 9, 24)]


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, dt):
    s = make(*size, dt, seed=sum(size))
    ref, tol = reference(s, dt)
    t = torch.full((size[0], size[4]), float("nan"), device="cuda")
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"], s["base"], t=t)
    close(t, ref["t"], tol["t"], "t")
    close(y, ref["y"], tol["y"], "y")
    # the same without t, into the base itself
    z = s["base"].clone()
    assert snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"], z, out=z) is z
    close(z, ref["y"], tol["y"], "y in place")


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradients(size, dt):
    s = make(*size, dt, seed=sum(size) + 1)
    ref, tol = reference(s, dt, grads=True)
    args = (s["dy"], s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    t = torch.empty(size[0], size[4], device="cuda")
    snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"], t=t)
    for kept in (None, t):
        dx, dA, dB = snk.lora_bwd(*args, t=kept, base=s["gbase"])
        close(dx, ref["dx"], tol["dx"], "dx")
        close(dA, ref["dA"], tol["dA"], "dA")
        close(dB, ref["dB"], tol["dB"], "dB")
    z = s["gbase"].clone()
    one = snk.lora_bwd(*args, base=z, out=z, want=(True, False, False))
    assert one[0] is z and one[1] is None and one[2] is None
    assert torch.equal(z, dx)
    assert torch.equal(snk.lora_bwd(*args, t=t, want=(False, True, False))[1], dA)
    assert torch.equal(snk.lora_bwd(*args, t=t, want=(False, False, True))[2], dB)


# More tokens than a workgroup sorts itself, more adapters than it counts, and
# long or lopsided runs of one adapter, whose gradients are summed in parts.
MANY = [(9000, 40, 72, 3, 8, "mixed"), (8300, 72, 40, 40, 20, "runs"), (20011, 24, 136, 5, 40, "1"),
        (300, 48, 64, 1500, 4, "mixed"), (100, 16, 24, 8192, 3, "mixed"),
        (2500, 264, 80, 9, 24, "4"), (8192, 64, 64, 2, 16, "mixed"), (6000, 136, 264, 1, 40, "0")]


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", MANY, ids=str)
def test_many_tokens_and_many_adapters(size, dt):
    *sizes, order = size
    s = make(*sizes, dt, seed=sum(sizes), ids=order)
    s["ids"][5] = -1
    ref, tol = reference(s, dt, grads=True)
    args = (s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    t = torch.full((sizes[0], sizes[4]), float("nan"), device="cuda")
    y = snk.lora_fwd(s["x"], *args, s["base"], t=t)
    close(t, ref["t"], tol["t"], "t")
    close(y, ref["y"], tol["y"], "y")
    for kept in (t, None):
        got = snk.lora_bwd(s["dy"], s["x"], *args, t=kept, base=s["gbase"])
        for k, v in zip(("dx", "dA", "dB"), got):
            close(v, ref[k], tol[k], k)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("K,M", [(3, 200), (200, 3), (7, 7), (8, 9), (63, 65), (127, 130), (66, 191)])
@pytest.mark.parametrize("T", [2, 90, 260])
def test_narrow_features(T, K, M, dt):
    """Rows shorter than a piece or a block, and last pieces and blocks that
    overlap the ones before them."""
    s = make(T, K, M, 2, 20, dt, seed=T + K + M)
    ref, tol = reference(s, dt, grads=True)
    args = (s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    z = s["base"].clone()
    snk.lora_fwd(s["x"], *args, z, out=z)
    close(z, ref["y"], tol["y"], "y in place")
    g = s["gbase"].clone()
    _, dA, dB = snk.lora_bwd(s["dy"], s["x"], *args, base=g, out=g)
    for k, v in (("dx", g), ("dA", dA), ("dB", dB)):
        close(v, ref[k], tol[k], k)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,R,r", [(3, 8, 5), (100, 16, 9), (100, 64, 33), (600, 40, 24)])
def test_infinity_in_the_last_rank(T, R, r, dt):
    """A rank count inside a step of the products: what stands in for the ranks
    past it adds nothing, not even to an infinite sum."""
    s = make(T, 72, 80, 1, R, dt, seed=T + r, ids="0", ranks=False)
    s["ranks"] = torch.tensor([r], dtype=torch.int32, device="cuda")
    s["A"], s["x"] = s["A"].abs() + 0.01, s["x"].abs() + 0.01
    s["B"][0, r - 1, 7] = float("inf")
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"], s["base"])
    assert (y[:, 7] == float("inf")).all()
    keep = torch.arange(80, device="cuda") != 7
    assert torch.isfinite(y[:, keep]).all()


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("ids", ["runs", "0", "-1", "2"])
@pytest.mark.parametrize("T", [5, 700])
def test_orders_of_tokens(T, ids, dt):
    s = make(T, 160, 144, 3, 20, dt, seed=T, ids=ids, ranks=False)
    s["scale"] = torch.tensor([0.5, 2.0, 1.0], device="cuda")
    ref, tol = reference(s, dt, grads=True)
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], None, s["base"])
    close(y, ref["y"], tol["y"], "y")
    dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], s["scale"], None,
                              base=s["gbase"])
    for k, v in (("dx", dx), ("dA", dA), ("dB", dB)):
        close(v, ref[k], tol[k], k)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,L", [(3, 2), (90, 2), (90, 1), (1100, 4), (1100, 1)])
def test_rows_without_adapter_keep_their_base(T, L, dt):
    """NaN and infinities in rows without an adapter, and in adapters without a
    row, reach nothing else; base alone, bit for bit, comes out."""
    s = make(T, 96, 80, L, 16, dt, seed=T, ranks=False)
    s["ids"][::3] = -1
    if L > 1:
        s["ids"][s["ids"] == 1] = 0
        s["A"][1], s["B"][1] = float("inf"), float("nan")
    off = s["ids"] < 0
    clean = {k: v.clone() if v is not None else None for k, v in s.items()}
    s["x"][off], s["dy"][off] = float("inf"), float("nan")
    clean["x"][off] = clean["dy"][off] = 0
    if L > 1:
        clean["A"][1] = clean["B"][1] = 0
    ref, tol = reference(clean, dt, grads=True)
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], None, s["base"])
    close(y, ref["y"], tol["y"], "y")
    assert torch.equal(y[off], s["base"][off])
    assert (snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"])[off] == 0).all()
    dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], s["scale"], None,
                              base=s["gbase"])
    assert torch.equal(dx[off], s["gbase"][off])
    for k, v in (("dx", dx), ("dA", dA), ("dB", dB)):
        close(v, ref[k], tol[k], k)


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [4, 200, 1200])
def test_infinite_inputs_stay_in_their_row(T, dt):
    s = make(T, 64, 64, 1, 16, dt, seed=T, ids="0", ranks=False)
    s["A"], s["B"] = s["A"].abs() + 0.1, s["B"].abs() + 0.1
    s["x"][1, 5] = float("inf")
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], None, s["base"])
    assert (y[1] == float("inf")).all()
    keep = torch.arange(T, device="cuda") != 1
    assert torch.isfinite(y[keep]).all()


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,L", [(6, 3), (150, 3), (150, 1), (1030, 3)])
def test_ids_past_the_last_adapter_read_nothing(T, L, dt):
    s = make(T, 40, 72, L, 4, dt, seed=T, ranks=False)
    s["ids"][1], s["ids"][T - 2] = L, 2 ** 31 - 1
    s["ids"][2] = -2 ** 31
    ref, tol = reference(s, dt, grads=True)
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], s["scale"], None, s["base"])
    dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], s["scale"], None,
                              base=s["gbase"])
    wrong = s["ids"] >= L
    assert torch.isnan(y[wrong]).all() and torch.isnan(dx[wrong]).all()
    ok = (~wrong).cpu()
    close(y[~wrong], ref["y"][ok], tol["y"][ok], "y")
    close(dx[~wrong], ref["dx"][ok], tol["dx"][ok], "dx")
    close(dA, ref["dA"], tol["dA"], "dA")
    close(dB, ref["dB"], tol["dB"], "dB")


@gpu
@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 9, 150, 1111])
def test_strided_and_unaligned_rows(T, dt):
    """Rows inside wider buffers, from an odd column on: read and written there
    and nowhere else."""
    K, M = 152, 136
    s = make(T, K, M, 3, 16, dt, seed=T)
    ref, tol = reference(s, dt, grads=True)

    def inside(v, left, right):
        w = torch.full((v.shape[0], left + v.shape[1] + right), 7.0, dtype=v.dtype, device="cuda")
        w[:, left:left + v.shape[1]] = v
        return w, w[:, left:left + v.shape[1]]

    _, x = inside(s["x"], 1, 2)
    _, dy = inside(s["dy"], 3, 0)
    wy, y = inside(s["base"], 5, 4)
    wx, dx = inside(s["gbase"], 1, 1)
    snk.lora_fwd(x, s["ids"], s["A"], s["B"], s["scale"], s["ranks"], base=y, out=y)
    close(y, ref["y"], tol["y"], "y")
    assert (wy[:, :5] == 7).all() and (wy[:, 5 + M:] == 7).all()
    _, dA, dB = snk.lora_bwd(dy, x, s["ids"], s["A"], s["B"], s["scale"], s["ranks"], base=dx,
                             out=dx)
    assert (wx[:, :1] == 7).all() and (wx[:, 1 + K:] == 7).all()
    for k, v in (("dx", dx), ("dA", dA), ("dB", dB)):
        close(v, ref[k], tol[k], k)
    # inputs whose rows do not lie contiguous are copied first
    z = snk.lora_fwd(s["x"].t().contiguous().t(), s["ids"], s["A"], s["B"], s["scale"],
                     s["ranks"], s["base"].t().contiguous().t())
    close(z, ref["y"], tol["y"], "transposed")


@gpu
@pytest.mark.parametrize("T", [6, 900])
def test_gradients_are_the_differences(T):
    """f is linear in x, in A and in B: <dy, f(. + d) - f(.)> is <grad, d>
    (64-bit formula for f, the library's gradients)."""
    s = make(T, 40, 56, 3, 8, "f32", seed=3)
    dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    _, tol = reference(s, "f32", grads=True)
    g = torch.Generator().manual_seed(9)
    f0 = reference(s, "f32")[0]["y"]
    for k, grad in (("x", dx), ("A", dA), ("B", dB)):
        d = torch.randint(-1, 2, s[k].shape, generator=g).double()
        moved = dict(s)
        moved[k] = s[k].double() + d.cuda()
        diff = ((reference(moved, "f32")[0]["y"] - f0) * s["dy"].double().cpu()).sum()
        t = tol["d" + k if k != "x" else "dx"].sum()
        assert abs(float((grad.double().cpu() * d).sum() - diff)) <= float(t) + 1e-9, k


@gpu
@pytest.mark.parametrize("T", [0, 5])
def test_no_tokens_and_no_rank(T):
    s = make(T, 24, 32, 2, 4, "f32", ranks=False)
    s["ranks"] = torch.zeros(2, dtype=torch.int32, device="cuda")
    y = snk.lora_fwd(s["x"], s["ids"], s["A"], s["B"], ranks=s["ranks"], base=s["base"])
    assert torch.equal(y, s["base"])
    dx, dA, dB = snk.lora_bwd(s["dy"], s["x"], s["ids"], s["A"], s["B"], ranks=s["ranks"])
    assert dx.shape == (T, 24) and (dx == 0).all() and (dA == 0).all() and (dB == 0).all()


@gpu
@pytest.mark.parametrize("T", [3, 200, 2500])
def test_same_bits_again_and_on_another_stream(T):
    s = make(T, 520, 264, 5, 16, "bf16", seed=4)
    args = (s["ids"], s["A"], s["B"], s["scale"], s["ranks"])
    y = snk.lora_fwd(s["x"], *args, s["base"])
    g = snk.lora_bwd(s["dy"], s["x"], *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y2 = snk.lora_fwd(s["x"], *args, s["base"])
        g2 = snk.lora_bwd(s["dy"], s["x"], *args)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, y2)
    assert all(torch.equal(p, q) for p, q in zip(g, g2))


@gpu
@pytest.mark.parametrize("T,L", [(4, 3), (600, 3), (600, 1)])
def test_captured_into_a_graph(T, L):
    s = make(T, 128, 192, L, 16, "bf16", seed=5, ranks=False)
    args = (s["ids"], s["A"], s["B"], s["scale"], None)
    out = torch.empty(T, 192, dtype=torch.bfloat16, device="cuda")
    t = torch.empty(T, 16, device="cuda")

    def step():
        snk.lora_fwd(s["x"], *args, s["base"], out=out, t=t)
        grads = snk.lora_bwd(out, s["x"], *args, t=t, base=s["gbase"])
        norm = snk.clip_grads(grads[1:], 0.5)
        return grads, norm

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_grads, g_norm = step()
    for k in range(4):
        s["x"].copy_(make(T, 128, 192, L, 16, "bf16", seed=50 + k)["x"])
        s["ids"].copy_(make(T, 128, 192, L, 16, "bf16", seed=60 + k)["ids"])
        graph.replay()
        torch.cuda.synchronize()
        y = out.clone()
        got = [v.clone() for v in (*g_grads, g_norm)]
        grads, norm = step()
        torch.cuda.synchronize()
        assert torch.equal(y, out)
        for p, q in zip(got, (*grads, norm)):
            assert torch.equal(p, q)


@gpu
def test_offsets_past_32_bits():
    # rows: 70,000 x 32,768 elements; the adapters: 2,048 x 256 x 4,112
    T, K, M, R = 70000, 64, 72, 8
    buf = torch.zeros(T, 32768, dtype=torch.bfloat16, device="cuda")
    x = buf[:, 32768 - K:]
    x.copy_(torch.randn(T, K, device="cuda"))
    out = buf[:, :M]
    A = (torch.randn(2, R, K, device="cuda") * 0.1).bfloat16()
    B = (torch.randn(2, R, M, device="cuda") * 0.3).bfloat16()
    ids = (torch.arange(T, device="cuda") % 2).int()
    snk.lora_fwd(x, ids, A, B, out=out)
    tail = slice(T - 300, T)
    s = dict(x=x[tail], A=A, B=B, ids=ids[tail], scale=torch.ones(2), ranks=None,
             dy=out[tail], base=torch.zeros(300, M), gbase=torch.zeros(300, K))
    ref, tol = reference(s, "bf16")
    close(out[tail], ref["y"], tol["y"], "rows")
    dx, dA, dB = snk.lora_bwd(out, x, ids, A, B)
    u = out.double() @ B.double().flatten(0, 1).t()
    mine = torch.nn.functional.one_hot(ids.long(), 2).double().repeat_interleave(R, 1)
    ref_dA = ((u * mine).t() @ x.double()).view(2, R, K)
    assert float((dA.double() - ref_dA).norm() / ref_dA.norm()) < 2.0 ** -8
    del buf, x, out
    L, R, K = 2048, 256, 4112
    A = torch.zeros(L, R, K, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(L, R, 16, dtype=torch.bfloat16, device="cuda")
    A[L - 1], B[L - 1] = torch.randn(R, K, device="cuda") / 64, torch.randn(R, 16, device="cuda")
    for T in (2, 300):
        x = torch.randn(T, K, device="cuda").bfloat16()
        ids = torch.full((T,), L - 1, dtype=torch.int32, device="cuda")
        y = snk.lora_fwd(x, ids, A, B)
        one = dict(x=x, A=A[L - 1:], B=B[L - 1:], ids=torch.zeros(T, dtype=torch.int32),
                   scale=torch.ones(1), ranks=None, dy=y, base=torch.zeros(T, 16),
                   gbase=torch.zeros(T, K))
        ref, tol = reference(one, "bf16")
        close(y, ref["y"], tol["y"], "last adapter")


@gpu
def test_module_and_autograd():
    torch.manual_seed(0)
    m = snk.LoraAdapters(48, 40, 3, 8, ranks=[8, 2, 5])
    x = torch.randn(30, 48, device="cuda", requires_grad=True)
    base = torch.randn(30, 40, device="cuda", requires_grad=True)
    ids = torch.arange(30, device="cuda").int() % 4 - 1
    assert torch.equal(m(x, ids, base), base)  # B starts at zero
    with torch.no_grad():
        m.B.normal_()
        free = m(x, ids, base)
    y = m(x, ids, base)
    assert torch.equal(y, free)
    gy = torch.randn(30, 40, device="cuda")
    y.backward(gy)
    s = dict(x=x.detach(), A=m.A.detach(), B=m.B.detach(), ids=ids, scale=m.scale, ranks=m.ranks,
             dy=gy, base=base.detach(), gbase=torch.zeros(30, 48))
    ref, tol = reference(s, "f32", grads=True)
    close(y.detach(), ref["y"], tol["y"], "y")
    close(x.grad, ref["dx"], tol["dx"], "dx")
    close(m.A.grad, ref["dA"], tol["dA"], "dA")
    close(m.B.grad, ref["dB"], tol["dB"], "dB")
    assert torch.equal(base.grad, gy)
    m.A.requires_grad_(False)
    m.A.grad = m.B.grad = None
    m(x.detach(), ids).backward(gy)
    close(m.B.grad, ref["dB"], tol["dB"], "dB alone")
    assert m.A.grad is None


@gpu
def test_a_training_step_captured_into_a_graph():
    """Forward, backward and clipping of the module in one graph, with no eager
    graph of the same parameters alive while it is captured."""
    torch.manual_seed(1)
    m = snk.LoraAdapters(96, 80, 3, 8, dtype=torch.bfloat16)
    with torch.no_grad():
        m.B.normal_(std=0.1)
    x = torch.randn(200, 96, device="cuda").bfloat16()
    ids = torch.randint(-1, 3, (200,), device="cuda").int()
    gy = torch.randn(200, 80, device="cuda").bfloat16()

    def step():
        m(x, ids).backward(gy)
        norm = snk.clip_grad_norm_(m.parameters(), 0.5)
        return norm

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    m.zero_grad(set_to_none=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = step()
    kept = m.A.grad, m.B.grad
    for k in range(3):
        x.copy_(torch.randn(200, 96, device="cuda"))
        ids.copy_(torch.randint(-1, 3, (200,), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in (norm, *kept)]
        t = torch.empty(200, 8, device="cuda")
        snk.lora_fwd(x, ids, m.A.detach(), m.B.detach(), m.scale, t=t)
        _, dA, dB = snk.lora_bwd(gy, x, ids, m.A.detach(), m.B.detach(), m.scale, t=t)
        want = snk.clip_grads([dA, dB], 0.5)
        for p, q in zip(got, (want, dA, dB)):
            assert torch.equal(p, q), k


@gpu
def test_example():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(__file__), "..", "examples"))
    import adapters
    first, last = adapters.finetune(steps=30)
    assert last < 0.5 * first
    adapters.serve()


# ------------------------------------------------------------------ refusals
def raw_fwd(lora=None, dtype=1, ids=8, T=4, X=16, ldx=64, base=None, ldb=32, Y=32, ldy=32, t=None,
            ws=64, ws_bytes=1 << 30, **bank):
    k = dict(A=4096, B=8192, M=32, K=64, L=2, R=8)
    k.update(bank)
    lora = b.snack_lora(**k) if lora is None else lora
    import ctypes
    return b.raw_status("snack_lora_fwd", ctypes.byref(lora), dtype, ids, T, X, ldx, base, ldb, Y,
                        ldy, t, ws, ws_bytes, None)


def raw_bwd(dtype=1, ids=8, t=None, T=4, X=16, ldx=64, dY=32, lddy=32, base=None, ldb=64, dX=48,
            lddx=64, dA=None, dB=None, ws=64, ws_bytes=1 << 30, **bank):
    k = dict(A=4096, B=8192, M=32, K=64, L=2, R=8)
    k.update(bank)
    import ctypes
    return b.raw_status("snack_lora_bwd", ctypes.byref(b.snack_lora(**k)), dtype, ids, t, T, X, ldx,
                        dY, lddy, base, ldb, dX, lddx, dA, dB, ws, ws_bytes, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), -3), (dict(dtype=-1), -3), (dict(M=0), -2), (dict(K=0), -2), (dict(L=0), -2),
    (dict(L=8193), -2), (dict(R=0), -2), (dict(R=257), -2), (dict(T=-1), -2), (dict(A=None), -1),
    (dict(B=None), -1), (dict(ids=None), -1), (dict(X=None), -1), (dict(ws=None), -1),
    (dict(ldx=63), -2), (dict(ws_bytes=16), -9),
    (dict(M=2 ** 23 + 1, ldy=2 ** 24, lddy=2 ** 24), -10), (dict(T=2 ** 31 - 1), -10)])
def test_refusals_of_both(bad, status):
    assert raw_fwd(**{k: v for k, v in bad.items() if k != "lddy"}) == status
    assert raw_bwd(**{k: v for k, v in bad.items() if k != "ldy"}) == status


def test_refusals():
    assert raw_fwd(Y=None) == -1
    assert raw_fwd(ldy=31) == -2 and raw_fwd(base=128, ldb=31) == -2
    assert raw_fwd(Y=16) == -2                          # Y is X
    assert raw_fwd(base=32, ldb=40) == -2               # Y is base with another stride
    assert raw_bwd(dY=None) == -1 and raw_bwd(lddy=31) == -2 and raw_bwd(lddx=63) == -2
    assert raw_bwd(base=128, ldb=63) == -2
    assert raw_bwd(dX=16) == -2 and raw_bwd(dX=32) == -2
    assert raw_bwd(base=48, ldb=70) == -2
    assert raw_fwd(T=0, ids=None, X=None, Y=None, ws=None, ws_bytes=0) == 0
    assert b.raw_status("snack_lora_fwd", None, 1, 8, 4, 16, 64, None, 32, 32, 32, None, 64, 64,
                        None) == -1
    assert b.raw_status("snack_lora_workspace", None, 1, 4, 0, None) == -1
    with pytest.raises(snk.SnackError) as e:
        b.snack_lora_workspace(b.snack_lora(1, 1, 32, 64, 2, 500), b.F32, 4)
    assert e.value.status == -2


def test_workspace_grows_with_the_work():
    bank = b.snack_lora(4096, 8192, 4096, 4096, 64, 64)
    for back in (False, True):
        sizes = [b.snack_lora_workspace(bank, b.BF16, T, back) for T in (0, 1, 64, 4096, 65536)]
        assert sizes == sorted(sizes) and sizes[-1] < 1 << 31


def test_wrappers_refuse_cpu_tensors():
    x, ids = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(TypeError):
        snk.lora_fwd(x, ids, torch.zeros(1, 2, 8), torch.zeros(1, 2, 4))
    with pytest.raises(ValueError):
        snk.lora_fwd(x, ids, torch.zeros(1, 2, 8), torch.zeros(1, 3, 4))
    with pytest.raises(TypeError):
        snk.lora_fwd(x.half(), ids, torch.zeros(1, 2, 8).half(), torch.zeros(1, 2, 4).half())
    with pytest.raises(ValueError):
        snk.LoraAdapters(8, 8, 2, 4, ranks=[4, 5], device="cpu")
    with pytest.raises(ValueError):
        snk.LoraAdapters(8, 8, 2, 4, ranks=[4], device="cpu")


@gpu
def test_wrappers_refuse_what_does_not_fit():
    s = make(6, 24, 32, 2, 4, "f32", ranks=False)
    x, ids, A, B = s["x"], s["ids"], s["A"], s["B"]
    for bad in (dict(ids=ids.long()), dict(ids=ids[:5]), dict(ids=ids.cpu()),
                dict(scale=torch.ones(2, device="cuda").double()),
                dict(scale=torch.ones(3, device="cuda")),
                dict(ranks=torch.ones(2, device="cuda")), dict(base=s["base"][:, :31]),
                dict(out=torch.empty(6, 33, device="cuda")),
                dict(out=torch.empty(32, 6, device="cuda").t()),
                dict(out=torch.empty(1, 32, device="cuda").expand(6, 32)),
                dict(t=torch.empty(6, 5, device="cuda")), dict(x=x[:, :23]),
                dict(A=A.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            snk.lora_fwd(**{**dict(x=x, ids=ids, A=A, B=B), **bad})
    for bad in (dict(A=A.bfloat16()), dict(base=s["base"].bfloat16()), dict(B=B.cpu())):
        with pytest.raises(TypeError):
            snk.lora_fwd(**{**dict(x=x, ids=ids, A=A, B=B), **bad})
    with pytest.raises(ValueError):
        snk.lora_bwd(s["dy"][:5], x, ids, A, B)
    with pytest.raises(snk.SnackError):  # the output over the input
        sq = make(6, 24, 24, 2, 4, "f32", ranks=False)
        snk.lora_fwd(sq["x"], sq["ids"], sq["A"], sq["B"], out=sq["x"])
