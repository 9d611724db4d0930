"""The embedding, its gradient, token log-probabilities and the logits'
gradient against their formulas in 64 bits.  Tolerances, with e = 2^-24 and
h = 2^-8 (of bf16 outputs):
  embedding  e + h of the value;
  gradient   (n + 4) e of the sum of magnitudes over a row's n tokens, one
             rounding with base, e + h;
  l = log sum exp(d), d = x - m: each term is off by (3 |d| + 4) e for its own
             exponential (the difference, the product with log2(e), that
             constant, the exponential's unit) and by as much again where its
             sum is scaled as the maximum grows, so weighted by the softmax
             (6 |d| + 8) e; a chain of V/256 + 64 additions, and the logarithm;
  logp       the difference's rounding, l's error, its own rounding;
  logits'    p is off by the error of its exponent and 4 e; at the target its
  gradient   difference from 1 by a rounding of that size too, 2 e of g."""
import ctypes

import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b

E = 2.0 ** -24
F, H = torch.float32, torch.bfloat16
ROUND = {F: 0.0, H: 2.0 ** -8}
TINY = 2.0 ** -125  # results below the normal range may come out as 0
gpu = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")
LOW = torch.finfo(F).min


def within(got, ref, tol, what=""):
    got, ref, tol = got.double().cpu(), ref.cpu(), tol.cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    bad = ~((got - ref).abs() <= tol + TINY) & ~torch.isnan(ref) & (got != ref)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside; first at {i}: "
                             f"got {got[i]} ref {ref[i]} tol {tol[i]}")


# -------------------------------------------------------------------- embedding
def ids_of(T, V, how, seed=0, wide=True):
    g = torch.Generator().manual_seed(seed)
    if how == "one":
        ids = torch.full((T,), V - 1)
    elif how == "few":
        ids = torch.randint(0, min(V, 3), (T,), generator=g)
    elif how == "text":
        ids = ((V + 1.0) ** torch.rand(T, generator=g).double()).long().sub(1).clamp(max=V - 1)
    else:
        ids = torch.randint(-2, V + (V > 3), (T,), generator=g)  # none, some, one past the end
    return (ids if wide else ids.int()).cuda()


def grad_formula(dy, ids, V, scale, base):
    ids, dy = ids.flatten().cpu().long(), dy.double().cpu().view(-1, dy.shape[-1])
    ok = (ids >= 0) & (ids < V)
    s = torch.zeros(V, dy.shape[1], dtype=torch.float64)
    a, n = s.clone(), torch.zeros(V, dtype=torch.float64)
    s.index_add_(0, ids[ok], dy[ok])
    a.index_add_(0, ids[ok], dy[ok].abs())
    n.index_add_(0, ids[ok], torch.ones(int(ok.sum()), dtype=torch.float64))
    b_ = torch.zeros_like(s) if base is None else base.double().cpu()
    ref = b_ + scale * s
    return ref, (n[:, None] + 4) * E * scale * a + E * ref.abs()


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("T,V,D,wide", [(1, 1, 1, True), (1, 7, 4096, False), (3, 5, 8, True),
                                        (37, 1000, 100, False), (5, 3, 9, True), (64, 9, 3, False),
                                        (1000, 300, 129, True), (257, 33, 1001, False)])
def test_lookup(T, V, D, wide, dt):
    g = torch.Generator().manual_seed(T)
    w = torch.randn(V, D, generator=g).to(dt).cuda()
    ids = ids_of(T, V, "mixed", T, wide)
    for scale in (1.0, 0.37, -2.5):
        y = snk.embed_fwd(ids, w, scale)
        i = ids.cpu().long()
        ref = w.cpu().double()[i.clamp(0, V - 1)] * float(torch.tensor(scale, dtype=F))
        ref[i < 0] = 0.0
        ref[i >= V] = NAN
        within(y, ref, 1.01 * (E + ROUND[dt]) * ref.abs().nan_to_num(), f"scale {scale}")
        if scale == 1.0:
            some = ids.long().clamp(0, V - 1) == ids
            assert torch.equal(y[some], w[ids[some].long()])


@gpu
@pytest.mark.parametrize("dt", [F, H])
def test_lookup_of_strided_tables_into_strided_rows(dt):
    for off, D in ((0, 24), (1, 24), (3, 31), (2, 5)):
        w = torch.randn(50, D + 9, device="cuda").to(dt)[:, off:off + D]
        ids = ids_of(40, 50, "text").view(8, 5)
        out = torch.full((8, 5, D + 4), 7.0, dtype=dt, device="cuda")
        y = out[..., 3:3 + D]
        assert snk.embed_fwd(ids, w, out=y) is y
        assert torch.equal(y, w[ids]) and (out[..., :3] == 7).all() and (out[..., 3 + D:] == 7).all()
        assert torch.equal(snk.embed_fwd(ids[:, ::2], w), w[ids[:, ::2]])


# one token, few, tiles that end inside, rows of many tokens, wide and odd
GRADS = [(0, 3, 8, "mixed"), (1, 1, 1, "one"), (1, 100, 33, "text"), (5, 7, 8, "few"),
         (31, 5, 40, "one"), (32, 64, 8, "one"), (33, 65, 129, "one"), (64, 3, 16, "few"),
         (65, 1000, 96, "mixed"), (97, 2, 5, "few"), (1000, 50, 100, "text"),
         (1024, 4, 264, "few"), (3000, 2000, 72, "text"), (4097, 513, 1001, "text"),
         (8192, 70000, 24, "mixed"), (2500, 1, 7, "one"), (5000, 140000, 8, "text"),
         (9000, 129, 48, "one")]


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("T,V,D,how", GRADS)
def test_gradient(T, V, D, how, dt):
    g = torch.Generator().manual_seed(T + V)
    dy = torch.randn(T, D, generator=g).to(dt).cuda()
    base = torch.randn(V, D, generator=g).to(dt).cuda()
    for wide in (True, False):
        ids = ids_of(T, V, how, T, wide)
        for bs in (None, base):
            ref, tol = grad_formula(dy, ids, V, 0.5, bs)
            tol = tol + 1.01 * ROUND[dt] * (ref.abs() + tol)
            dW = snk.embed_bwd(dy, ids, V, 0.5, base=bs)
            within(dW, ref, tol, f"dW, base {bs is not None}")
            assert torch.equal(dW, snk.embed_bwd(dy, ids, V, 0.5, base=bs))
    z = base.clone()
    assert snk.embed_bwd(dy, ids, V, 0.5, base=z, out=z) is z and torch.equal(z, dW)
    if V > 1 and how == "one":  # rows without a token: not a bit changes
        assert torch.equal(z[:-1], base[:-1])


@gpu
@pytest.mark.parametrize("dt", [F, H])
def test_gradient_of_strided_rows(dt):
    T, V = 300, 40
    for off, D in ((0, 24), (1, 33), (3, 8), (2, 5)):
        dy = torch.randn(T, D + 7, device="cuda").to(dt)[:, off:off + D]
        ids = ids_of(T, V, "text", off)
        ref, tol = grad_formula(dy, ids, V, 1.0, None)
        tol = tol + 1.01 * ROUND[dt] * (ref.abs() + tol)
        out = torch.full((V, D + 9), 7.0, dtype=dt, device="cuda")
        within(snk.embed_bwd(dy, ids, V, out=out[:, 5:5 + D]), ref, tol, "dW")
        assert (out[:, :5] == 7).all() and (out[:, 5 + D:] == 7).all()
        base = torch.randn(V, D + 1, device="cuda").to(dt)[:, 1:]
        ref, tol = grad_formula(dy, ids, V, 1.0, base)
        tol = tol + 1.01 * ROUND[dt] * (ref.abs() + tol)
        within(snk.embed_bwd(dy, ids, V, base=base, out=base), ref, tol, "in place")
        shaped = snk.embed_bwd(dy.reshape(3, 100, D), ids.view(3, 100), V)
        assert torch.equal(shaped, snk.embed_bwd(dy, ids, V))


@gpu
def test_infinities_and_nan_stay_in_their_rows():
    ids = ids_of(500, 60, "text", 3)
    ids[::7] = -1
    ids[3::50] = 60
    dy = torch.randn(500, 20, device="cuda")
    clean = snk.embed_bwd(dy, ids, 60)
    dy[::7] = NAN  # tokens of no row
    dy[3::50] = INF
    assert torch.equal(snk.embed_bwd(dy, ids, 60), clean)
    v = int(ids[ids < 60].max())
    dy[ids == v] = INF
    got = snk.embed_bwd(dy, ids, 60)
    assert (got[v] == INF).all()
    keep = torch.arange(60, device="cuda") != v
    assert torch.equal(got[keep], clean[keep])


@gpu
def test_tables_past_32_bits():
    V, D = 600000, 4096  # 2.5 * 10^9 elements
    w = torch.zeros(V, D, dtype=H, device="cuda")
    ids = torch.tensor([0, V - 1, 524288, 524289, V - 1], device="cuda")
    w[ids] = torch.arange(5.0, device="cuda").to(H)[:, None]
    y = snk.embed_fwd(ids, w)
    assert torch.equal(y, w[ids])
    dy = torch.randn(5, D, device="cuda").to(H)
    out = snk.embed_bwd(dy, ids, V, base=w, out=w)
    assert out is w
    within(w[ids[:4]], torch.stack([y[0].double() + dy[0].double(),
                                    y[1].double() + dy[1].double() + dy[4].double(),
                                    y[2].double() + dy[2].double(),
                                    y[3].double() + dy[3].double()]),
           2.0 ** -8 * 1.01 * (y[:4].double().abs() + 9), "rows")
    del out
    dW = snk.embed_bwd(dy, ids, V)
    assert int((dW != 0).any(1).sum()) == 4
    assert torch.equal(dW[524289], dy[3])


@gpu
def test_embedding_module():
    m = snk.TokenEmbedding(70, 24, scale=24 ** 0.5)
    ids = ids_of(90, 69, "mixed").view(9, 10)
    y = m(ids)
    assert y.shape == (9, 10, 24)
    gy = torch.randn_like(y)
    gy[ids >= 69] = 0
    y.backward(gy)
    ref, tol = grad_formula(gy, ids, 70, float(torch.tensor(24 ** 0.5, dtype=F)), None)
    within(m.weight.grad, ref, tol, "weight")
    # the gradient is the difference: the lookup is linear
    d = torch.randn(70, 24, device="cuda")
    real = ((ids >= 0) & (ids < 70))[..., None]
    lhs = torch.where(real, snk.embed_fwd(ids, d, m.scale).double() * gy.double(), 0.0).sum()
    rhs = (d.double() * m.weight.grad.double()).sum()
    # every product is off by 100 roundings at most (rows have under 96 tokens)
    scale = (torch.where(real, snk.embed_fwd(ids, d, m.scale).double() * gy.double(), 0.0)).abs().sum()
    assert abs(float(lhs - rhs)) <= 100 * E * float(scale)


# ------------------------------------------------------------ log-probabilities
def logits_of(T, V, dt, seed=0, std=3.0, wide=True, strided=0):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, V + strided, generator=g) * std).to(dt).cuda()[:, :V]
    t = torch.randint(-1, V, (T,), generator=g)
    return x, (t if wide else t.int()).cuda()


def logp_formula(x, t):
    """(logp, m, l, tolerances of logp and l) in 64 bits."""
    x, t = x.double().cpu(), t.cpu().long()
    V = x.shape[1]
    m = x.amax(1)
    d = x - m[:, None]
    w = d.exp()
    l = w.sum(1).log()
    p = w / w.sum(1, keepdim=True)
    part = torch.where(p > 0, p * (6 * d.abs() + 8), 0.0).sum(1)
    tol_l = E * (part + V / 256 + 64 + l.abs())
    dt_ = d.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    logp = torch.where(t < 0, 0.0, dt_ - l)
    return logp, m, l, tol_l + E * (dt_.abs() + logp.abs()), tol_l


SIZES = [(1, 1), (1, 2), (2, 7), (3, 8), (1, 100), (5, 1001), (4, 32000), (1, 128000), (3, 50001),
         (300, 257), (64, 1024), (65, 2047), (1100, 513), (2, 65537), (1025, 4099), (7, 8193)]


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("T,V", SIZES)
def test_logp(T, V, dt):
    for wide, strided in ((True, 0), (False, 3)):
        x, t = logits_of(T, V, dt, T + V, wide=wide, strided=strided)
        logp, norm = snk.logp_fwd(x, t)
        ref, m, l, tol, tol_l = logp_formula(x, t)
        assert torch.equal(norm[:, 0].double().cpu(), m)
        within(norm[:, 1], l, tol_l, "l")
        within(logp, ref, tol, "logp")
        again = snk.logp_fwd(x, t)
        assert torch.equal(again[0], logp) and torch.equal(again[1], norm)


def logp_grad_formula(x, t, g):
    logp, m, l, _, tol_l = logp_formula(x, t)
    xd, t, g = x.double().cpu(), t.cpu().long(), g.double().cpu()
    V = xd.shape[1]
    lp = (xd - m[:, None]) - l[:, None]
    p = lp.exp()
    off = E * ((xd - m[:, None]).abs() + 3 * lp.abs() + 8) + tol_l[:, None]
    one = torch.zeros_like(xd).scatter_(1, t.clamp(0, V - 1)[:, None], 1.0)
    at = torch.where(one > 0, -torch.expm1(lp), -p)
    g = torch.where(t < 0, 0.0, g)[:, None]
    ref = g * at
    return ref, (torch.where(p > 0, g.abs() * p * off, 0.0) + 5 * E * ref.abs()
                 + 2 * E * g.abs() * one)


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("T,V", SIZES)
def test_logits_gradient(T, V, dt):
    for wide, strided in ((True, 0), (False, 5)):
        x, t = logits_of(T, V, dt, T + V + 1, wide=wide, strided=strided)
        g = torch.randn(T, device="cuda")
        g[::3] = 0
        norm = snk.logp_fwd(x, t)[1]
        ref, tol = logp_grad_formula(x, t, g)
        tol = tol + 1.01 * ROUND[dt] * (ref.abs() + tol)
        dx = snk.logp_bwd(g, x, t, norm)
        within(dx, ref, tol, "dx")
        assert (dx[::3] == 0).all()
        wide_x = torch.full((T, V + 6), 7.0, dtype=dt, device="cuda")
        y = wide_x[:, 1:V + 1]
        y.copy_(x)
        assert snk.logp_bwd(g, y, t, norm, out=y) is y and torch.equal(y, dx)
        assert (wide_x[:, 0] == 7).all() and (wide_x[:, V + 1:] == 7).all()


@gpu
def test_a_sure_model_and_large_logits():
    """Sums of 1 and a little keep the steps of fp32 above 1, 2^-23: l is good to
    the absolute error of its sum, as logp_formula has it, and no further.  Logits
    that are large together lose nothing, for m and l are apart."""
    x = torch.zeros(4, 1000, device="cuda")
    x[:, 5] = torch.tensor([20.0, 30.0, 1e4, 40.0])
    x[3] += 12345.0
    t = torch.full((4,), 5, device="cuda")
    t[3] = 6
    g = torch.ones(4, device="cuda")
    logp, norm = snk.logp_fwd(x, t)
    want = logp_formula(x, t)
    within(logp, want[0], want[3], "logp")
    within(snk.logp_bwd(g, x, t, norm), *logp_grad_formula(x, t, g), "dx")


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("T,V", [(9, 100), (9, 3001), (9, 70001), (1200, 77)])
def test_masks_infinities_and_nan(T, V, dt):
    x, t = logits_of(T, V, dt, 5)
    t = t.clamp(min=0)
    t[0] = -5
    low = torch.finfo(dt).min
    x[1, ::2] = -INF           # half of a vocabulary is masked
    x[2] = -INF                # nothing is left
    x[3] = low                 # the type's lowest value everywhere: all alike
    x[4, 1:] = low             # and beside a finite one
    t[4] = 0
    x[5, V // 2] = NAN
    x[6, V - 1] = INF
    t[7] = V                   # past the end
    x[8, 1:] = -INF            # one is left, and not the target
    t[8] = V - 1
    logp, norm = snk.logp_fwd(x, t)
    ref, m, l, tol, tol_l = logp_formula(x, t)
    ref[2], m[2], l[2], ref[7] = -INF, LOW, -INF, NAN
    ref[5] = ref[6] = NAN
    for i in (2, 5, 6):
        tol[i] = tol_l[i] = 0
    fine = torch.ones(T, dtype=torch.bool)
    fine[5] = fine[6] = False
    within(logp, ref, tol.nan_to_num(), "logp")
    within(norm[:, 1].cpu()[fine], l[fine], tol_l[fine].nan_to_num(), "l")
    assert torch.isnan(norm[5, 1]) and torch.isnan(norm[6, 1])
    assert torch.equal(norm[:, 0].double().cpu()[fine], m[fine])
    g = torch.linspace(1, 2, T).cuda()
    dx = snk.logp_bwd(g, x, t, norm)
    rg, tg = logp_grad_formula(x, t, g)
    rg[2], tg[2] = 0, 0
    for i in (5, 6, 7):
        rg[i] = NAN
    tg = tg.nan_to_num() + 1.01 * ROUND[dt] * (rg.abs().nan_to_num() + tg.nan_to_num())
    within(dx, rg, tg, "dx")
    # rows that nothing flows into are zeros whatever they hold
    g[5] = g[6] = 0
    dx = snk.logp_bwd(g, x, t, norm)
    assert (dx[5] == 0).all() and (dx[6] == 0).all() and (dx[0] == 0).all()


@gpu
def test_extreme_logits():
    big = torch.finfo(F).max
    x = torch.tensor([[big, -big, 0.0, big], [1e30, 1e30 * (1 - 2.0 ** -23), 0.0, 0.0],
                      [-1e30, -1e30, -1e30, -2e30], [1e-40, 0.0, -1e-40, 0.0]], device="cuda")
    t = torch.tensor([0, 1, 2, 3], device="cuda")
    logp, norm = snk.logp_fwd(x, t)
    want = logp_formula(x, t)
    within(logp, want[0], want[3], "logp")
    g = torch.ones(4, device="cuda")
    ref, tol = logp_grad_formula(x, t, g)
    within(snk.logp_bwd(g, x, t, norm), ref, tol.nan_to_num(), "dx")


@gpu
def test_gradient_is_the_difference_and_autograd():
    x, t = logits_of(6, 50, F, 2)
    x = x.view(2, 3, 50).clone().requires_grad_(True)
    t = t.view(2, 3)
    logp = snk.token_logps(x, t)
    assert logp.shape == (2, 3) and logp.dtype == F
    logp.sum().backward()  # an expanded gradient
    h = 1e-5
    d = torch.randn(2, 3, 50, generator=torch.Generator().manual_seed(1)).double()
    up, down = (logp_formula((x.detach().double().cpu() + s * h * d).view(6, 50), t.view(-1))[0]
                for s in (1, -1))
    want = (up - down).sum() / (2 * h)
    got = (x.grad.double().cpu() * d).sum()
    # the difference is good to h^2 of a third derivative below |d|^3 <= 4^3
    assert abs(float(got - want)) <= 6 * h * h * 64 + 300 * 20 * E + 1e-9
    assert x.grad.shape == x.shape


@gpu
def test_offsets_past_32_bits():
    T, V = 20000, 128001  # 2.56 * 10^9 logits
    x = torch.zeros(T, V, dtype=H, device="cuda")
    x[-1, 7] = 3.0
    t = torch.full((T,), 7, device="cuda")
    logp, norm = snk.logp_fwd(x, t)
    want = logp_formula(x[-2:], t[-2:])
    within(logp[-2:], want[0], want[3], "logp")
    assert (logp[:-1] == logp[0]).all()
    g = torch.zeros(T, device="cuda")
    g[-1] = g[3] = 1.0
    snk.logp_bwd(g, x, t, norm, out=x)
    assert float(x[:-1].abs().sum(dtype=torch.float64)) > 0 and (x[4:-1] == 0).all()
    row = torch.zeros(2, V, dtype=H)
    row[1, 7] = 3.0
    ref, tol = logp_grad_formula(row, torch.tensor([7, 7]), torch.ones(2))
    within(x[[3, T - 1]], ref, tol + 1.01 * 2.0 ** -8 * ref.abs(), "dx")


@gpu
@pytest.mark.parametrize("V", [65536, 65541])
def test_gradients_past_128_megabytes(V):
    """Stored past the caches: the same bits as in parts that are not."""
    T = 1100
    x = (torch.randn(T, V, device="cuda") * 2).to(H)
    t = torch.randint(-1, V, (T,), device="cuda")
    g = torch.randn(T, device="cuda")
    norm = snk.logp_fwd(x, t)[1]
    whole = snk.logp_bwd(g, x, t, norm)
    for rows in (slice(0, 500), slice(500, T)):
        part = snk.logp_bwd(g[rows], x[rows], t[rows], norm[rows])
        assert torch.equal(whole[rows], part)
    assert torch.equal(snk.logp_bwd(g, x, t, norm, out=x), whole)


@gpu
@pytest.mark.parametrize("how", ["text", "one", "few", "mixed"])
def test_gradient_of_many_tokens(how):
    """More numbers than a wave lists, and rows of tens of thousands of tokens."""
    T, V, D = 150001, 5000, 16
    ids = ids_of(T, V, how, 1)
    dy = torch.randn(T, D, device="cuda")
    ref, tol = grad_formula(dy, ids, V, 1.0, None)
    within(snk.embed_bwd(dy, ids, V), ref, tol, how)


# --------------------------------------------------------------------- together
@gpu
def test_other_streams_graphs_and_the_binding():
    x, t = logits_of(70, 9001, H, 8)
    ids = ids_of(70, 50, "text", 4)
    w = torch.randn(50, 40, device="cuda")
    dy = torch.randn(70, 40, device="cuda")
    g = torch.randn(70, device="cuda")

    def all_of():
        logp, norm = snk.logp_fwd(x, t)
        return [logp, norm, snk.logp_bwd(g, x, t, norm), snk.embed_fwd(ids, w, 3.0),
                snk.embed_bwd(dy, ids, 50, 3.0, base=w)]

    want = all_of()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = all_of()
        all_of()
    s.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(want, other))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    for gr in graphs:  # two graphs, whose workspaces must not meet
        with torch.cuda.graph(gr):
            outs.append(all_of())
    for k in range(3):
        x.copy_(torch.randn(70, 9001, device="cuda"))
        dy.copy_(torch.randn(70, 40, device="cuda"))
        ids.copy_(ids.roll(3))
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        want = all_of()
        for o in outs:
            assert all(torch.equal(a, c) for a, c in zip(want, o)), k
    logp, norm = torch.empty(70, device="cuda"), torch.empty(70, 2, device="cuda")
    ws = torch.empty(snk.snack_logp_workspace(b.BF16, 70, 9001), dtype=torch.uint8, device="cuda")
    snk.snack_logp_fwd(x, 9001, 70, 9001, t, 8, logp, norm, ws)
    dx = torch.empty_like(x)
    snk.snack_logp_bwd(g, x, 9001, 70, 9001, t, 8, norm, dx, 9001)
    y, dW = torch.empty(70, 40, device="cuda"), torch.empty(50, 40, device="cuda")
    snk.snack_embed_fwd(ids, 8, 70, w, 40, 50, 40, 3.0, y, 40)
    ws = torch.empty(snk.snack_embed_workspace(b.F32, 70, 50, 40), dtype=torch.uint8, device="cuda")
    snk.snack_embed_bwd(ids, 8, 70, dy, 40, 50, 40, 3.0, w, 40, dW, 40, ws)
    assert all(torch.equal(a, c) for a, c in zip(want, [logp, norm, dx, y, dW]))


@gpu
def test_nothing_and_written_tensors():
    w = torch.randn(5, 8, device="cuda")
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    assert snk.embed_fwd(none, w).shape == (0, 8)
    assert (snk.embed_bwd(torch.empty(0, 8, device="cuda"), none, 5) == 0).all()
    z = w.clone()
    snk.embed_bwd(torch.empty(0, 8, device="cuda"), none, 5, base=z, out=z)
    assert torch.equal(z, w)
    assert snk.embed_bwd(torch.empty(0, 8, device="cuda"), none, 0).shape == (0, 8)
    assert (snk.embed_fwd(torch.tensor([-1, -7], device="cuda"), w[:0]) == 0).all()
    assert torch.isnan(snk.embed_fwd(torch.tensor([0, 2 ** 40], device="cuda"), w[:0])).all()
    logp, norm = snk.logp_fwd(w[:0], none)
    assert logp.shape == (0,) and norm.shape == (0, 2)
    assert snk.logp_bwd(logp, w[:0], none, norm).shape == (0, 8)
    ids = torch.tensor([1, 2], device="cuda")
    out = torch.empty(2, 8, device="cuda")
    v = out._version
    snk.embed_fwd(ids, w, out=out)
    assert out._version > v
    v = w._version
    snk.embed_bwd(out, ids, 5, base=w, out=w)
    assert w._version > v
    x, t = logits_of(2, 8, F)
    norm = snk.logp_fwd(x, t)[1]
    v = x._version
    snk.logp_bwd(torch.ones(2, device="cuda"), x, t, norm, out=x)
    assert x._version > v


EMBED = dict(dtype=0, ids=0x1000, id_bytes=8, T=7, W=0x10000, ldw=10, V=5, D=10, scale=1.0,
             Y=0x20000, ldy=10, stream=None)
EMBED_BWD = dict(dtype=0, ids=0x1000, id_bytes=8, T=7, dY=0x10000, lddy=10, V=5, D=10, scale=1.0,
                 base=0x30000, ldb=10, dW=0x20000, lddw=10, ws=0x100000, ws_bytes=1 << 20,
                 stream=None)
LOGP = dict(dtype=0, X=0x10000, ldx=10, T=7, V=10, targets=0x1000, id_bytes=8, logp=0x20000,
            norm=0x30000, ws=None, ws_bytes=0, stream=None)
LOGP_BWD = dict(dtype=0, dlogp=0x20000, X=0x10000, ldx=10, T=7, V=10, targets=0x1000, id_bytes=8,
                norm=0x30000, dX=0x40000, lddx=10, stream=None)


@pytest.mark.parametrize("name,args,bad,status", [
    (n, a, bad, st) for n, a, cases in (
        ("snack_embed_fwd", EMBED, [
            (dict(dtype=3), -3), (dict(id_bytes=2), -3), (dict(T=-1), -2), (dict(V=-1), -2),
            (dict(D=-1), -2), (dict(ldw=9), -2), (dict(ldy=9), -2), (dict(ids=None), -1),
            (dict(W=None), -1), (dict(Y=None), -1), (dict(Y=0x10004), -2), (dict(Y=0x1008), -2),
            (dict(T=(1 << 28) + 1), -10), (dict(V=(1 << 30) + 1), -10),
            (dict(D=(1 << 23) + 1, ldw=1 << 24, ldy=1 << 24), -10),
            (dict(T=1 << 28, D=128, ldw=128, ldy=128), -10)]),
        ("snack_embed_bwd", EMBED_BWD, [
            (dict(dtype=3), -3), (dict(id_bytes=5), -3), (dict(T=-1), -2), (dict(V=-1), -2),
            (dict(lddy=9), -2), (dict(ldb=9), -2), (dict(lddw=9), -2), (dict(dW=None), -1),
            (dict(ws=None), -1), (dict(dY=None), -1), (dict(ids=None), -1),
            (dict(ws_bytes=100), -9), (dict(dW=0x30000, ldb=11), -2), (dict(dW=0x30004), -2),
            (dict(dW=0x10000), -2), (dict(dW=0x1000), -2), (dict(ws=0x10000), -2),
            (dict(ws=0x20000), -2), (dict(ws=0x30000), -2), (dict(V=1 << 30, D=64, lddy=64, ldb=64,
                                                                  lddw=64), -10)]),
        ("snack_logp_fwd", LOGP, [
            (dict(dtype=3), -3), (dict(id_bytes=1), -3), (dict(T=-1), -2), (dict(V=0), -2),
            (dict(ldx=9), -2), (dict(X=None), -1), (dict(targets=None), -1), (dict(logp=None), -1),
            (dict(norm=None), -1), (dict(logp=0x10000), -2), (dict(norm=0x20008), -2),
            (dict(logp=0x1010), -2), (dict(V=(1 << 30) + 1, ldx=1 << 31), -10),
            (dict(T=1 << 24), -10), (dict(V=100000, ldx=100000), -1),
            (dict(V=100000, ldx=100000, ws=0x400000), -9)]),
        ("snack_logp_bwd", LOGP_BWD, [
            (dict(dtype=3), -3), (dict(id_bytes=1), -3), (dict(V=0), -2), (dict(lddx=9), -2),
            (dict(dlogp=None), -1), (dict(X=None), -1), (dict(targets=None), -1),
            (dict(norm=None), -1), (dict(dX=None), -1), (dict(dX=0x10000, lddx=11), -2),
            (dict(dX=0x10004), -2), (dict(dX=0x20000), -2), (dict(dX=0x30000), -2),
            (dict(dX=0x1000), -2), (dict(T=1 << 24), -10)]))
    for bad, st in cases])
def test_refusals(name, args, bad, status):
    a = dict(args, **bad)
    if "scale" in a:
        a["scale"] = ctypes.c_float(a["scale"])
    assert b.raw_status(name, *a.values()) == status


def test_workspaces():
    for what, args in ((snk.snack_embed_workspace, (b.F32, 10, 20, 30)),
                       (snk.snack_logp_workspace, (b.F32, 10, 20))):
        assert what(*args) >= 0
    with pytest.raises(snk.SnackError):
        snk.snack_embed_workspace(7, 1, 1, 1)
    with pytest.raises(snk.SnackError):
        snk.snack_logp_workspace(b.F32, 1, 0)
    # sums of rows with many tokens, two slots for every 32 at least
    assert snk.snack_embed_workspace(b.BF16, 6400, 10, 64) >= 2 * 200 * 64 * 4
    assert b.raw_status("snack_embed_workspace", 0, 1, 1, 1, None) == -1
    assert b.raw_status("snack_logp_workspace", 0, 1, 1, None) == -1


def test_wrappers_refuse_cpu_tensors():
    ids, w = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8)
    for call in (lambda: snk.embed_fwd(ids, w), lambda: snk.embed_bwd(torch.zeros(3, 8), ids, 4),
                 lambda: snk.logp_fwd(torch.zeros(3, 8), ids),
                 lambda: snk.logp_bwd(torch.zeros(3), torch.zeros(3, 8), ids, torch.zeros(3, 2))):
        with pytest.raises(TypeError, match="on the GPU"):
            call()


@gpu
def test_wrappers_refuse_what_does_not_fit():
    c = dict(device="cuda")
    ids, w, dy = torch.zeros(3, dtype=torch.int64, **c), torch.zeros(4, 8, **c), torch.zeros(3, 8, **c)
    x, g, norm = torch.zeros(3, 8, **c), torch.zeros(3, **c), torch.zeros(3, 2, **c)
    for kind, call in [
            (TypeError, lambda: snk.embed_fwd(ids.float(), w)),
            (TypeError, lambda: snk.embed_fwd(ids.cpu(), w)),
            (TypeError, lambda: snk.embed_fwd(ids, w.half())),
            (ValueError, lambda: snk.embed_fwd(ids, w[0])),
            (ValueError, lambda: snk.embed_fwd(ids, w, out=torch.zeros(3, 7, **c))),
            (TypeError, lambda: snk.embed_fwd(ids, w, out=torch.zeros(3, 8, **c).to(H))),
            (snk.SnackError, lambda: snk.embed_fwd(ids, w, out=w[:3])),
            (ValueError, lambda: snk.embed_bwd(dy[:2], ids, 4)),
            (ValueError, lambda: snk.embed_bwd(dy, ids, -1)),
            (ValueError, lambda: snk.embed_bwd(dy, ids, 4, base=torch.zeros(3, 8, **c))),
            (ValueError, lambda: snk.embed_bwd(dy, ids, 4, out=torch.zeros(1, 8, **c).expand(4, 8))),
            (snk.SnackError, lambda: snk.embed_bwd(dy, ids, 3, out=dy)),
            (TypeError, lambda: snk.logp_fwd(x, ids.float())),
            (ValueError, lambda: snk.logp_fwd(x, ids[:2])),
            (ValueError, lambda: snk.logp_fwd(x[:, :0], ids)),
            (TypeError, lambda: snk.logp_bwd(g.to(H), x, ids, norm)),
            (ValueError, lambda: snk.logp_bwd(g[:2], x, ids, norm)),
            (ValueError, lambda: snk.logp_bwd(g, x, ids, norm[:, :1])),
            (ValueError, lambda: snk.logp_bwd(g, x, ids, norm, out=torch.zeros(3, 9, **c)))]:
        with pytest.raises(kind):
            call()
