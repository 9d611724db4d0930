"""Adapters where values, tensors or sizes are special: infinities and NaN in
the gradients, outputs that other tensors share, moves of the module between
types, sizes past what a launch holds.  Formulas and tolerances are those of
the adapters' other tests."""
import pytest
import torch

import unstructured_sparse_nn_amd as snk
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
