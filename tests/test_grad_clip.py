"""The norm over many gradients and their clipping against the formula in 64
bits.  Tolerances: the squares are exact and summed in 64 bits, so the norm is
off by its rounding to fp32, 2^-24; an output by the factor's and the
product's, 2 x 2^-24, and in bf16 by half a step more, 2^-8."""
import math

import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b

E = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}
gpu = pytest.mark.gpu


def grads_of(sizes, dtypes, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(dtypes[i % len(dtypes)]).cuda()
            for i, n in enumerate(sizes)]


def formula(grads, max_norm, eps=1e-6):
    norm = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    c = min(1.0, max_norm / (norm + eps))
    return norm, [g.double() * c for g in grads]


def check(got, norm, want, ref):
    if want > torch.finfo(torch.float32).max:  # the factor still comes from 64 bits
        assert float(norm) == float("inf")
    else:
        assert abs(float(norm) - want) <= 1.01 * E * want
    for o, r in zip(got, ref):
        tol = (2.02 * E + ROUND[o.dtype] * (1 + 3 * E)) * r.abs() + 2.0 ** -133
        assert ((o.double() - r).abs() <= tol).all()


F, H = torch.float32, torch.bfloat16
LISTS = [([1], [F]), ([0, 1, 0], [H]), ([0], [F]), ([5, 0, 8192, 8193, 7, 16384], [F, H]),
         ([100003], [H]), ([3] * 112, [F]), ([17] * 113, [H, F]), (list(range(300)), [H, F]),
         ([1000001, 2, 333333], [F, H, H]), ([4194304], [F]), ([20000] * 250, [H])]


@gpu
@pytest.mark.parametrize("max_norm", [0.25, 1e9, 0.0])
@pytest.mark.parametrize("which", range(len(LISTS)))
def test_clip(which, max_norm):
    grads = grads_of(*LISTS[which], seed=which)
    want, ref = formula(grads, max_norm)
    assert abs(float(snk.grad_norm(grads)) - want) <= 1.01 * E * want
    out = [torch.full_like(g, 7.0) for g in grads]
    before = [g.clone() for g in grads]
    norm = snk.clip_grads(grads, max_norm, out=out)
    check(out, norm, want, ref)
    assert all(torch.equal(g, w) for g, w in zip(grads, before))
    again = snk.clip_grads(grads, max_norm)
    assert torch.equal(again, norm)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))
    if max_norm == 1e9:  # below the limit: not a bit changes
        assert all(torch.equal(g, w) for g, w in zip(grads, before))


@gpu
@pytest.mark.parametrize("dtype", [F, H])
def test_views_of_a_bucket_at_any_alignment(dtype):
    sizes = [1, 2, 3, 5, 8191, 7, 8200, 40000, 1, 11]
    flat = grads_of([sum(sizes) + 2], [dtype], seed=3)[0]
    flat[0] = flat[-1] = 99.0
    grads = list(flat[1:-1].split(sizes))
    want, ref = formula(grads, 1.0)
    for shift in range(8):  # outputs aligned alike and otherwise
        wide = torch.full((sum(sizes) + 16,), 7.0, dtype=dtype, device="cuda")
        out = list(wide[shift:shift + sum(sizes)].split(sizes))
        norm = snk.clip_grads(grads, 1.0, out=out)
        check(out, norm, want, ref)
        assert (wide[:shift] == 7).all() and (wide[shift + sum(sizes):] == 7).all()
    norm = snk.clip_grads(grads, 1.0)
    check(grads, norm, want, ref)
    assert float(flat[0]) == 99.0 and float(flat[-1]) == 99.0


@gpu
def test_large_small_and_special_values():
    big = [torch.full((1000,), 3e37, device="cuda"), torch.full((9,), 1e38, device="cuda").to(H)]
    want, ref = formula(big, 1.0)
    norm = snk.clip_grads(big, 1.0)
    check(big, norm, want, ref)
    fits = [torch.full((30,), -3e37, device="cuda"), torch.full((9,), 5e37, device="cuda").to(H)]
    want, ref = formula(fits, 2.0)  # every square past fp32's range, the norm within it
    check(fits, snk.clip_grads(fits, 2.0), want, ref)
    tiny = [torch.full((100,), 1e-42, device="cuda")]
    assert abs(float(snk.grad_norm(tiny)) - float(tiny[0][0].double()) * 10) <= 2.0 ** -149
    zero = [torch.zeros(50, device="cuda"), torch.zeros(3, device="cuda", dtype=H)]
    assert float(snk.clip_grads(zero, 0.0)) == 0.0 and float(zero[0].abs().max()) == 0.0
    nan = [torch.ones(5, device="cuda"), torch.tensor([1.0, float("nan")], device="cuda")]
    assert math.isnan(float(snk.clip_grads(nan, 1.0)))
    assert all(torch.isnan(g).all() for g in nan)
    inf = [torch.ones(5, device="cuda"), torch.tensor([1.0, float("-inf")], device="cuda")]
    assert float(snk.clip_grads(inf, 1.0)) == float("inf")
    assert (inf[0] == 0).all() and float(inf[1][0]) == 0.0 and math.isnan(float(inf[1][1]))


@gpu
def test_more_than_2_to_the_31_elements():
    n = 2 ** 31 + 9
    g = torch.zeros(n, dtype=H, device="cuda")
    g[0], g[2 ** 31 + 1], g[-1] = 3.0, 4.0, 12.0
    small = torch.zeros(3, device="cuda")
    norm = snk.clip_grads([small, g], 6.5)
    assert abs(float(norm) - 13.0) <= 13.0 * E
    assert [float(g[i]) for i in (0, 2 ** 31 + 1, n - 1)] == [1.5, 2.0, 6.0]


@gpu
def test_dense_but_permuted_gradients_and_parameters():
    w = torch.nn.Parameter(torch.randn(6, 5, 4, device="cuda"))
    w.grad = torch.randn(6, 4, 5, device="cuda").transpose(1, 2)
    v = torch.nn.Parameter(torch.randn(7, device="cuda"))
    none = torch.nn.Parameter(torch.zeros(3, device="cuda"))
    v.grad = torch.randn(7, device="cuda")
    want, ref = formula([w.grad, v.grad], 0.5)
    version = w.grad._version
    norm = snk.clip_grad_norm_([w, none, v], 0.5)
    check([w.grad, v.grad], norm, want, ref)
    assert w.grad._version > version
    assert torch.equal(snk.grad_norm(w.grad for _ in range(1)), snk.grad_norm([w.grad]))


@gpu
def test_same_bits_again_and_on_another_stream():
    grads = grads_of([50000, 3, 700001], [F, H], seed=8)
    out = [torch.empty_like(g) for g in grads]
    norm = snk.clip_grads(grads, 1.0, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out2 = [torch.empty_like(g) for g in grads]
        norm2 = snk.clip_grads(grads, 1.0, out=out2)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(norm, norm2) and all(torch.equal(p, q) for p, q in zip(out, out2))


@gpu
def test_wrappers_refuse_what_does_not_fit():
    g = [torch.ones(4, 4, device="cuda"), torch.ones(3, device="cuda")]
    o = [torch.empty_like(x) for x in g]
    for bad in ([g[0].half()], [g[0].t()[:, ::2]], [torch.ones(1, device="cuda").expand(4)],
                [g[0], torch.ones(2)], [torch.ones(2)]):
        with pytest.raises((TypeError, ValueError)):
            snk.clip_grads(bad, 1.0)
        with pytest.raises((TypeError, ValueError)):
            snk.grad_norm(bad)
    for bad in (o[:1], [o[0], torch.empty(4, device="cuda")], [o[0], o[1].bfloat16()],
                [o[0].t(), o[1]]):
        with pytest.raises((TypeError, ValueError)):
            snk.clip_grads(g, 1.0, out=bad)
    for limit in (float("nan"), -1.0):
        with pytest.raises(snk.SnackError):
            snk.clip_grads(g, limit)


def test_nothing_to_clip():
    assert float(snk.grad_norm([])) == 0.0 and float(snk.clip_grads([], 1.0)) == 0.0
    assert float(snk.clip_grad_norm_([torch.nn.Parameter(torch.ones(2))], 1.0)) == 0.0
    with pytest.raises(ValueError):
        snk.clip_grads([], 1.0, out=[torch.ones(1)])


def test_refusals():
    from array import array
    tab = array("q", [4096, 4096, 10, 0])

    def clip(rows=tab, count=1, max_norm=1.0, eps=0.0, norm=64, ws=64, ws_bytes=1 << 20):
        return b.raw_status("snack_grad_clip", rows.buffer_info()[0] if rows else None, count,
                            max_norm, eps, norm, ws, ws_bytes, None)

    assert clip(count=-1) == -8 and clip(rows=None) == -1
    assert clip(max_norm=float("nan")) == -7 and clip(eps=float("nan")) == -7
    assert clip(max_norm=-1.0) == -2 and clip(eps=-1.0) == -2
    assert clip(ws=None) == -1 and clip(ws_bytes=8) == -9
    assert clip(rows=array("q", [4096, 4096, 10, 2])) == -3
    assert clip(rows=array("q", [4096, 4096, -1, 0])) == -2
    assert clip(rows=array("q", [0, 0, 10, 0])) == -1
    assert clip(rows=array("q", [4096, 4096, 2 ** 41, 0])) == -10
    assert b.raw_status("snack_grad_norm", tab.buffer_info()[0], 1, None, 64, 1 << 20, None) == -1
    assert b.raw_status("snack_grad_norm", tab.buffer_info()[0], 1, 64, 64, 8, None) == -9
    assert b.raw_status("snack_grad_workspace", -1, None) == -1
    assert b.snack_grad_workspace(113) == 2 * b.snack_grad_workspace(112)
