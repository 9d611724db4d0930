"""Embedding, dropout, a sparse layer with adapters, log-probabilities and the
losses run together, as a fine-tuning step uses them.  The gradients are
compared with torch's own differentiation of the same formulas in 64 bits from
the same masks: fp32 sums of at most 2,000 terms, chained through five
operators, are within 10^-4 of the largest gradient."""
import os
import sys

import pytest
import torch

import unstructured_sparse_nn_amd as snk

gpu = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))


def dropped(x, p, seed, step):
    """The mask times its scale, from the kernel on ones (tested by itself)."""
    return snk.dropout_fwd(torch.ones_like(x, dtype=torch.float32), p, seed, step).double()


def near(got, ref):
    assert got.shape == ref.shape
    assert float((got.detach().double() - ref).abs().max()) <= 1e-4 * float(ref.abs().max())


@gpu
@pytest.mark.parametrize("p", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("on_gpu", [False, True])
def test_adapters_with_dropout(p, on_gpu):
    torch.manual_seed(3)
    T, K, M = 70, 96, 40
    m = snk.LoraAdapters(K, M, 3, 8, dropout=p, seed=17)
    m.B.data.normal_(std=0.2)
    x = torch.randn(T, K, device="cuda", requires_grad=True)
    base = torch.randn(T, M, device="cuda", requires_grad=True)
    ids = torch.randint(-1, 3, (T,), device="cuda").int()
    step = torch.tensor([5], device="cuda") if on_gpu else 5
    y = m(x, ids, base, step=step)
    gy = torch.randn_like(y)
    y.backward(gy)
    xd, A, B, bd = (v.detach().double().requires_grad_(True) for v in (x, m.A, m.B, base))
    mask = dropped(x, p, 17, 5) if p > 0 else 1.0
    t = (A[ids.long().clamp(min=0)] * (xd * mask)[:, None, :]).sum(-1)
    add = (t[:, :, None] * B[ids.long().clamp(min=0)]).sum(1) * m.scale[ids.long().clamp(min=0)][:, None].double()
    want = bd + torch.where((ids >= 0)[:, None], add, 0.0)
    want.backward(gy.double())
    near(y, want.detach())
    for a, c in ((x, xd), (m.A, A), (m.B, B), (base, bd)):
        if float(c.grad.abs().max()) == 0.0:
            assert (a.grad == 0).all()
        else:
            near(a.grad, c.grad)


@gpu
def test_adapters_without_dropout_are_as_before():
    torch.manual_seed(5)
    m = snk.LoraAdapters(32, 24, 2, 4)
    after = torch.randn(3)
    torch.manual_seed(5)
    n = snk.LoraAdapters(32, 24, 2, 4, dropout=0.2, seed=1)
    assert torch.equal(m.A, n.A) and torch.equal(torch.randn(3), after)
    assert set(m.state_dict()) == set(n.state_dict()) == {"A", "B", "scale"}
    m.B.data.normal_()
    n.load_state_dict(m.state_dict())
    x, ids = torch.randn(9, 32, device="cuda"), torch.zeros(9, dtype=torch.int32, device="cuda")
    assert torch.equal(n.eval()(x, ids), m(x, ids)) and n.step == 0
    assert not torch.equal(n.train()(x, ids), m(x, ids)) and n.step == 1
    for bad in (-0.1, 1.1, float("nan")):
        with pytest.raises(ValueError):
            snk.LoraAdapters(4, 4, 1, 1, dropout=bad)


def model_step(loss_of, seed=0):
    """One step of a small model: its parameters with gradients, and the same
    gradients in 64 bits."""
    from adapters import sparse_layer
    torch.manual_seed(seed)
    V, D, M, T = 61, 48, 64, 200
    emb = snk.TokenEmbedding(V, D, scale=D ** 0.5)
    drop = snk.Dropout(0.1, seed=1)
    layer = sparse_layer(D, M, 0.2, T)
    ad = snk.LoraAdapters(D, M, 2, 8, dropout=0.2, seed=2)
    ad.B.data.normal_(std=0.1)
    head = (torch.randn(M, V, device="cuda") * M ** -0.5).requires_grad_(True)
    ids = torch.randint(0, V, (T,), device="cuda")
    targets = ids.roll(-1)
    targets[::9] = -1
    of = torch.randint(0, 2, (T,), device="cuda").int()
    h = drop(emb(ids))
    h = ad(h, of, layer(h))
    logps = snk.token_logps(h @ head, targets)
    loss = loss_of(logps)
    loss.backward()
    assert float(snk.clip_grad_norm_([emb.weight, ad.A, ad.B, head], 1e9)) > 0
    # the same in 64 bits
    W, A, B, H = (v.detach().double().requires_grad_(True) for v in (emb.weight, ad.A, ad.B, head))
    x = W[ids] * D ** 0.5 * dropped(torch.empty(T, D, device="cuda"), 0.1, 1, 0)
    S = torch.zeros(M, D, dtype=torch.float64, device="cuda")
    S[layer.topo.row.long(), layer.topo.col.long()] = layer.vals.detach().double()
    z = x * dropped(torch.empty(T, D, device="cuda"), 0.2, 2, 0)
    y = x @ S.t()
    for l in range(2):
        y = y + torch.where((of == l)[:, None], (z @ A[l].t()) @ B[l] * float(ad.scale[l]), 0.0)
    lp = torch.log_softmax(y @ H, 1).gather(1, targets.clamp(min=0)[:, None])[:, 0]
    lp = torch.where(targets < 0, 0.0, lp)
    return loss, logps, lp, list(zip((emb.weight, ad.A, ad.B, head), (W, A, B, H)))


@gpu
def test_a_preference_step():
    starts = torch.tensor([0, 40, 90, 150, 200], dtype=torch.int32, device="cuda")
    loss, logps, lp, params = model_step(lambda v: snk.preference_loss(v, starts, beta=0.05)[0])
    near(logps, lp.detach())
    d = torch.stack([lp[a:c].sum() for a, c in ((0, 40), (40, 90), (90, 150), (150, 200))])
    want = -torch.nn.functional.logsigmoid(0.05 * (d[0::2] - d[1::2])).mean()
    want.backward()
    assert abs(float(loss) - float(want)) <= 1e-5 * float(want)
    for a, c in params:
        near(a.grad, c.grad)


@gpu
def test_a_policy_step():
    g = torch.Generator().manual_seed(4)
    noise = (torch.randn(200, generator=g) * 0.05).cuda()
    adv = torch.randn(10, generator=g).cuda()
    kept = {}

    def loss_of(v):
        kept["old"], kept["ref"] = v.detach() + noise, v.detach() - noise
        return snk.policy_loss(v.view(10, 20), kept["old"].view(10, 20), adv,
                               ref=kept["ref"].view(10, 20), kl=0.1, clip=(0.9, 9.0))[0]

    loss, logps, lp, params = model_step(loss_of, 1)
    r = (lp - kept["old"].double()).exp()
    k = kept["ref"].double() - lp
    want = (-r * adv.double().repeat_interleave(20) + 0.1 * (k.exp() - k - 1)).mean()
    want.backward()
    assert abs(float(loss) - float(want)) <= 1e-5 * (1 + abs(float(want)))
    for a, c in params:
        near(a.grad, c.grad)


@gpu
def test_a_captured_step_draws_anew():
    """Forward and backward in one graph, the step's number on the GPU."""
    torch.manual_seed(6)
    emb = snk.TokenEmbedding(50, 32)
    ad = snk.LoraAdapters(32, 50, 1, 4, dropout=0.5, seed=3)
    ad.B.data.normal_()
    ids = torch.randint(0, 50, (64,), device="cuda")
    of = torch.zeros(64, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    step = torch.tensor([0], device="cuda")
    params = [emb.weight, ad.A, ad.B]

    def run():
        logps = snk.token_logps(ad(emb(ids), of, step=step), ids)
        loss = snk.preference_loss(logps, starts, beta=1.0)[0]
        return [loss.detach(), *torch.autograd.grad(loss, params)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    seen = []
    for k in (1, 2, 3, 1):
        step.fill_(k)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        want = run()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip(got, want)), k
        seen.append(got[2])
    assert torch.equal(seen[0], seen[3]) and not torch.equal(seen[0], seen[1])
