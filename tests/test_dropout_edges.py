"""What a dropout module does beside one plain call: where its seed comes from,
calls that are run again in the backward, capture, copies, and the longest rows.
On the CPU the kernel is replaced by the definition of its mask."""
import pytest
import torch

import unstructured_sparse_nn_amd as snk

gpu = pytest.mark.gpu


@pytest.mark.parametrize("make", [lambda: snk.Dropout(0.1).seed,
                                  lambda: snk.dropout.random_seed()])
def test_seeds_come_from_the_cpus_generator_whatever_the_default_device(make):
    torch.manual_seed(11)
    want = make()
    torch.manual_seed(11)
    with torch.device("meta"):
        assert make() == want


# ------------------------------------------------------------- calls run again
class PlainCalls:
    """The mask by its definition, for tensors on the CPU."""

    @staticmethod
    def dropout(x, p, seed, step, more, residual, out):
        from test_dropout import formula
        assert more is None
        y = formula(x, p, seed, step, residual)[0].to(x.dtype)
        return y if out is None else out.copy_(y)


@pytest.fixture
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(snk.dropout, "calls", PlainCalls)

    def lora_fwd(x, ids, A, B, scale, ranks=None, base=None, t=None):
        v = (A[ids.long()] * x[:, None, :]).sum(-1)
        t.copy_(v)
        y = (v[:, :, None] * B[ids.long()]).sum(1) * scale[ids.long()][:, None]
        return y if base is None else base + y

    def lora_bwd(gy, x, ids, A, B, scale, ranks, t, want):
        with torch.enable_grad():
            x, A, B = (v.detach().requires_grad_(True) for v in (x, A, B))
            y = lora_fwd(x, ids, A, B, scale, t=torch.empty_like(t))
        got = torch.autograd.grad(y, (x, A, B), gy)
        return tuple(g if w else None for g, w in zip(got, want))

    monkeypatch.setattr(snk.adapters, "lora_fwd", lora_fwd)
    monkeypatch.setattr(snk.adapters, "lora_bwd", lora_bwd)


class Block(torch.nn.Module):
    """Two calls of one dropout, an adapter with dropout, and a product whose
    gradient needs what was dropped."""

    def __init__(self, device):
        super().__init__()
        g = torch.Generator().manual_seed(3)
        self.drop = snk.Dropout(0.4, seed=5)
        self.ad = snk.LoraAdapters(12, 12, 2, 4, dropout=0.3, seed=6, device=device)
        with torch.no_grad():
            self.ad.A.copy_(torch.randn(2, 4, 12, generator=g))
            self.ad.B.copy_(torch.randn(2, 4, 12, generator=g))
        self.w = torch.nn.Parameter(torch.randn(12, generator=g).to(device))

    def forward(self, x, ids):
        h = self.drop(x) * self.w
        h = self.ad(h, ids, h)
        return self.drop(h.tanh(), x) * self.w


def gradients(run, block, xs, ids):
    """Forwards of all xs, then their backwards, the last first."""
    for p in block.parameters():
        p.grad = None
    ys = [run(x, ids) for x in xs]
    for y in reversed(ys):
        (y * y).sum().backward()
    grads = [x.grad for x in xs] + [p.grad.clone() for p in block.parameters()]
    for x in xs:
        x.grad = None
    return [y.detach() for y in ys] + grads


def forms_of_checkpoint(device):
    from torch.utils.checkpoint import checkpoint
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(9, 12, generator=g).to(device).requires_grad_(True) for _ in range(3)]
    ids = torch.randint(0, 2, (9,), generator=g).int().to(device)
    plain = Block(device)
    want = gradients(plain, plain, xs, ids)
    assert plain.drop.step == 6 and plain.ad.step == 3
    assert not torch.equal(plain(xs[0], ids), plain(xs[0], ids))
    for form in (True, False):
        block = Block(device)

        def run(x, i):
            return checkpoint(block, x, i, use_reentrant=form)

        for a, c in zip(want, gradients(run, block, xs, ids)):
            assert torch.equal(a, c), form
        assert block.drop.step == 6 and block.ad.step == 3  # a call that is run again counts once
        # one step after another, and the generator set back between two of them
        for x in xs:
            block.drop.step = block.ad.step = 20
            torch.manual_seed(4)
            got = gradients(run, block, [x], ids)
            block.drop.step = block.ad.step = 20
            for a, c in zip(got, gradients(block, block, [x], ids)):
                assert torch.equal(a, c), form
            torch.manual_seed(4)
            a = gradients(run, block, [x], ids)
            torch.manual_seed(4)
            for a, c in zip(a, gradients(block, block, [x], ids)):
                assert torch.equal(a, c), form


def what_cannot_be_known_is_refused(device):
    from torch.utils.checkpoint import checkpoint
    x = torch.ones(4, 8, device=device, requires_grad=True)
    for form in (True, False):
        m = snk.Dropout(0.5, seed=1)
        y = checkpoint(lambda v: m(v) * v, x, use_reentrant=form, preserve_rng_state=False)
        with pytest.raises(RuntimeError, match="name the step"):
            y.sum().backward()
        # a step that the call names needs no generator
        y = checkpoint(lambda v: m(v, step=3) * v, x, use_reentrant=form,
                       preserve_rng_state=False)
        x.grad = None
        y.sum().backward()
        assert torch.equal(x.grad, 2 * m(x.detach(), step=3))


def test_checkpointed_calls_on_the_cpu(on_the_cpu):
    forms_of_checkpoint("cpu")


def test_unknown_steps_are_refused_on_the_cpu(on_the_cpu):
    what_cannot_be_known_is_refused("cpu")


def test_what_a_module_remembers_is_bounded(on_the_cpu, monkeypatch):
    import copy
    import gc
    import pickle
    m = snk.Dropout(0.5, seed=1)
    monkeypatch.setattr(snk.dropout, "RECENT", 5)
    for _ in range(12):
        m(torch.ones(3))
    assert m.step == 12 and len(snk.dropout._known[m][1]) == 5
    again = pickle.loads(pickle.dumps(m))
    assert again.seed == 1 and again.step == 12 and set(vars(again)) == set(vars(m))
    assert copy.copy(m).step == 12
    before = len(snk.dropout._known)
    del m
    gc.collect()
    assert len(snk.dropout._known) == before - 1


@gpu
def test_checkpointed_calls():
    forms_of_checkpoint("cuda")
    what_cannot_be_known_is_refused("cuda")


# ------------------------------------------------------------------ in a graph
def modules_of_a_capture(device):
    return ((snk.Dropout(0.5, seed=1), ()),
            (snk.LoraAdapters(8, 8, 1, 4, dropout=0.5, seed=1, device=device),
             (torch.zeros(4, dtype=torch.int32, device=device),)))


def test_a_captured_call_has_to_name_its_step(on_the_cpu, monkeypatch):
    class OnGpu(torch.Tensor):
        is_cuda = True

    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    x = torch.ones(4, 8).as_subclass(OnGpu)
    for m, ids in modules_of_a_capture("cpu"):
        with pytest.raises(RuntimeError, match="captured.*step"):
            m(x, *ids)
        assert m.step == 0


@gpu
def test_captures_with_and_without_a_step():
    x = torch.ones(4, 8, device="cuda")
    step = torch.tensor([2], device="cuda")
    s = torch.cuda.Stream()
    for m, ids in modules_of_a_capture("cuda"):
        with torch.cuda.stream(s):
            m(x, *ids, step=step)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            with pytest.raises(RuntimeError, match="captured.*step"):
                m(x, *ids)
            y = m(x, *ids, step=step)
            z = m(x, *ids, step=4)  # a number of the caller's own stays what it is
        for k in (3, 2 ** 33, 3):
            step.fill_(k)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, m(x, *ids, step=k)) and torch.equal(z, m(x, *ids, step=4))
        assert m.step == 0


# -------------------------------------------------------------------- deep copies
def copies_drop_other_elements(device):
    import copy

    class Layer(torch.nn.Module):
        def __init__(self):
            super().__init__()
            self.drop = snk.Dropout(0.5, seed=1)
            self.same = self.drop
            self.ad = snk.LoraAdapters(8, 8, 1, 4, dropout=0.5, seed=2, device=device)
            self.plain = snk.LoraAdapters(8, 8, 1, 4, device=device)

    first = Layer()
    first.drop(torch.ones(2, 8, device=device))
    state = torch.get_rng_state()
    a, c = copy.deepcopy(first), copy.deepcopy(first)
    d = copy.deepcopy(a)
    assert torch.equal(torch.get_rng_state(), state)  # the program's random numbers are as before
    layers = [first, a, c, d]
    x = torch.ones(40, 8, device=device)
    masks = [layer.drop(x, step=3) for layer in layers]
    for i in range(4):
        assert layers[i].same is layers[i].drop and layers[i].plain.seed is None
        assert layers[i].drop.step == 1 and layers[i].drop.p == 0.5
        assert torch.equal(layers[i].ad.A, first.ad.A) and layers[i].ad.ranks is None
        for j in range(i):
            assert not torch.equal(masks[i], masks[j])
            assert layers[i].drop.seed != layers[j].drop.seed
            assert layers[i].ad.seed != layers[j].ad.seed
            assert layers[i].ad.A is not layers[j].ad.A
    # the same program has the same seeds
    again = Layer()
    assert [copy.deepcopy(again).drop.seed for _ in range(2)] == [a.drop.seed, c.drop.seed]


def test_deep_copies_on_the_cpu(on_the_cpu):
    copies_drop_other_elements("cpu")


@gpu
def test_deep_copies():
    copies_drop_other_elements("cuda")


# ------------------------------------------------------------------ longest rows
@gpu
def test_more_elements_than_one_launch_holds():
    """2^32 work items of eight elements in fp32 are 2^35: 128 GiB, in place."""
    n = 2 ** 35 + 3 * 2 ** 12 + 5
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 5 * n:
        pytest.skip("160 GiB of free memory needed")
    from test_dropout import field
    x = torch.ones(n, device="cuda")
    try:
        snk.dropout_fwd(x, 0.5, 21, 22, out=x)
        for at in (0, 2 ** 32 - 300, 2 ** 33 - 300, 2 ** 34 - 300, 2 ** 35 - 300, n - 600):
            want = [0.0 if field(21, 22, i) < 32768 else 2.0 for i in range(at, at + 600)]
            assert x[at:at + 600].tolist() == want, at
    finally:
        del x
        torch.cuda.empty_cache()


def test_draws_under_modes_of_torch(on_the_cpu):
    """The number is the program's own also where tensors are made otherwise."""
    import threading
    want = {}

    def draws():
        torch.manual_seed(5)
        with torch.inference_mode():
            a = snk.dropout._draw()
        with torch.device("meta"), torch.no_grad():
            c = snk.dropout._draw()
        want[threading.get_ident()] = a, c, snk.dropout._draw()

    t = threading.Thread(target=draws)
    t.start()
    t.join()
    draws()
    one, two = want.values()
    assert one == two and len(set(one)) == 3
    # the generator moves on by each call, so a block that is run again meets the same
    m = snk.Dropout(0.5, seed=1)
    torch.manual_seed(5)
    m(torch.ones(3))
    assert list(snk.dropout._known[m][1]) == [one[0]]
