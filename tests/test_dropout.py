"""Dropout against the generator's definition on whole numbers and the formula
in 64 bits.  Tolerances, with e = 2^-24 and h = 2^-8: the scale's rounding and
the product's, e each of the product, the sum's, e, and in bf16 h of the result."""
import ctypes

import numpy as np
import pytest
import torch

import unstructured_sparse_nn_amd as snk
from unstructured_sparse_nn_amd import binding as b

E = 2.0 ** -24
F, H = torch.float32, torch.bfloat16
ROUND = {F: 0.0, H: 2.0 ** -8}
gpu = pytest.mark.gpu
M64 = (1 << 64) - 1


def mix(z):
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & M64
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & M64
    return z ^ (z >> 31)


def field(seed, step, i):
    """The 16 bits of element i, from the definition."""
    g = 0x9E3779B97F4A7C15
    stream = mix((seed + (step + 1) * g) & M64)
    return (mix((stream + (i // 4 + 1) * g) & M64) >> (16 * (i % 4))) & 0xFFFF


def fields(n, seed, step):
    u = np.uint64
    with np.errstate(over="ignore"):
        stream = u(mix((seed + (step + 1) * 0x9E3779B97F4A7C15) & M64))
        z = stream + np.arange(1, -(-n // 4) + 1, dtype=u) * u(0x9E3779B97F4A7C15)
        z = (z ^ (z >> u(30))) * u(0xBF58476D1CE4E5B9)
        z = (z ^ (z >> u(27))) * u(0x94D049BB133111EB)
        z = z ^ (z >> u(31))
    return z.astype("<u8").view("<u2")[:n].astype(np.int64)


def level(p):
    return int(p * 65536 + 0.5)


def formula(x, p, seed, step, residual=None):
    """(values, tolerance) in 64 bits, of x's shape on the CPU."""
    n = level(p)
    keep = torch.from_numpy(fields(x.numel(), seed, step) >= n).view(x.shape)
    scale = 65536 / (65536 - n) if n < 65536 else 0.0
    v = torch.where(keep, x.double().cpu() * scale, 0.0)
    r = torch.zeros_like(v) if residual is None else residual.double().cpu()
    y = v + r
    return y, 2.02 * E * v.abs() + (E + ROUND[x.dtype]) * 1.01 * y.abs() + 2.0 ** -133


def close(got, ref):
    y, tol = ref
    bad = ~((got.double().cpu() - y).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0], got.shape)


def test_the_streams_definition():
    n = 37
    want = [field(2 ** 63 + 5, 2 ** 40, i) for i in range(n)]
    assert fields(n, 2 ** 63 + 5, 2 ** 40).tolist() == want
    # the same stream of streams as the restructuring: output 0 of seed 0 is published
    assert mix(0x9E3779B97F4A7C15) == 16294208416658607535


SHAPES = [(1,), (3,), (4,), (8,), (9,), (1, 1), (7, 1), (1, 5), (515, 1001), (64, 4096), (3, 5, 7),
          (2, 0, 5), (0,), (1023, 8), (4099,), (8192,), (4097 * 2,), (2, 3, 4, 24)]


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_forward_and_backward(shape, dt):
    g = torch.Generator().manual_seed(len(shape))
    x, r = (torch.randn(*shape, generator=g).to(dt).cuda() for _ in range(2))
    seed, step = 0xDEADBEEFCAFEBABE, 3
    close(snk.dropout_fwd(x, 0.3, seed, step), formula(x, 0.3, seed, step))
    close(snk.dropout_fwd(x, 0.3, seed, step, residual=r), formula(x, 0.3, seed, step, r))
    assert torch.equal(snk.dropout_bwd(x, 0.3, seed, step), snk.dropout_fwd(x, 0.3, seed, step))
    want = snk.dropout_fwd(x, 0.3, seed, step, residual=r)
    a, c = x.clone(), r.clone()
    assert snk.dropout_fwd(a, 0.3, seed, step, residual=r, out=a) is a and torch.equal(a, want)
    assert snk.dropout_fwd(x, 0.3, seed, step, residual=c, out=c) is c and torch.equal(c, want)


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("cols", [1, 2, 3, 5, 7, 8, 9, 12, 24, 31, 100, 1001, 4096])
def test_strided_rows_at_any_alignment(cols, dt):
    rows = 37
    for off in (0, 1, 3):
        wide = torch.randn(rows, cols + 13, device="cuda").to(dt)
        x = wide[:, off:off + cols]
        r = torch.randn(rows, 2 * cols, device="cuda").to(dt)[:, cols:]
        out = torch.full((rows, cols + 7), 7.0, dtype=dt, device="cuda")
        y = out[:, 2:2 + cols]
        snk.dropout_fwd(x, 0.5, 11, 12, residual=r, out=y)
        close(y, formula(x.contiguous(), 0.5, 11, 12, r))
        assert (out[:, :2] == 7).all() and (out[:, 2 + cols:] == 7).all()
        # strides change nothing of the mask
        assert torch.equal(snk.dropout_fwd(x, 0.5, 11, 12), snk.dropout_fwd(x.contiguous(), 0.5, 11, 12))
        snk.dropout_fwd(x, 0.5, 11, 12, residual=r, out=x)  # in place, strided
        assert torch.equal(x, y)
        t = torch.randn(cols, rows, device="cuda").to(dt).t()  # no rows at all: copied
        close(snk.dropout_fwd(t, 0.5, 11, 12), formula(t.contiguous(), 0.5, 11, 12))


@gpu
@pytest.mark.parametrize("p", [0.0, 1.0, 0.5, 2.0 ** -17, 2.0 ** -18, 1 - 2.0 ** -16, 0.1])
def test_probabilities(p):
    x = torch.randn(100, 1000, device="cuda")
    y = snk.dropout_fwd(x, p, 5, 6)
    close(y, formula(x, p, 5, 6))
    if level(p) == 0:
        assert torch.equal(x, y)
    if p == 1.0:
        assert (y == 0).all()


@gpu
@pytest.mark.parametrize("dt", [F, H])
def test_what_is_dropped_is_gone(dt):
    x = torch.randn(33, 1000, device="cuda").to(dt)
    x[::2] = float("nan")
    x[1::4] = float("inf")
    r = torch.randn(33, 1000, device="cuda").to(dt)
    drop = torch.from_numpy(fields(33000, 1, 2) < level(0.4)).view(33, 1000).cuda()
    y = snk.dropout_fwd(x, 0.4, 1, 2)
    assert (y[drop] == 0).all() and torch.equal(torch.isnan(y), torch.isnan(x) & ~drop)
    y = snk.dropout_fwd(x, 0.4, 1, 2, residual=r)
    assert torch.equal(y[drop], r[drop])


@gpu
def test_steps_and_seeds_differ():
    x = torch.ones(20000, device="cuda")
    kept = [snk.dropout_fwd(x, 0.5, *k) > 0 for k in ((1, 1), (1, 2), (2, 1), (2, 2))]
    for i in range(4):
        # binomial, 20,000 trials: six standard deviations are 0.0212
        assert abs(float(kept[i].float().mean()) - 0.5) < 0.0212
        for j in range(i):
            assert abs(float((kept[i] == kept[j]).float().mean()) - 0.5) < 0.0212


@gpu
def test_step_on_the_gpu_and_in_a_graph():
    x = torch.randn(64, 300, device="cuda")
    step = torch.tensor([7], device="cuda")
    assert torch.equal(snk.dropout_fwd(x, 0.2, 9, step), snk.dropout_fwd(x, 0.2, 9, 7))
    out = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        snk.dropout_fwd(x, 0.2, 9, step, out=out)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        snk.dropout_fwd(x, 0.2, 9, step, out=out)
    for k in (7, 8, 2 ** 40, 9):
        step.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, snk.dropout_fwd(x, 0.2, 9, k)), k


@gpu
def test_places_past_32_bits():
    n = 2 ** 32 + 4 * 1024
    x = torch.ones(n, dtype=H, device="cuda")
    y = snk.dropout_fwd(x, 0.5, 21, 22, out=x)
    for at in (0, 2 ** 31 - 512, 2 ** 32 - 512, n - 1024):
        want = [0.0 if field(21, 22, i) < 32768 else 2.0 for i in range(at, at + 1024)]
        assert y[at:at + 1024].tolist() == want
    del x, y
    # rows farther apart than their elements: offsets past 2^31, places past 2^32
    big = torch.empty(3, 2 ** 31 + 8, dtype=H, device="cuda")
    v = big[:, :1003]
    v.fill_(1.0)
    close(snk.dropout_fwd(v, 0.5, 1, 2), formula(v.contiguous(), 0.5, 1, 2))


@gpu
def test_module_and_autograd():
    torch.manual_seed(4)
    m = snk.Dropout(0.25)
    x = torch.randn(40, 50, device="cuda", requires_grad=True)
    r = torch.randn(40, 50, device="cuda", requires_grad=True)
    y = m(x, r)
    close(y, formula(x.detach(), 0.25, m.seed, 0, r.detach()))
    gy = torch.randn_like(y)
    y.backward(gy)
    close(x.grad, formula(gy, 0.25, m.seed, 0))
    assert torch.equal(r.grad, gy)
    assert m.step == 1 and not torch.equal(m(x), m(x)) and m.step == 3
    assert torch.equal(m(x, step=1), m(x, step=torch.tensor([1], device="cuda")))
    m.eval()
    assert m(x) is x and torch.equal(m(x, r), r + x)
    assert snk.Dropout(0.0)(x) is x
    # a step on the GPU that changes before the backward is noticed
    step = torch.tensor([1], device="cuda")
    y = m.train()(x, step=step)
    step += 1
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    out = torch.empty(40, 50, device="cuda")
    v = out._version
    snk.dropout_fwd(x.detach(), 0.1, 1, out=out)
    assert out._version > v


@gpu
def test_another_stream_and_the_binding():
    x = torch.randn(3000, 77, device="cuda")
    want = snk.dropout_fwd(x, 0.1, 2 ** 64 - 1, 5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = snk.dropout_fwd(x, 0.1, -1, 5)
    s.synchronize()
    assert torch.equal(other, want)
    y = torch.empty_like(x)
    snk.snack_dropout(x, 77, None, 0, y, 77, 3000, 77, 0.1, 2 ** 64 - 1, 5)
    assert torch.equal(y, want)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), -3), (dict(rows=-1), -2), (dict(cols=-1), -2), (dict(p=-0.1), -2),
    (dict(p=1.1), -2), (dict(p=float("nan")), -7), (dict(ldx=9), -2), (dict(ldy=9), -2),
    (dict(ldr=9), -2), (dict(X=None), -1), (dict(Y=None), -1), (dict(Y=0x10004), -2),
    (dict(Y=0x10000, ldy=11), -2), (dict(Y=0x20000, ldy=11), -2), (dict(Y=0x20000 - 4), -2),
    (dict(rows=1 << 30, cols=1 << 10, ldx=1 << 10, ldr=1 << 10, ldy=1 << 10), -10), (dict(step_dev=0x40008), -2),
    (dict(rows=1 << 26, cols=513, ldx=514, ldr=514, ldy=514, X=1 << 40, residual=None,
          Y=1 << 44), -10)])
def test_refusals(bad, status):
    a = dict(dtype=0, X=0x10000, ldx=10, residual=0x20000, ldr=10, Y=0x40000, ldy=10, rows=7,
             cols=10, p=0.5, seed=1, step=2, step_dev=None, stream=None)
    a.update(bad)
    a["p"] = ctypes.c_double(a["p"])
    assert b.raw_status("snack_dropout", *a.values()) == status


def test_nothing_to_do():
    assert b.raw_status("snack_dropout", 0, None, 0, None, 0, None, 0, 0, 0, 0.5, 0, 0, None,
                        None) == 0


def test_wrappers_refuse_what_does_not_fit():
    x = torch.zeros(3, 4)
    with pytest.raises(TypeError, match="on the GPU"):
        snk.dropout_fwd(x, 0.5, 1)
    with pytest.raises(TypeError, match="unsupported dtype"):
        snk.dropout_fwd(x.half(), 0.5, 1)
    with pytest.raises(TypeError, match="expected a tensor"):
        snk.dropout_fwd([1.0], 0.5, 1)
    for p in (-0.5, 1.5, float("nan")):
        with pytest.raises(ValueError):
            snk.Dropout(p)


@gpu
def test_wrappers_refuse_on_the_gpu():
    x = torch.zeros(3, 4, device="cuda")
    for bad in (dict(residual=x.to(H)), dict(out=x.to(H)), dict(residual=x.cpu()),
                dict(step=torch.tensor([1], dtype=torch.int32, device="cuda")),
                dict(step=torch.tensor([1, 2], device="cuda")), dict(step=torch.tensor([1]))):
        with pytest.raises(TypeError):
            snk.dropout_fwd(x, 0.5, 1, **bad)
    for bad in (dict(residual=x[:2]), dict(out=x[:, :3]), dict(out=torch.zeros(4, 3, device="cuda").t()),
                dict(out=torch.zeros(1, 4, device="cuda").expand(3, 4))):
        with pytest.raises(ValueError):
            snk.dropout_fwd(x, 0.5, 1, **bad)
    with pytest.raises(snk.SnackError):
        snk.dropout_fwd(x, 1.5, 1)
    flat = torch.zeros(13, device="cuda")
    with pytest.raises(snk.SnackError):  # an output shifted against its input
        snk.dropout_fwd(flat[:12].view(3, 4), 0.5, 1, out=flat[1:].view(3, 4))
