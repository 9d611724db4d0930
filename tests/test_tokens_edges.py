"""Values of the lookup and of the logits' gradient at infinities and NaN."""
import pytest
import torch

import unstructured_sparse_nn_amd as snk
from test_tokens import F, H, INF, NAN, logits_of

gpu = pytest.mark.gpu


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("V", [100, 3001, 9001])  # pieces of all short rows, and rows
def test_a_gradient_of_nan_is_kept_where_nothing_is_left(V, dt):
    """A row of -infinity throughout has a zero gradient, but for a target past the end
    and a NaN that comes in: those make every row NaN."""
    x, t = logits_of(6, V, dt, 5)
    x[:5] = -INF
    t = t.clamp(min=0)
    t[1], t[3], t[4] = V, -1, V + 7
    g = torch.tensor([1.0, 1.0, NAN, NAN, 0.0, NAN], device="cuda")
    logp, norm = snk.logp_fwd(x, t)
    assert torch.isnan(logp[[1, 4]]).all() and float(logp[0]) == -INF and float(logp[3]) == 0
    dx = snk.logp_bwd(g, x, t, norm)
    nan = torch.tensor([False, True, True, False, True, True])
    assert torch.isnan(dx[nan.cuda()]).all() and (dx[~nan.cuda()] == 0).all()


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("V", [100, 3001, 9001])
def test_a_gradient_of_infinity_is_infinite_at_the_target(V, dt):
    """dlogp times 1 - p and -p, which have no zero here."""
    x, t = logits_of(2, V, dt, 7)
    x = (x.float().clamp(-3, 3)).to(dt)
    t = torch.tensor([3, V - 1], device="cuda")
    norm = snk.logp_fwd(x, t)[1]
    for v in (INF, -INF):
        dx = snk.logp_bwd(torch.full((2,), v, device="cuda"), x, t, norm)
        want = torch.full_like(dx, -v)
        want[[0, 1], t] = v
        assert torch.equal(dx, want)


@gpu
@pytest.mark.parametrize("dt", [F, H])
@pytest.mark.parametrize("D", [3, 8, 33])
def test_no_token_is_a_row_of_zeros_under_every_scale(D, dt):
    w = torch.rand(5, D, device="cuda").to(dt) + 1
    ids = torch.tensor([-1, 2, -9, 5], device="cuda")
    for scale, there in ((INF, INF), (-INF, -INF), (NAN, NAN), (-1.0, None), (0.0, 0.0)):
        y = snk.embed_fwd(ids, w, scale)
        assert torch.equal(y[[0, 2]], torch.zeros(2, D, dtype=dt, device="cuda"))
        assert not torch.signbit(y[[0, 2]].float()).any() and torch.isnan(y[3]).all()
        if there is not None:
            row = torch.full((D,), there, dtype=dt, device="cuda")
            assert torch.equal(y[1].nan_to_num(7.0), row.nan_to_num(7.0))
