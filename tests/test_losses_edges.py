"""Values of the losses at infinities, on the paths of small and of large batches,
and a policy's large batches: items of 512 tokens, sequences of many items,
masks that are counted by a launch of their own."""
import math

import pytest
import torch

import unstructured_sparse_nn_amd as snk
from test_losses import INF, NAN, batch, close, policy

gpu = pytest.mark.gpu
PADS = [0, 9000, 300000]  # one workgroup, items of 128 tokens, items of 512


def padded(values, pad):
    """Sequences of one token each, the last with `pad` tokens more (zeros)."""
    lp = torch.zeros(len(values) + pad, device="cuda")
    lp[:len(values)] = torch.tensor(values)
    starts = list(range(len(values))) + [len(values) + pad]
    return lp, torch.tensor(starts, dtype=torch.int32, device="cuda")


@gpu
@pytest.mark.parametrize("pad", PADS)
def test_the_kl_estimate_of_a_token_that_cannot_be_drawn(pad):
    """exp(k) - k - 1 is infinite at both ends of k, and NaN stays."""
    lp, st = padded([-1.0, -INF, -1.0, NAN], pad)
    ref = lp.clone()
    ref[1:4] = torch.tensor([-1.0, -INF, -1.0])  # k infinite, -infinite, NaN
    adv, keep = torch.zeros(4, device="cuda"), torch.ones_like(lp, dtype=torch.bool)
    old = torch.where(torch.isfinite(lp), lp, -1.0)
    # and -(exp(k) - 1), a fourth of it for the share of a sequence
    for one, value, slope in ((1, INF, -INF), (2, INF, 0.25), (3, NAN, NAN)):
        keep[1:4] = False
        keep[one] = True
        loss, stats, g = snk.policy_grads(lp, old, adv, st, ref=ref, mask=keep, kl=1.0,
                                          average="sequences")
        for got, want in ((loss, value), (stats[0], value), (g[one], slope)):
            assert float(got) == want or math.isnan(want) and math.isnan(float(got)), (one, want)


@gpu
@pytest.mark.parametrize("pad", PADS)
def test_a_kl_weight_of_zero_leaves_the_term_out(pad):
    """The estimate may be past every float where it is only looked at."""
    lp, st = padded([-1.0, -200.0, -INF, -2.0], pad)
    ref, old = lp.clone(), lp.clone()
    ref[1:3] = -1.0  # exp(199) and exp(inf)
    old[2] = -100.0  # a ratio of 0
    adv = torch.tensor([1.0, -0.5, 2.0, 1.0], device="cuda")
    for average in ("tokens", "sequences"):
        loss, stats, g = snk.policy_grads(lp, old, adv, st, ref=ref, average=average, kl=0.0)
        want = snk.policy_grads(lp, old, adv, st, average=average)
        assert torch.equal(loss, want[0]) and torch.isfinite(loss)
        assert torch.equal(g, want[2]) and torch.isfinite(g).all()
        assert float(stats[0]) == INF and torch.equal(stats[1], want[1][1])
        some = snk.policy_grads(lp, old, adv, st, ref=ref, average=average, kl=0.1)
        assert float(some[0]) == INF and float(some[2][1]) == -INF


@gpu
@pytest.mark.parametrize("pad", [0, 9000])
def test_all_smoothing_has_no_product_of_zero_and_infinity(pad):
    """smoothing 1 is the loss of the pair turned round: 0 at z = -infinity."""
    for worse in (0, 1):
        lp, st = padded([0.0, 0.0], pad)
        lp[worse] = -INF
        loss, _, g = snk.preference_grads(lp, st, beta=1.0, smoothing=1.0)
        turned = 0.0 if worse == 0 else INF
        assert float(loss) == turned
        # its derivative by h is sigmoid(z) of z = -infinity or infinity
        assert float(g[0]) == (0.0 if worse == 0 else 1.0) and float(g[1]) == -float(g[0])


@gpu
@pytest.mark.parametrize("pad", PADS)
@pytest.mark.parametrize("by", ["tokens", "sequences"])
def test_an_advantage_of_zero_adds_nothing(pad, by):
    """However far the ratio is past every float; NaN is kept."""
    lp, st = padded([-1.0, -1.0, -1.0, -1.0, -1.0], pad)
    old, ref = lp.clone(), lp - 0.5
    old[1], old[2], old[3] = -101.0, -INF, NAN  # ratios of exp(100), infinity, NaN
    adv = torch.zeros(5, device="cuda")
    adv[4] = 1.0
    if by == "tokens":
        adv = torch.cat([adv, torch.ones(pad, device="cuda")])
    keep = torch.ones_like(lp, dtype=torch.bool)
    keep[3] = False
    loss, stats, g = snk.policy_grads(lp, old, adv, st, by=by, mask=keep)
    fine = snk.policy_grads(lp, lp, adv, st, by=by, mask=keep)
    assert torch.equal(loss, fine[0]) and torch.equal(g, fine[2]) and torch.isfinite(loss)
    assert (g[:3] == 0).all() and float(stats[1]) == 0.0
    # with a KL term the token has that alone
    a, c = (snk.policy_grads(lp, o, adv, st, by=by, mask=keep, ref=ref, kl=0.1) for o in (old, lp))
    assert torch.equal(a[0], c[0]) and torch.equal(a[2], c[2]) and float(a[2][1]) > 0
    loss, _, g = snk.policy_grads(lp, old, adv, st, by=by)
    assert math.isnan(float(loss)) and torch.isnan(g).nonzero().tolist() == [[3]]


@gpu
@pytest.mark.parametrize("pad", PADS)
def test_without_old_the_ratio_is_one(pad):
    """Also where a token cannot be drawn; NaN stays."""
    lp, st = padded([-INF, -1.0, INF, NAN, -2.0], pad)
    adv = torch.tensor([3.0, -0.5, 2.0, 1.0, 1.0], device="cuda")
    keep = ~torch.isnan(lp)
    fine = torch.where(keep & torch.isfinite(lp), lp, -1.0)
    for average in ("tokens", "sequences"):
        got = snk.policy_grads(lp, None, adv, st, mask=keep, average=average)
        want = snk.policy_grads(fine, fine, adv, st, mask=keep, average=average)
        assert all(torch.equal(a, c) for a, c in zip(got, want))
        assert float(got[2][0]) < 0
        loss, _, g = snk.policy_grads(lp, None, adv, st, average=average)
        assert math.isnan(float(loss)) and torch.isnan(g).nonzero().tolist() == [[3]]


# S, T: what takes items of 512 tokens, S + T / 128 of them being more than 2,048
LARGE = [(1024, 400003),  # of every length up to several items, masked beyond 65,536 bytes
         (2, 300001),     # a sequence over hundreds of items, some runs of 256 tokens whole
         (1, 262144),     # items that are full to the last token
         (700, 180001),   # few tokens beyond an item
         (3, 1100000)]


@gpu
@pytest.mark.parametrize("average", ["tokens", "sequences"])
@pytest.mark.parametrize("by", ["tokens", "sequences"])
@pytest.mark.parametrize("S,T", LARGE)
def test_large_policies(S, T, by, average):
    assert S + T // 128 > 2048 and T > 65536
    for k, (old, ref, mask) in enumerate(((True, True, True), (True, True, False),
                                          (True, False, True))):
        d = batch(S, T, S + T + k, outside=k > 0, empty=k == 0)
        d["mask"][::3] = False if k == 2 else d["mask"][::3]
        adv = d["adv_t"] if by == "tokens" else d["adv_s"]
        want = policy(d, 0.2, 0.3, 0.05, average, by, old, ref, mask, 1.5)
        args = (d["logps"], d["old"], adv, d["starts"])
        more = dict(ref=d["ref"] if ref else None, mask=d["mask"] if mask else None,
                    clip=(0.2, 0.3), kl=0.05, average=average, by=by)
        up = torch.tensor(1.5, device="cuda")
        loss, stats, g = snk.policy_grads(*args, **more, dloss=up)
        close(loss, want[0], want[3], "loss")
        close(stats, want[1], want[4], "stats")
        close(g, want[2], want[5], "gradient")
        only = snk.policy_grads(*args, **more, dloss=up, want=(False, True))
        assert torch.equal(only[2], g)
        again = snk.policy_grads(*args, **more, want=(True, False))
        assert torch.equal(again[0], loss) and torch.equal(again[1], stats)


@gpu
def test_large_masks_of_nothing_and_of_everything():
    S, T = 1024, 400003
    d = batch(S, T, 1)
    for average in ("tokens", "sequences"):
        args = (d["logps"], d["old"], d["adv_s"], d["starts"])
        none = snk.policy_grads(*args, mask=torch.zeros_like(d["mask"]), average=average)
        assert float(none[0]) == 0 and (none[1] == 0).all() and (none[2] == 0).all()
        every = snk.policy_grads(*args, mask=torch.ones_like(d["mask"]), average=average)
        assert all(torch.equal(a, c) for a, c in zip(every, snk.policy_grads(*args, average=average)))
