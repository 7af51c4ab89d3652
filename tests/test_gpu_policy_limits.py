"""Policy and preference losses where values leave float32's range: ratios far above and below their
limits, log probabilities of -inf, advantages that are NaN beyond every limit.  What is finite is
compared with the float64 oracle within policy_cases' bounds; infinities and NaN have to be where the
definitions put them."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import policy_cases as P
from gpu_helpers import say
from oracle import policy as OP

pytestmark = pytest.mark.gpu
INF = np.float32(np.inf)

# One work-group, and three launches with several chunks a sequence.
SIZES = [(12, [0, 3, 4, 9, 12]), (5000, [0, 700, 701, 2500, 5000])]


def _rng(*key):
    return np.random.default_rng([int(v) for v in key] + [37])


def _clipped_everywhere(n, offsets, gaps, advantage):
    """Sequence s has the mean log ratio gaps[s] (about), and advantages of the sign advantage[s]."""
    rng = _rng(n)
    x = P.rollout(rng, n, None, ignored=0.2, entropy=False)
    old = x["lp"].copy()
    A = x["A"].copy()
    for a, b, gap, sign in zip(offsets, offsets[1:], gaps, advantage):
        old[a:b] = (x["lp"][a:b] - np.float32(gap)).astype(np.float32)
        A[a:b] = sign * np.abs(A[a:b])
        x["w"][a] = 0.5
    return dict(x, old=old, A=A)


@pytest.mark.parametrize("n,offsets", SIZES)
@pytest.mark.parametrize("kl", [0.0, 0.1])
def test_a_sequence_clipped_at_an_infinite_ratio_has_no_slope(n, offsets, kl):
    """exp of the mean log ratio is inf in float32; every token is clipped, so that what is left of
    the slope is the KL term's."""
    c = OP.constants(0.2, 0.2, 3.0, kl)
    x = _clipped_everywhere(n, offsets, [100.0, 95.0, 1000.0, 0.01], [1, -1, 1, -1])
    say(f"clipped sequences of {n} tokens, kl={kl}")
    got = P.run_policy(c, x, offsets)
    P.check_policy(c, x, offsets, got, "clipped")
    assert np.isfinite(got["dlogprob"]).all() and np.isfinite(got["loss"]).all()
    if kl == 0:
        assert (got["dlogprob"][:offsets[3]] == 0).all()
    # one token that the old policy gave no chance
    x["old"][offsets[2]] = -INF
    got = P.run_policy(c, x, offsets)
    P.check_policy(c, x, offsets, got, "old -inf")
    assert np.isfinite(got["dlogprob"]).all()


@pytest.mark.parametrize("n,offsets", SIZES)
def test_a_sequence_of_both_signs_clipped_at_an_infinite_ratio(n, offsets):
    c = OP.constants(0.2, 0.2, 3.0)
    x = _clipped_everywhere(n, offsets, [100.0, 95.0, 1000.0, 0.01], [1, 1, 1, 1])
    x["A"] = (x["A"] * np.where(np.arange(n) % 2, -1, 1)).astype(np.float32)
    got = P.run_policy(c, x, offsets)
    P.check_policy(c, x, offsets, got, "both signs")
    assert (got["dlogprob"][:offsets[3]] == 0).all()


@pytest.mark.parametrize("n,offsets", SIZES)
def test_what_an_infinite_ratio_does_not_clip_goes_on(n, offsets):
    """Without a dual limit a negative advantage is not clipped above, so its slope is infinite;
    positive ones of another sequence are clipped."""
    c = OP.constants()
    x = _clipped_everywhere(n, offsets, [100.0, 0.01, 1000.0, 0.02], [-1, 1, 1, -1])
    got = P.run_policy(c, x, offsets)
    counted = x["w"] != 0
    a, b = offsets[0], offsets[1]
    assert (got["dlogprob"][a:b] == np.where(counted[a:b], INF, 0)).all()
    assert (got["loss"][a:b] == np.where(counted[a:b], INF, 0)).all()
    assert (got["dlogprob"][offsets[2]:offsets[3]] == 0).all()
    assert np.isfinite(got["dlogprob"][b:]).all()


@pytest.mark.parametrize("n,offsets", SIZES)
@pytest.mark.parametrize("gap", [2.0, 100.0, -2.0])
def test_a_bad_advantage_reaches_its_sequence_beyond_every_limit(n, offsets, gap):
    """A NaN is clipped by no limit, so that it is in the sequence's slope whatever the ratio is."""
    c = OP.constants(0.2, 0.2, 3.0)
    x = _clipped_everywhere(n, offsets, [0.01, 0.02, gap, 0.03], [1, -1, 1, 1])
    clean = P.run_policy(c, x, offsets)
    at = offsets[2]
    x["A"][at] = np.nan
    got = P.run_policy(c, x, offsets)
    a, b = offsets[2], offsets[3]
    counted = x["w"][a:b] != 0
    assert np.isnan(got["dlogprob"][a:b][counted]).all()
    assert (got["dlogprob"][a:b][~counted] == 0).all()
    assert np.isnan(got["loss"][at]) and np.isnan(got["totals"][0])
    for lo, hi in ((0, a), (b, n)):
        assert np.array_equal(got["dlogprob"][lo:hi], clean["dlogprob"][lo:hi])
    want = OP.policy(c, x["lp"], x["A"], x["w"], x["old"], x["ref"], None, offsets)
    assert got["counts"].tolist() == want["counts"].tolist()
    assert np.array_equal(np.isnan(got["dlogprob"]), np.isnan(want["dlogprob"]))


# Log ratios past 2^25, whose float32 rounding leaves a rest of a whole or more.
FAR = [(-3.0, -1e9), (-1.0, -1e8), (-5.0, -3e7), (-7.0, -1e29), (-0.5, -3e38), (-1.0, -200.0)]


@pytest.mark.parametrize("offsets", [None, list(range(len(FAR) + 1))])
@pytest.mark.parametrize("sign", [1, -1])
def test_ratios_of_a_filled_in_log_probability(offsets, sign):
    """An old (or a new) log probability of a large negative value: the ratio is inf, or 0."""
    lp, old = (np.array(v, np.float32) for v in zip(*FAR))
    n = len(lp)
    x = dict(lp=lp, old=old, A=np.full(n, sign, np.float32), w=np.full(n, 0.5, np.float32), ref=None,
             H=None)
    got = P.run_policy(OP.constants(), x, offsets)
    if sign > 0:                                         # clipped
        assert (got["loss"] == np.float32(-0.5) * np.float32(1.2)).all()
        assert (got["dlogprob"] == 0).all() and got["counts"].tolist() == [n, n]
    else:
        assert (got["loss"] == INF).all() and (got["dlogprob"] == INF).all()
    got = P.run_policy(OP.constants(clip_low=1.0, clip_high=np.inf), x, offsets)
    assert (got["loss"] == -sign * INF).all() and (got["dlogprob"] == -sign * INF).all()
    x = dict(x, lp=old, old=lp)                          # the ratio is 0
    got = P.run_policy(OP.constants(clip_low=1.0), x, offsets)
    assert (got["loss"] == 0).all() and (got["dlogprob"] == 0).all()


def test_ratios_of_a_filled_in_log_probability_over_logits():
    rows, vocab = len(FAR), 1000
    x = torch.zeros(rows, vocab, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    old = torch.tensor([o for _, o in FAR], **f)
    loss, out = torch.empty(rows, **f), torch.empty_like(x)
    ids = torch.arange(rows, device="cuda")
    for sign, want in ((1.0, -1.2), (-1.0, float("inf"))):
        F.policy_logits_loss_grad(x, ids, torch.full((rows,), sign, **f), torch.ones(rows, **f), loss,
                                  out, old_logprob=old)
        assert torch.equal(loss.cpu(), torch.full((rows,), want)), loss


# pairs (chosen, rejected) of one token each
ENDS = np.array([-1.0, -np.inf, -np.inf, -1.0, -1.0, -2.0], np.float32)


@pytest.mark.parametrize("tokens", [6, 4000])
@pytest.mark.parametrize("smoothing", [0.0, 0.25])
def test_preference_of_a_sequence_without_a_chance(tokens, smoothing):
    """log(1 + exp(-h)) and its slope at h = inf and -inf, where a product of 0 and inf must not
    arise."""
    lp = np.concatenate([ENDS, np.full(tokens - 6, -1.0, np.float32)])
    x = dict(lp=lp, ref=np.zeros(tokens, np.float32), w=np.ones(tokens, np.float32))
    g = np.array([2.0, 2.0, 2.0], np.float32)
    say(f"preference at infinity, {tokens} tokens, smoothing {smoothing}")
    got = P.run_preference(x, np.arange(7), g, beta=0.5, label_smoothing=smoothing)
    assert got["loss"][0] == (INF if smoothing else 0) and got["loss"][1] == INF
    assert np.isfinite(got["loss"][2])
    up, down = 2 * 0.5 * smoothing, 2 * 0.5 * (smoothing - 1)
    assert got["dlogprob"][:4].tolist() == [up, -up, down, -down]
    assert got["rewards"][:2].tolist() == [[-0.5, -np.inf], [-np.inf, -0.5]]
    want = OP.preference(lp, np.arange(7), x["ref"], x["w"], g, beta=0.5, smoothing=smoothing)
    assert np.array_equal(want["loss"][:2], got["loss"][:2])
