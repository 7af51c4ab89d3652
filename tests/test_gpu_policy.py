"""Policy and preference losses over log probabilities on the GPU against the float64 oracle, with the
error bounds of policy_cases: one token to a million, odd sizes and phases, empty sequences, tokens
behind the last one, weights of zero over bad values, each option, and differences of the kernel's
own loss."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import policy_cases as P
from gpu_helpers import say
from oracle import policy as OP

pytestmark = pytest.mark.gpu

# around a lane's four tokens, a wave's 256, the one work-group's 2,560, and beyond it
SIZES = [1, 2, 3, 4, 5, 63, 255, 256, 257, 1023, 2559, 2560, 2561, 16385, 70001]
FULL = OP.constants(0.2, 0.28, 1.4, 0.1, 0.02)


VARIANTS = [dict(), dict(kind="hinge", beta=0.5, margin=0.2), dict(kind="squared", beta=0.5),
            dict(beta=2.0, margin=0.5, label_smoothing=0.1, length_normalised=True),
            dict(kind="squared", beta=0.1, length_normalised=True, margin=0.1)]


def _seed(*key):
    return np.random.default_rng([int(v) for v in key] + [23])


@pytest.mark.parametrize("n", SIZES)
def test_policy_of_tokens(n):
    for i, (c, kw) in enumerate([(FULL, {}), (OP.constants(), dict(ref=False, entropy=False)),
                                 (OP.constants(0.1, 0.1, 0, 0, 0.5), dict(ref=False)),
                                 (OP.constants(2.0, float("inf"), 0, 1.0, 0), dict(entropy=False)),
                                 (FULL, dict(old=False))]):
        say(f"policy n={n} variant {i}")
        x = P.rollout(_seed(n, i), n, **kw)
        P.check_policy(c, x, None, P.run_policy(c, x, shift=i % 4), f"n={n} variant {i}")


@pytest.mark.parametrize("n,sequences,behind", [(1, 1, 0), (5, 2, 1), (300, 9, 7), (300, 300, 0),
                                                (3, 2, 0), (2560, 16, 1), (2560, 17, 0), (2561, 16, 0),
                                                (4099, 1, 0), (16384, 70, 300), (16385, 70, 0),
                                                (2000, 600, 3), (70001, 130, 5000),
                                                (70001, 5000, 1)])
def test_policy_of_sequences(n, sequences, behind):
    rng = _seed(n, sequences, behind)
    offsets = P.cuts(rng, n, sequences, n - behind)
    for i, (c, kw) in enumerate([(FULL, {}), (OP.constants(0.02, 0.03), dict(ref=False,
                                                                            entropy=False)),
                                 (FULL, dict(old=False))]):
        say(f"policy n={n} sequences={sequences} variant {i}")
        x = P.rollout(rng, n, offsets, **kw)
        P.check_policy(c, x, offsets, P.run_policy(c, x, offsets, shift=(i + 1) % 4),
                       f"n={n} sequences={sequences} variant {i}")


# Sequences around the chunks of a team of 64 or 256 threads (256 and 1,024 tokens) and that start
# and end where its chunks do or next to it; means on both sides of 256 tokens.
LENGTHS = [[256, 257, 1, 255], [1024, 1025, 1023, 4096, 1], [1, 511, 1024, 512, 1536], [5000],
           [0, 257, 0, 0, 600, 3], [100, 9000, 100, 1, 1], [1023, 1, 1025, 9000, 7, 1024],
           [3] * 300 + [600, 5, 2500] + [2] * 200, [10] * 500 + [9000, 1], [513] * 9, [1025] * 9]


def _offsets(lengths, first=0):
    return np.concatenate([[0], np.cumsum(lengths)]) + first


@pytest.mark.parametrize("lengths", LENGTHS, ids=range(len(LENGTHS)))
@pytest.mark.parametrize("first,behind", [(0, 0), (3, 2), (600, 700)])
def test_policy_of_long_sequences(lengths, first, behind):
    offsets = _offsets(lengths, first)
    n = int(offsets[-1]) + behind
    rng = _seed(n, len(lengths))
    x = P.rollout(rng, n, offsets)
    say(f"policy of {len(lengths)} sequences, {n} tokens")
    P.check_policy(FULL, x, offsets, P.run_policy(FULL, x, offsets, shift=first % 4), f"{n}")


@pytest.mark.parametrize("lengths", LENGTHS, ids=range(len(LENGTHS)))
@pytest.mark.parametrize("first,behind", [(0, 0), (3, 2), (600, 700)])
def test_preference_of_long_sequences(lengths, first, behind):
    lengths = lengths + [77] * (len(lengths) % 2)
    offsets = _offsets(lengths, first)
    n, pairs = int(offsets[-1]) + behind, len(lengths) // 2
    rng = _seed(n, len(lengths), 1)
    x = P.rollout(rng, n)
    g = rng.standard_normal(pairs).astype(np.float32)
    say(f"preference of {pairs} pairs, {n} tokens")
    for v in (VARIANTS[0], VARIANTS[3]):
        got = P.run_preference(x, offsets, g, shift=first % 4, **v)
        P.check_preference(x, offsets, g, got, f"{n}", **v)
    got = P.run_preference(x, offsets, None)
    P.check_preference(x, offsets, None, got, f"{n} loss only")


def test_policy_sequences_that_start_late():
    rng = _seed(77)
    x = P.rollout(rng, 900)
    offsets = np.array([200, 350, 351, 700])             # tokens before the first one, too
    P.check_policy(FULL, x, offsets, P.run_policy(FULL, x, offsets), "late")


@pytest.mark.parametrize("offsets", [None, [0, 100, 5000, 40000]])
def test_policy_outputs_are_optional(offsets):
    x = P.rollout(_seed(4), 40000, offsets)
    full = P.run_policy(FULL, x, offsets)
    for name in full:
        one = P.run_policy(FULL, x, offsets, only=[name])
        assert np.array_equal(one[name], full[name]), name


@pytest.mark.parametrize("n", [700, 20000])
@pytest.mark.parametrize("seq", [False, True])
def test_policy_ignores_what_has_no_weight(n, seq):
    rng = _seed(n, 5)
    offsets = P.cuts(rng, n, 7) if seq else None
    x = P.rollout(rng, n, offsets, ignored=0.5)
    want = P.run_policy(FULL, x, offsets)
    out = x["w"] == 0
    for bad in (np.nan, np.inf, -np.inf):
        y = {k: v.copy() for k, v in x.items()}
        for k in ("lp", "A", "old", "ref", "H"):
            y[k][out] = bad
        got = P.run_policy(FULL, y, offsets)
        for name in want:
            assert np.array_equal(got[name], want[name]), (bad, name)
    nothing = {k: v.copy() for k, v in x.items()}
    nothing["w"][:] = 0
    got = P.run_policy(FULL, nothing, offsets)
    for name in got:
        assert (got[name] == 0).all(), name


def test_policy_bad_values_of_counted_tokens_stay_with_them():
    x = P.rollout(_seed(6), 20000, ignored=0.0)
    clean = P.run_policy(FULL, x)
    x["lp"][100], x["old"][5000], x["A"][19999] = np.nan, np.nan, np.nan
    got = P.run_policy(FULL, x)
    bad = np.zeros(20000, bool)
    bad[[100, 5000, 19999]] = True
    for name in ("loss", "dlogprob"):
        assert np.isnan(got[name][bad]).all() and np.array_equal(got[name][~bad],
                                                                 clean[name][~bad])
    assert np.isnan(got["totals"][0]) and got["counts"][0] == 20000


def test_policy_bad_advantage_reaches_its_whole_sequence():
    """A sequence's slope is the sum over its tokens, so one NaN makes it NaN, and no other's."""
    n, offsets = 3000, np.array([0, 700, 1500, 3000])
    x = P.rollout(_seed(61), n, offsets, ignored=0.0, spread=0.01)
    c = OP.constants()
    clean = P.run_policy(c, x, offsets)
    x["A"][900] = np.nan
    got = P.run_policy(c, x, offsets)
    assert np.isnan(got["dlogprob"][700:1500]).all() and np.isnan(got["loss"][900])
    for a, b in ((0, 700), (1500, 3000)):
        assert np.array_equal(got["dlogprob"][a:b], clean["dlogprob"][a:b])
    keep = np.arange(n) != 900
    assert np.array_equal(got["loss"][keep], clean["loss"][keep])


def test_policy_far_ratios():
    lp = np.array([-60.0, 0.0, -1e-3, -80.0, -1.0, -30.0], np.float32)
    old = np.array([0.0, -60.0, -1e-3, 0.0, -1.0 + 1e-6, -70.0], np.float32)
    ref = np.array([-40.0, -1e-5, -50.0, -79.9, -1.0, -30.3], np.float32)
    for A in (1.0, -1.0):
        x = dict(lp=lp, old=old, ref=ref, A=np.full(6, A, np.float32), w=np.ones(6, np.float32),
                 H=None)
        for c in (OP.constants(kl_coef=0.3), OP.constants(0.2, 0.2, 3.0, 0.3),
                  OP.constants(5.0, 1e30, 0, 0.3)):
            P.check_policy(c, x, None, P.run_policy(c, x), f"far A={A} {c}")


def test_policy_on_the_borders():
    """Ratios a last bit apart around the limits fall on the side that float64 says."""
    c = OP.constants(0.2, 0.2, 2.0)
    rows = []
    for border in (np.log1p(0.2), np.log1p(-0.2), np.log(2.0), 0.0):
        base = np.float32(border)
        v = np.nextafter(base, np.float32(-9))
        for _ in range(3):
            rows.append(v)
            v = np.nextafter(v, np.float32(9))
    lp = np.array(rows * 3, np.float32)
    n = len(lp)
    x = dict(lp=lp, old=np.zeros(n, np.float32), ref=None, H=None,
             A=np.repeat(np.float32([1, -1, 0]), len(rows)), w=np.ones(n, np.float32))
    P.check_policy(c, x, None, P.run_policy(c, x), "borders")


@pytest.mark.parametrize("offsets", [None, [0, 3, 11]])
def test_policy_gradient_matches_differences_of_the_kernel(offsets):
    """Central differences of the kernel's own total; its float32 rounding over 2 h bounds the
    difference quotient, as does h^2 times a third derivative of the size of the terms."""
    x = P.rollout(_seed(9), 11, offsets, ignored=0.0, spread=0.05)
    base = P.run_policy(FULL, x, offsets)
    S = (np.abs(x["w"]) * (np.abs(x["A"]) * 1.4 + 0.1 * 20 + 0.02 * 5)).sum()
    for t in range(11):
        up, down = dict(x, lp=x["lp"].copy()), dict(x, lp=x["lp"].copy())
        up["lp"][t] += np.float32(2.0 ** -8)
        down["lp"][t] -= np.float32(2.0 ** -8)
        h = float(up["lp"][t]) - float(down["lp"][t])
        d = (float(P.run_policy(FULL, up, offsets)["totals"][0])
             - float(P.run_policy(FULL, down, offsets)["totals"][0])) / h
        # a token whose ratio crosses a border within the step has no one gradient
        cut = [OP.policy(FULL, y["lp"], x["A"], x["w"], x["old"], x["ref"], x["H"], offsets)["cut"]
               for y in (up, down)]
        if np.array_equal(*cut):
            assert abs(d - base["dlogprob"][t]) <= 40 * P.U * S / h + 2.0 ** -14 * S, t


@pytest.mark.parametrize("n", [0, 40000])
def test_policy_without_tokens_or_sequences(n):
    f = dict(dtype=torch.float32, device="cuda")
    totals, counts = torch.full((4,), 55.0, **f), torch.full((2,), 55, dtype=torch.int64,
                                                             device="cuda")
    z = torch.zeros(n, **f)
    F.policy_loss(z, z, z, totals=totals, counts=counts,
                  offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))
    assert (totals == 0).all() and (counts == 0).all()


def test_policy_offsets_past_the_tokens():
    """The nearest valid value counts, so nothing outside the arrays is touched."""
    x = P.rollout(_seed(12), 1000)
    want = P.run_policy(FULL, x, [0, 400, 1000, 1000])
    got = P.run_policy(FULL, x, [-(1 << 63), 400, 1 << 50, (1 << 63) - 1])
    for name in want:
        assert np.array_equal(got[name], want[name]), name


@pytest.mark.parametrize("n,pairs,behind", [(2, 1, 0), (7, 1, 2), (300, 4, 9), (300, 200, 0),
                                            (3, 1, 0), (2560, 8, 1), (2560, 9, 0), (2561, 8, 0),
                                            (5000, 3, 0), (16384, 256, 1), (16384, 257, 0),
                                            (16385, 5, 100), (70001, 37, 0), (90000, 2, 80000)])
def test_preference(n, pairs, behind):
    rng = _seed(n, pairs, behind)
    offsets = P.cuts(rng, n, 2 * pairs, n - behind)
    x = P.rollout(rng, n, ignored=0.3)
    g = rng.standard_normal(pairs).astype(np.float32)
    g[rng.random(pairs) < 0.1] = 0
    for i, v in enumerate(VARIANTS):
        say(f"preference n={n} pairs={pairs} variant {i}")
        for weight, ref, dloss in ((True, True, g), (False, True, g), (True, False, None)):
            got = P.run_preference(x, offsets, dloss, shift=i % 4, weight=weight, ref=ref,
                                   rewards=i != 2, **v)
            P.check_preference(x, offsets, dloss, got, f"n={n} pairs={pairs} variant {i}",
                               weight=weight, ref=ref, **v)


def test_preference_ignores_what_has_no_weight():
    rng = _seed(31)
    for n in (900, 30000):
        offsets = P.cuts(rng, n, 10)
        x = P.rollout(rng, n, ignored=0.5)
        a, b = offsets[6], offsets[7]
        x["w"][a:b] = 0                                  # pair 3 loses a member
        g = np.ones(5, np.float32)
        want = P.run_preference(x, offsets, g)
        for bad in (np.nan, np.inf):
            y = {k: v.copy() for k, v in x.items()}
            for k in ("lp", "ref"):
                y[k][x["w"] == 0] = bad
            got = P.run_preference(y, offsets, g)
            for name in want:
                assert np.array_equal(got[name], want[name]), (n, bad, name)
        assert want["loss"][3] == 0 and (want["rewards"][3] == 0).all()
        assert (want["dlogprob"][offsets[6]:offsets[8]] == 0).all()


def test_preference_of_far_margins():
    """The logistic loss neither overflows nor loses the small side."""
    lp = np.array([0.0, -900.0, -900.0, 0.0, -1.0, -1.0], np.float32)
    x = dict(lp=lp, ref=np.zeros(6, np.float32), w=np.ones(6, np.float32))
    offsets = np.arange(7)
    for v in (dict(beta=1.0), dict(beta=1.0, label_smoothing=0.25), dict(beta=0.05)):
        got = P.run_preference(x, offsets, np.ones(3, np.float32), **v)
        P.check_preference(x, offsets, np.ones(3, np.float32), got, f"far {v}", **v)


def test_preference_gradient_matches_differences_of_the_kernel():
    rng = _seed(33)
    x = P.rollout(rng, 12, ignored=0.0)
    offsets = np.array([0, 2, 6, 9, 12])
    g = np.array([1.0, -2.0], np.float32)
    for v in (dict(beta=0.5, label_smoothing=0.1), dict(kind="squared", beta=0.5),
              dict(beta=1.0, length_normalised=True)):
        base = P.run_preference(x, offsets, g, **v)
        for t in range(12):
            up, down = dict(x, lp=x["lp"].copy()), dict(x, lp=x["lp"].copy())
            up["lp"][t] += np.float32(2.0 ** -7)
            down["lp"][t] -= np.float32(2.0 ** -7)
            h = float(up["lp"][t]) - float(down["lp"][t])
            lu, ld = (P.run_preference(y, offsets, None, **v)["loss"] for y in (up, down))
            d = float(((lu.astype(np.float64) - ld) * g).sum()) / h
            size = float((np.abs(lu) + np.abs(ld)) @ np.abs(g))
            # a rounding of each loss; the third derivative is at most beta^3 / 6 of w^3 <= 2
            assert abs(d - base["dlogprob"][t]) <= 2 * P.U * size / h + 2.0 ** -14 * 4, (v, t)


def test_repeated_calls_give_the_same_bits():
    rng = _seed(51)
    n = 300007
    offsets = P.cuts(rng, n, 200)
    x = P.rollout(rng, n, None)
    for off in (None, offsets):
        a, b = P.run_policy(FULL, x, off), P.run_policy(FULL, x, off)
        for name in a:
            assert np.array_equal(a[name].view(np.uint8), b[name].view(np.uint8)), name
    g = rng.standard_normal(100).astype(np.float32)
    a, b = P.run_preference(x, offsets, g), P.run_preference(x, offsets, g)
    for name in a:
        assert np.array_equal(a[name].view(np.uint8), b[name].view(np.uint8)), name


def test_beyond_2_31_tokens():
    """Places, chunks and counts pass 32 bits; all weight is on the last few tokens."""
    n, last = (1 << 31) + 1001, 300
    f = dict(dtype=torch.float32, device="cuda")
    lp, w, d = (torch.zeros(n, **f) for _ in range(3))
    lp[-last:] = -0.25
    w[-last:] = 0.5
    A = torch.ones(n, **f)
    old = torch.zeros(n, **f)                            # ratio e^-0.25 at the end
    totals, counts = torch.empty(4, **f), torch.empty(2, dtype=torch.int64, device="cuda")
    r = np.exp(np.float64(-0.25))
    for offsets in (None, torch.tensor([0, 7, n - 100, n]).cuda()):
        d.fill_(3)
        say(f"policy of {n} tokens, sequences: {offsets is not None}")
        F.policy_loss(lp, A, w, d, totals=totals, counts=counts, old_logprob=old, offsets=offsets)
        assert counts.tolist() == [last, 0]
        assert abs(float(totals[0]) + 0.5 * last * r) <= 1e-5 * last
        assert torch.allclose(d[-last:], torch.full((last,), float(-0.5 * r), **f), rtol=1e-6)
        assert float(d[:-last].abs().max()) == 0.0
    say(f"preference of {n} tokens")
    loss, won = torch.empty(1, **f), torch.empty(1, 2, **f)
    F.preference_loss(lp, torch.tensor([0, n - 100, n]).cuda(), loss, rewards=won, weight=w,
                      dloss=torch.ones(1, **f), dlogprob=d, beta=1.0)
    assert won.tolist() == [[-0.125 * 200, -0.125 * 100]]     # exact sums
    h = -12.5
    assert abs(float(loss) - np.log1p(np.exp(-h))) <= 1e-6 * abs(h)
    slope = -1 / (1 + np.exp(h))
    assert torch.allclose(d[-300:-100], torch.full((200,), float(0.5 * slope), **f), rtol=1e-6)
    assert torch.allclose(d[-100:], torch.full((100,), float(-0.5 * slope), **f), rtol=1e-6)
    assert float(d[:-300].abs().max()) == 0.0
