"""Pins of the oracles of the policy and preference losses where a ratio or a margin is infinite."""

import numpy as np

from oracle import policy as OP

INF = np.inf


def test_a_clipped_sequence_has_no_slope_at_an_infinite_ratio():
    c = OP.constants(dual_clip=3.0)
    for old in ([-1000.0, -900.0], [-INF, -1.0]):
        for A in ([1.0, 2.0], [-1.0, -2.0], [1.0, -2.0]):
            out = OP.policy(c, [-1.0, -1.0], A, [0.5, 0.5], old, offsets=[0, 2])
            assert out["dlogprob"].tolist() == [0.0, 0.0] and out["counts"].tolist() == [2, 2]
            assert np.isfinite(out["loss"]).all()
    out = OP.policy(OP.constants(), [-1.0, -1.0], [-1.0, 1.0], [0.5, 0.5], [-1000.0, -900.0],
                    offsets=[0, 2])
    assert out["dlogprob"].tolist() == [INF, INF]            # A < 0 is not clipped above


def test_a_bad_advantage_is_in_its_sequences_slope():
    out = OP.policy(OP.constants(dual_clip=3.0), [-1.0] * 3, [np.nan, 1.0, 1.0], [1.0] * 3,
                    [-5.0, -5.0, -1.0], offsets=[0, 2, 3])
    assert np.isnan(out["dlogprob"][:2]).all() and out["dlogprob"][2] == -1.0


def test_preference_at_infinite_margins():
    lp = [-1.0, -INF, -INF, -1.0]
    for s in (0.0, 0.25):
        out = OP.preference(lp, range(5), dloss=[1.0, 1.0], beta=0.5, smoothing=s)
        assert out["loss"].tolist() == [INF if s else 0.0, INF]
        np.testing.assert_allclose(out["dlogprob"],
                                   [0.5 * s, -0.5 * s, 0.5 * (s - 1), -0.5 * (s - 1)], atol=1e-300)
