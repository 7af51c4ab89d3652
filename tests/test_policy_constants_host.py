"""Constants of the policy loss that float32, in which a token's terms are added up, does not hold:
refused, since their product with a term of 0 would be NaN.  No GPU: every call stops in the checks,
or has nothing to do."""

import ctypes

import pytest

import fsdp_sharded_optimizer_layout_amd as F
from test_policy_host import INVALID, OK, _logits, _terms, over_logits, policy

LARGEST = (2 - 2.0 ** -23) * 2.0 ** 127


@pytest.mark.parametrize("name", ["dual_clip", "kl_coef", "entropy_coef"])
def test_constants_beyond_float32_are_refused(name):
    for bad in (1e39, 1.7e308, LARGEST * (1 + 2.0 ** -24)):
        assert policy(terms=_terms(**{name: bad})) == INVALID, bad
        assert over_logits(terms=_terms(**{name: bad})) == INVALID, bad
    none = dict(tokens=0, totals=None, counts=None)
    assert policy(terms=_terms(**{name: LARGEST}), **none) == OK
    assert over_logits(x=_logits(rows=0, data=None), terms=_terms(**{name: LARGEST})) == OK


def test_an_entropy_coefficient_of_either_sign():
    assert policy(terms=_terms(entropy_coef=-1e39)) == INVALID
    assert policy(terms=_terms(entropy_coef=-LARGEST), tokens=0, totals=None, counts=None) == OK


def test_limits_beyond_float32_are_no_limits():
    none = dict(tokens=0, totals=None, counts=None)
    assert policy(terms=_terms(clip_high=1e300), **none) == OK
    assert ctypes.sizeof(F._Policy) == 40
