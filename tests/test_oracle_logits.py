"""Pins of the oracle's operators over logits: closed forms, PyTorch in float64 (values and
autograd), central differences, and the conventions for masks and bad rows."""

import math

import numpy as np
import pytest
import torch

from oracle import logits as OL


def _x(seed, rows=4, vocab=11, std=3.0):
    return np.random.default_rng(seed).standard_normal((rows, vocab)) * std


def test_uniform_and_peaked_rows_have_closed_forms():
    out = OL.token_logprobs(np.zeros((1, 8)), [3], top_k=3)
    assert out["logprob"][0] == pytest.approx(-math.log(8), rel=1e-15)
    assert out["entropy"][0] == pytest.approx(math.log(8), rel=1e-15)
    assert out["top_ids"][0].tolist() == [0, 1, 2]            # ties: the lowest index first
    x = np.full((1, 5), -40.0)
    x[0, 2] = 0.0
    out = OL.token_logprobs(x, [2])
    rest = 4 * math.exp(-40.0)
    assert out["logprob"][0] == pytest.approx(-rest, rel=1e-12)   # not lost next to 1
    # the type's lowest value is an ordinary logit
    out = OL.token_logprobs(np.full((1, 4), -3.4e38), [0])
    assert out["logprob"][0] == pytest.approx(-math.log(4), rel=1e-15)


@pytest.mark.parametrize("scale", [1.0, 0.5, 1 / 0.7])
def test_logprobs_and_gradient_match_torch(scale):
    x = _x(1)
    ids = [0, 10, 4, 7]
    g, h = np.array([1.0, -0.5, 0.0, 2.0]), np.array([0.0, 0.3, -1.0, 0.1])
    out = OL.token_logprobs(x, ids, scale, top_k=4)
    t = torch.tensor(x, requires_grad=True)
    lp = torch.log_softmax(t * scale, 1)
    H = -(lp.exp() * lp).sum(1)
    at = lp[torch.arange(4), torch.tensor(ids)]
    np.testing.assert_allclose(out["logprob"], at.detach().numpy(), rtol=1e-13)
    np.testing.assert_allclose(out["entropy"], H.detach().numpy(), rtol=1e-13)
    top = lp.detach().topk(4, 1)
    assert (out["top_ids"] == top.indices.numpy()).all()
    np.testing.assert_allclose(out["top_logprobs"], top.values.numpy(), rtol=1e-13)
    ((at * torch.tensor(g)).sum() + (H * torch.tensor(h)).sum()).backward()
    np.testing.assert_allclose(OL.token_logprobs_grad(x, ids, g, h, scale), t.grad.numpy(),
                               rtol=1e-11, atol=1e-14)


def _torch_distill(t, ids, values, scale, tail):
    """The loss written with torch, for lists of distinct tokens."""
    lp = torch.log_softmax(t * scale, 1)
    v = torch.tensor(values)
    if not tail:
        lq = torch.log_softmax(v * scale, 1)
        return (lq.exp() * (lq - lp.gather(1, torch.tensor(ids)))).sum(1)
    q = v.exp()
    loss = (q * (v - lp.gather(1, torch.tensor(ids)))).sum(1)
    rest = 1 - q.sum(1)
    pt = 1 - lp.exp().gather(1, torch.tensor(ids)).sum(1)
    return loss + rest * (rest.log() - pt.log())


@pytest.mark.parametrize("tail", [False, True])
def test_distill_and_gradient_match_torch(tail):
    x, scale = _x(2), 0.7
    teacher = torch.log_softmax(torch.tensor(_x(3)) * 0.4, 1)
    values, ids = (a.numpy() for a in teacher.topk(3, 1))
    g = np.array([1.0, 0.5, -2.0, 0.25])
    t = torch.tensor(x, requires_grad=True)
    want = _torch_distill(t, ids, values, scale, tail)
    loss, stats = OL.distill_topk(x, ids, values, scale, tail)
    np.testing.assert_allclose(loss, want.detach().numpy(), rtol=1e-11)
    (want * torch.tensor(g)).sum().backward()
    np.testing.assert_allclose(OL.distill_topk_grad(x, ids, values, g, scale, tail),
                               t.grad.numpy(), rtol=1e-9, atol=1e-13)


@pytest.mark.parametrize("tail", [False, True])
def test_distill_gradient_matches_differences(tail):
    """Also with empty places and a token that stands twice.  Central differences with step e err
    by e^2/6 times the third derivative (at most 2 here, probabilities' products): about 1e-9 for
    e = 5e-5, and by rounding, 1e-16 times the loss over e."""
    x = _x(5, rows=2, vocab=7)
    ids = np.array([[2, 5, 2, -1], [0, -1, 6, 3]])
    values = np.log(np.array([[0.3, 0.2, 0.1, 0.9], [0.5, 0.9, 0.2, 0.1]]))
    g = np.array([1.0, -1.5])
    grad = OL.distill_topk_grad(x, ids, values, g, 0.8, tail)
    e = 5e-5
    for r in range(2):
        for i in range(7):
            hi, lo = x.copy(), x.copy()
            hi[r, i] += e
            lo[r, i] -= e
            diff = (OL.distill_topk(hi, ids, values, 0.8, tail)[0][r]
                    - OL.distill_topk(lo, ids, values, 0.8, tail)[0][r]) / (2 * e)
            assert abs(g[r] * diff - grad[r, i]) < 1e-8


def test_logprob_gradient_matches_differences():
    x, ids, scale, e = _x(6, rows=2, vocab=6), [1, 4], 1.3, 5e-5
    g, h = np.array([0.7, -0.4]), np.array([0.2, 1.1])
    grad = OL.token_logprobs_grad(x, ids, g, h, scale)

    def value(x, r):
        o = OL.token_logprobs(x, ids, scale)
        return g[r] * o["logprob"][r] + h[r] * o["entropy"][r]

    for r in range(2):
        for i in range(6):
            hi, lo = x.copy(), x.copy()
            hi[r, i] += e
            lo[r, i] -= e
            assert abs((value(hi, r) - value(lo, r)) / (2 * e) - grad[r, i]) < 1e-7


def test_masked_empty_and_bad_rows():
    inf, nan = np.inf, np.nan
    x = np.array([[1.0, -inf, 2.0], [-inf, -inf, -inf], [0.0, nan, 1.0], [0.0, inf, 1.0],
                  [0.0, 1.0, 2.0], [0.0, 1.0, 2.0]])
    ids = [1, 0, 0, 1, -5, 3]
    o = OL.token_logprobs(x, ids, top_k=4)
    assert o["logprob"][0] == -inf and o["logprob"][1] == -inf and o["logprob"][4] == 0.0
    assert np.isnan(o["logprob"][[2, 3, 5]]).all()
    assert o["entropy"][1] == 0.0 and np.isnan(o["entropy"][[2, 3]]).all()
    assert o["top_ids"][0].tolist() == [2, 0, -1, -1]
    assert o["top_ids"][1].tolist() == [-1] * 4 and o["top_ids"][2].tolist() == [-1] * 4
    assert o["top_ids"][5].tolist() == [2, 1, 0, -1]
    d = OL.token_logprobs_grad(x, ids, np.ones(6), np.zeros(6))
    assert (d[1] == 0).all() and np.isnan(d[2]).all() and (d[4] == 0).all()
    assert np.isnan(d[5]).all() and d[0, 1] == 1.0      # -g expm1(-inf)
    assert (OL.token_logprobs_grad(x, ids, np.zeros(6), np.zeros(6)) == 0).all()


def test_distill_conventions():
    x = np.array([[0.0, 1.0, 2.0]])
    v = np.log(np.array([[0.25, 0.75]]))
    none = np.array([[-1, -1]])
    assert OL.distill_topk(x * np.nan, none, v)[0][0] == 0.0
    assert (OL.distill_topk_grad(x * np.nan, none, v, [1.0]) == 0).all()
    assert np.isnan(OL.distill_topk(x, [[0, 3]], v)[0][0])
    masked = np.array([[0.0, -np.inf, 2.0]])
    assert OL.distill_topk(masked, [[0, 1]], v)[0][0] == np.inf
    # nothing outside the list: the rest of the teacher's mass is dropped
    loss, stats = OL.distill_topk(x, [[0, 1, 2]], np.log([[0.2, 0.2, 0.5]]), tail=True)
    assert math.isfinite(loss[0]) and stats[0, 2] == -np.inf
    # a teacher equal to the student has no divergence and no gradient
    lp = (x - x.max()) - math.log(np.exp(x - x.max()).sum())
    for tail in (False, True):
        assert abs(OL.distill_topk(x, [[0, 1, 2]], lp, tail=tail)[0][0]) < 1e-15
        assert np.abs(OL.distill_topk_grad(x, [[0, 1, 2]], lp, [1.0], tail=tail)).max() < 1e-15
