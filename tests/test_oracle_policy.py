"""Pins of the oracles of the policy and preference losses and of the embedding: closed forms,
PyTorch's autograd in float64, central differences, and the conventions."""

import math

import numpy as np
import pytest
import torch

from oracle import embedding as OE
from oracle import policy as OP


def _tokens(seed, n):
    rng = np.random.default_rng(seed)
    lp = np.log(rng.random(n))
    return rng, lp, lp - rng.standard_normal(n) * 0.3, lp - rng.standard_normal(n) * 0.4, \
        rng.standard_normal(n), np.where(rng.random(n) < 0.2, 0, rng.random(n)), rng.random(n) * 3


def _torch_policy(c, lp, A, w, old, ref, H, offsets):
    d = lp - old
    if offsets is not None:
        parts = []
        for a, b in zip(offsets, offsets[1:]):
            keep = (w[a:b] != 0).double()
            parts.append((d[a:b] * keep).sum() / keep.sum().clamp_min(1) + 0 * d[a:b])
        d = torch.cat(parts)
    r = d.exp()
    f = torch.minimum(r * A, r.clamp(1 - c["clip_low"], 1 + c["clip_high"]) * A)
    if c["dual_clip"]:
        f = torch.where(A < 0, torch.maximum(f, c["dual_clip"] * A), f)
    k = (ref - lp).exp() - (ref - lp) - 1
    return (w * (-f + c["kl_coef"] * k - c["entropy_coef"] * H)).sum()


@pytest.mark.parametrize("offsets", [None, [0, 7, 7, 8, 30, 41]])
@pytest.mark.parametrize("dual", [0.0, 1.3])
def test_policy_matches_torch(offsets, dual):
    rng, lp, old, ref, A, w, H = _tokens(3, 41)
    if offsets is not None:
        old = lp - 0.3 * rng.standard_normal(5).repeat(np.diff(offsets))
    c = OP.constants(0.1, 0.15, dual, 0.3, 0.2)
    out = OP.policy(c, lp, A, w, old, ref, H, offsets)
    t = {k: torch.tensor(v, dtype=torch.float64) for k, v in
         dict(lp=lp, A=A, w=w, old=old, ref=ref, H=H).items()}
    t["lp"].requires_grad_()
    t["H"].requires_grad_()
    total = _torch_policy(c, t["lp"], t["A"], t["w"], t["old"], t["ref"], t["H"], offsets)
    total.backward()
    assert out["totals"][0] == pytest.approx(float(total.detach()), rel=1e-12)
    assert out["loss"].sum() == pytest.approx(float(total.detach()), rel=1e-12)
    np.testing.assert_allclose(out["dlogprob"], t["lp"].grad.numpy(), rtol=1e-10, atol=1e-14)
    np.testing.assert_allclose(out["dentropy"], t["H"].grad.numpy(), rtol=1e-12, atol=0)
    assert 0 < out["counts"][1] < out["counts"][0] == (w != 0).sum()


@pytest.mark.parametrize("offsets", [None, [0, 4, 9]])
def test_policy_gradient_matches_differences(offsets):
    _, lp, old, ref, A, w, H = _tokens(5, 9)
    c = OP.constants(0.2, 0.2, 2.0, 0.1, 0.05)
    base = OP.policy(c, lp, A, w, old, ref, H, offsets)
    for t in range(9):
        e = 1e-6
        up, down = lp.copy(), lp.copy()
        up[t] += e
        down[t] -= e
        num = (OP.policy(c, up, A, w, old, ref, H, offsets)["totals"][0]
               - OP.policy(c, down, A, w, old, ref, H, offsets)["totals"][0]) / (2 * e)
        assert base["dlogprob"][t] == pytest.approx(num, rel=1e-6, abs=1e-9)


def test_policy_closed_forms():
    c = OP.constants(kl_coef=0.5)
    lp = np.array([-1.0, -1.0, -2.0])
    out = OP.policy(c, lp, [1.0, -1.0, 1.0], [1.0, 0.5, 0.0], None, lp, None)
    assert out["loss"].tolist() == [-1.0, 0.5, 0.0]           # ratio 1, no divergence
    assert out["dlogprob"].tolist() == [-1.0, 0.5, 0.0]
    out = OP.policy(OP.constants(), [0.0, 0.0], [1.0, -1.0], [1, 1], [-1.0, 1.0])
    assert out["loss"].tolist() == [-1.2, 0.8] and out["counts"].tolist() == [2, 2]
    assert out["dlogprob"].tolist() == [0.0, 0.0]
    less1, k = OP._growth(1e-9)
    assert k == pytest.approx(5e-19, rel=1e-8) and less1 == pytest.approx(1e-9, rel=1e-8)


@pytest.mark.parametrize("kind", ["logistic", "hinge", "squared"])
@pytest.mark.parametrize("normalised", [False, True])
def test_preference_matches_torch(kind, normalised):
    rng, lp, _, ref, _, w, _ = _tokens(7, 50)
    offsets = [0, 9, 20, 29, 34, 34, 50]                     # the last pair has an empty member
    g = rng.standard_normal(3)
    eps = 0.2 if kind == "logistic" else 0.0
    out = OP.preference(lp, offsets, ref, w, g, kind, 0.7, 0.3, eps, normalised)
    t = torch.tensor(lp, requires_grad=True)
    s = [(torch.tensor(w) * (t - torch.tensor(ref)))[a:b].sum() /
         (w[a:b].sum() if normalised else 1.0) for a, b in zip(offsets, offsets[1:])]
    total = 0
    for p in range(2):
        lead = s[2 * p] - s[2 * p + 1]
        h = 0.7 * lead - 0.3
        sure = torch.nn.functional.logsigmoid
        loss = {"logistic": -(1 - eps) * sure(h) - eps * sure(-h), "hinge": torch.relu(1 - h),
                "squared": (lead - 0.3 - 1 / 1.4) ** 2}[kind]
        assert out["loss"][p] == pytest.approx(float(loss.detach()), rel=1e-12)
        assert out["rewards"][p, 0] == pytest.approx(0.7 * float(s[2 * p].detach()), rel=1e-12)
        total = total + g[p] * loss
    total.backward()
    np.testing.assert_allclose(out["dlogprob"], t.grad.numpy(), rtol=1e-11, atol=1e-15)
    assert out["loss"][2] == 0 and (out["dlogprob"][34:] == 0).all()


def test_preference_of_equal_sequences():
    out = OP.preference([-1.0, -1.0], [0, 1, 2], dloss=[2.0], beta=0.5)
    assert out["loss"][0] == pytest.approx(math.log(2), rel=1e-15)
    assert out["dlogprob"].tolist() == [-0.5, 0.5]            # -beta / 2 times 2


def test_embedding_matches_torch():
    rng = np.random.default_rng(2)
    table, ids = rng.standard_normal((6, 4)), [5, -1, 0, 5, 2]
    t = torch.tensor(table, requires_grad=True)
    out = torch.nn.functional.embedding(torch.tensor([5, 0, 0, 5, 2]), t) * 1.5
    want = out.detach().numpy().copy()
    want[1] = 0
    assert np.array_equal(OE.lookup(table, ids, 1.5), want)
    assert np.isnan(OE.lookup(table, [6])).all()
    dout = rng.standard_normal((5, 4))
    keep = torch.tensor([1.0, 0, 1, 1, 1], dtype=torch.float64)[:, None]
    (out * torch.tensor(dout) * keep).sum().backward()
    d, size, count = OE.grad(ids, dout, 6, 1.5)
    np.testing.assert_allclose(d, t.grad.numpy(), rtol=1e-14)
    assert count.tolist() == [1, 0, 1, 0, 0, 2] and (size >= np.abs(d) - 1e-15).all()
    # by differences
    e = 1e-6
    for v, j in ((5, 1), (2, 3), (1, 0)):
        up, down = table.copy(), table.copy()
        up[v, j] += e
        down[v, j] -= e
        num = ((OE.lookup(up, ids, 1.5) - OE.lookup(down, ids, 1.5)) * dout).sum() / (2 * e)
        assert d[v, j] == pytest.approx(num, rel=1e-6, abs=1e-9)
