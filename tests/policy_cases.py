"""Inputs, error bounds and checks shared by the GPU tests of the policy and preference losses.

Error bounds, with u = 2^-24 (half a step of float32).  Log ratios d and e are float64 differences of
float32 values, off by 2^-53 of themselves.
  * r = exp d: an exponential good to a step (2 u), a factor 1 + l rounded (u), a product (u): 4 u.
  * f = r A, or a float32 limit (u) times A: 5 u.  The slope w r A: 6 u.
  * exp(e) - 1: a step (2 u), one fused multiply-add with a sum rounded before it (2 u): 4 u.
  * k: beyond |e| = 1/2 (where exp(e) - 1 is 0.65 and -0.39) the same 4 u of exp(e) - 1, a
    difference (u of its size) and another (u of k); below it 2 u of e's rounding, and the series'
    coefficients, steps and products, 8 u: in all 10 u k + 5 u |exp(e) - 1| beyond it, 10 u k below.
  * The loss adds f, kl_coef k and entropy_coef H in float32: two roundings of a constant and a
    product each, two of the sums, each at most the sum S of the three sizes, and the weight's.
  * A sequence's slope comes from float64 sums: r's 4 u and a rounding; then the KL term is added.
  * Totals are float64 sums of float32 values: their tokens' bounds added up, and one rounding.
Denormals aside (2^-120, in logits_cases.close).
"""

import numpy as np
import torch

import fsdp_sharded_optimizer_layout_amd as F
from logits_cases import close
from oracle import policy as OP

U = 2.0 ** -24
KEYS = ("lp", "A", "w", "old", "ref", "H")


def rollout(rng, n, offsets=None, old=True, ref=True, entropy=True, ignored=0.2, spread=0.25):
    """float32 arrays of n tokens (None where not wanted); with offsets, a sequence's tokens drift
    together."""
    f = np.float32
    lp = np.log(rng.random(n) + 1e-7).astype(f)
    d = rng.standard_normal(n) * spread
    if offsets is not None:
        for a, b in zip(offsets, offsets[1:]):
            d[a:b] = rng.standard_normal() * spread + 0.2 * d[a:b]
    w = np.where(rng.random(n) < ignored, 0, rng.random(n) + 0.1).astype(f)
    return dict(lp=lp, A=rng.standard_normal(n).astype(f), w=w,
                old=(lp - d).astype(f) if old else None,
                ref=(lp - rng.standard_normal(n) * 0.6).astype(f) if ref else None,
                H=(rng.random(n) * 5).astype(f) if entropy else None)


def shifted(x, shift=0):
    """x (numpy) on the GPU, ``shift`` elements past the start of an allocation."""
    if x is None:
        return None
    buf = torch.zeros(x.size + shift + 8, dtype=torch.from_numpy(x).dtype, device="cuda")
    buf[shift:shift + x.size] = torch.from_numpy(x).cuda()
    return buf[shift:shift + x.size]


def run_policy(c, x, offsets=None, shift=0, only=None, **kw):
    """dict of the outputs (numpy, 55 where nothing was written)."""
    n = len(x["lp"])
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(loss=torch.full((n,), 55.0, **f), dlogprob=torch.full((n,), 55.0, **f),
               dentropy=torch.full((n,), 55.0, **f), totals=torch.full((4,), 55.0, **f),
               counts=torch.full((2,), 55, dtype=torch.int64, device="cuda"))
    out = {k: v for k, v in out.items() if only is None or k in only}
    d = {k: shifted(x[k], shift) for k in KEYS}
    off = None if offsets is None else torch.as_tensor(np.asarray(offsets, np.int64)).cuda()
    F.policy_loss(d["lp"], d["A"], d["w"], old_logprob=d["old"], ref_logprob=d["ref"],
                  entropy=d["H"], offsets=off, **c, **out, **kw)
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_policy(c, x, offsets, got, what):
    n = len(x["lp"])
    want = OP.policy(c, x["lp"], x["A"], x["w"], x["old"], x["ref"], x["H"], offsets)
    counted = want["inside"] & (x["w"] != 0)
    w, A = np.abs(np.where(counted, x["w"], 0)).astype(np.float64), x["A"].astype(np.float64)
    H = np.zeros(n) if x["H"] is None else np.abs(x["H"].astype(np.float64))
    far = 5 * np.abs(want["less1"]) * ((want["less1"] > 0.6) | (want["less1"] < -0.38))
    kl, eta = c["kl_coef"], abs(c["entropy_coef"])
    tol_k = 10 * want["k"] + far
    S = np.abs(want["f"]) + kl * want["k"] + eta * H
    tol_loss = U * w * (5 * np.abs(want["f"]) + kl * (tol_k + 2 * want["k"]) + 2 * eta * H + 4 * S)
    flow = np.where(want["cut"] | ~counted, 0, w * np.abs(A) * want["r"])
    klslope = w * kl * np.abs(want["less1"])
    if offsets is None:
        pull = flow
    else:
        pull = np.abs(want["dlogprob"] + np.where(counted, x["w"], 0) * kl * want["less1"])
    inside = want["inside"]
    assert np.array_equal(got["loss"][~inside], np.full((~inside).sum(), 55.0)), what
    assert np.array_equal(got["dlogprob"][~inside], np.full((~inside).sum(), 55.0)), what
    assert np.array_equal(got["dentropy"][~inside], np.full((~inside).sum(), 55.0)), what
    close(got["loss"][inside], want["loss"][inside], tol_loss[inside], what + " loss")
    close(got["dlogprob"][inside], want["dlogprob"][inside],
          U * (8 * pull + 8 * klslope)[inside], what + " dlogprob")
    close(got["dentropy"][inside], want["dentropy"][inside], 2 * U * eta * w[inside],
          what + " dentropy")
    sizes = np.array([tol_loss.sum(), U * (5 * w * np.abs(want["f"])).sum(),
                      U * (w * tol_k).sum(), U * (w * H).sum()])
    close(got["totals"], want["totals"], sizes + U * np.abs(want["totals"]), what + " totals")
    assert got["counts"].tolist() == want["counts"].tolist(), what + " counts"


def cuts(rng, n, sequences, end=None):
    """Rising offsets over the first `end` tokens: some sequences empty, some of one token."""
    end = n if end is None else end
    c = np.sort(rng.integers(0, end + 1, sequences + 1))
    c[0], c[-1] = 0, end
    if sequences > 5:
        c[2] = c[1]                                     # an empty one
        c[3] = min(c[2] + 1, c[4])
    return np.maximum.accumulate(c)


def run_preference(x, offsets, dloss=None, shift=0, weight=True, ref=True, rewards=True, **kw):
    n, pairs = len(x["lp"]), (len(offsets) - 1) // 2
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(loss=torch.full((pairs,), 55.0, **f))
    if rewards:
        out["rewards"] = torch.full((pairs, 2), 55.0, **f)
    if dloss is not None:
        out["dlogprob"] = torch.full((n,), 55.0, **f)
    F.preference_loss(shifted(x["lp"], shift), torch.as_tensor(np.asarray(offsets, np.int64)).cuda(),
                      ref_logprob=shifted(x["ref"], shift) if ref else None,
                      weight=shifted(x["w"], shift) if weight else None,
                      dloss=None if dloss is None else torch.from_numpy(dloss).cuda(), **out, **kw)
    return {k: v.cpu().numpy() for k, v in out.items()}


def check_preference(x, offsets, dloss, got, what, weight=True, ref=True, kind="logistic", beta=0.1,
                     margin=0.0, label_smoothing=0.0, length_normalised=False):
    """Scores are float64 sums, off by about 2^-50 of their terms' sizes (a chain of a few dozen
    additions), the loss by its slope times that, through |1 / (2 beta)| and the margin where they
    are added; then one rounding to float32, and two for a token's gradient."""
    want = OP.preference(x["lp"], offsets, x["ref"] if ref else None, x["w"] if weight else None,
                         dloss, kind, beta, margin, label_smoothing, length_normalised)
    slack = 2.0 ** -46 * (want["size"] + abs(margin) + 1 / beta)
    steep = {"logistic": beta, "hinge": beta}.get(kind) or 2 * (want["size"] + abs(margin)
                                                                + 1 / beta)
    close(got["loss"], want["loss"], U * np.abs(want["loss"]) + steep * slack + beta * slack,
          what + " loss")
    if "rewards" in got:
        close(got["rewards"], want["rewards"],
              U * np.abs(want["rewards"]) + beta * slack[:, None], what + " rewards")
    if "dlogprob" in got:
        inside = want["inside"]
        assert np.array_equal(got["dlogprob"][~inside], np.full((~inside).sum(), 55.0)), what
        w = np.abs(x["w"]).astype(np.float64) if weight else np.ones(len(x["lp"]))
        move = np.zeros(len(x["lp"]))
        for p in range(len(dloss)):
            # the slope moves by at most beta^2 (logistic) or 2 (squared) of the score
            a, b = offsets[2 * p], offsets[2 * p + 2]
            move[a:b] = abs(dloss[p]) * max(beta ** 2, 2.0 * (kind == "squared")) * slack[p]
        close(got["dlogprob"][inside], want["dlogprob"][inside],
              (3 * U * np.abs(want["dlogprob"]) + move * w)[inside], what + " dlogprob")
