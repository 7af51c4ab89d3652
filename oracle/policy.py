"""Losses of post-training over log probabilities in float64 (oracle; test infrastructure only),
token by token and pair by pair from the definitions:

  r = exp(lp - old), f = min(r A, clip(r, 1 - low, 1 + high) A), for A < 0 at least dual A,
  k = exp(ref - lp) - (ref - lp) - 1,  loss = w (-f + kl k - eta H)

with lp - old the mean over a sequence's counted tokens where they share one ratio; and for a pair of
sequences of scores s = sum w (lp - ref) [/ sum w]: h = beta (s_c - s_r) - margin, and the logistic,
hinge or squared loss of it.  A token of weight 0 is not counted.
"""

import math

import numpy as np


def _growth(e):
    """(exp(e) - 1, exp(e) - e - 1), the second one without cancellation near 0."""
    less1 = math.expm1(e) if e < 700 else math.inf
    if abs(e) < 1e-2:
        return less1, sum(e ** n / math.factorial(n) for n in range(2, 9))
    return less1, less1 - e


def _token(c, w, A, d, lp, ref, H, flow=None):
    """dict of one counted token's values; `d` is its (or its sequence's) log ratio."""
    r = math.exp(d) if d < 700 else math.inf
    cut = (A > 0 and d > math.log1p(c["clip_high"])) or \
        (A < 0 and (c["clip_low"] < 1 and d < math.log1p(-c["clip_low"]) or
                    c["dual_clip"] > 0 and d > math.log(c["dual_clip"])))
    f = min(r * A, min(max(r, 1 - c["clip_low"]), 1 + c["clip_high"]) * A)
    if c["dual_clip"] > 0 and A < 0:
        f = max(f, c["dual_clip"] * A)
    if not cut:
        f = r * A
    less1, k = _growth(ref - lp) if ref is not None else (0.0, 0.0)
    loss = w * (-f + c["kl_coef"] * k - (c["entropy_coef"] * H if H is not None else 0.0))
    return dict(r=r, cut=cut, f=f, k=k, less1=less1, loss=loss)


def constants(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0):
    return dict(clip_low=clip_low, clip_high=clip_high, dual_clip=dual_clip, kl_coef=kl_coef,
                entropy_coef=entropy_coef)


def policy(c, lp, A, w, old=None, ref=None, H=None, offsets=None):
    """dict(loss, dlogprob, dentropy, totals, counts, inside, and the pieces f, k, less1, r, cut)."""
    n = len(lp)
    out = {k: np.zeros(n) for k in ("loss", "dlogprob", "dentropy", "f", "k", "less1", "r")}
    out["cut"], out["inside"] = np.zeros(n, bool), np.zeros(n, bool)
    groups = [[t] for t in range(n)] if offsets is None else \
        [list(range(a, b)) for a, b in zip(offsets, offsets[1:])]
    totals, counts = np.zeros(4), np.zeros(2, np.int64)
    for group in groups:
        out["inside"][group] = True
        group = [t for t in group if w[t] != 0]
        if not group:
            continue
        ratios = [float(lp[t]) - float(old[t]) if old is not None else 0.0 for t in group]
        d = math.fsum(ratios) / len(group) if offsets is not None else ratios[0]
        flows = []
        for t in group:
            x = _token(c, float(w[t]), float(A[t]), d, float(lp[t]),
                       None if ref is None else float(ref[t]), None if H is None else float(H[t]))
            for name in ("loss", "f", "k", "less1", "r", "cut"):
                out[name][t] = x[name]
            if not x["cut"]:
                flows.append(float(w[t]) * float(A[t]))
            out["dlogprob"][t] = -float(w[t]) * c["kl_coef"] * x["less1"]
            out["dentropy"][t] = -c["entropy_coef"] * float(w[t])
            totals += [x["loss"], -float(w[t]) * x["f"], float(w[t]) * x["k"],
                       0.0 if H is None else float(w[t]) * float(H[t])]
            counts += [1, int(x["cut"])]
        r = math.exp(d) if d < 700 else math.inf
        if not flows:                           # 0, also where r is inf
            continue
        for t in group:
            out["dlogprob"][t] -= r * math.fsum(flows) / len(group)
    out["totals"], out["counts"] = totals, counts
    return out


def preference(lp, offsets, ref=None, w=None, dloss=None, kind="logistic", beta=0.1, margin=0.0,
               smoothing=0.0, normalised=False):
    """dict(loss, rewards, dlogprob, inside, size): size is each pair's sum of |w (lp - ref)|."""
    n, pairs = len(lp), (len(offsets) - 1) // 2
    out = dict(loss=np.zeros(pairs), rewards=np.zeros((pairs, 2)), dlogprob=np.zeros(n),
               inside=np.zeros(n, bool), size=np.zeros(pairs))
    for p in range(pairs):
        score, norm, members = [], [], []
        for s in (2 * p, 2 * p + 1):
            every = range(offsets[s], offsets[s + 1])
            out["inside"][list(every)] = True
            toks = [t for t in every if w is None or w[t] != 0]
            ws = [1.0 if w is None else float(w[t]) for t in toks]
            gaps = [float(lp[t]) - (0.0 if ref is None else float(ref[t])) for t in toks]
            terms = [a * b for a, b in zip(ws, gaps)]
            norm.append(math.fsum(ws) if normalised else 1.0)
            members.append((toks, ws))
            score.append(math.fsum(terms) / norm[-1] if toks else 0.0)
            out["size"][p] += sum(abs(x) for x in terms) / (abs(norm[-1]) if toks else 1.0)
        if not members[0][0] or not members[1][0]:
            continue
        lead = score[0] - score[1]
        h = beta * lead - margin
        if kind == "logistic":
            # -(1 - smoothing) log sigmoid(h) - smoothing log sigmoid(-h); a factor of 0 leaves its
            # term out, also where h is infinite
            small = math.log1p(math.exp(-abs(h)))
            loss = sum(a * (small + max(z, 0.0))
                       for a, z in ((1 - smoothing, -h), (smoothing, h)) if a)
            slope = beta * (smoothing - 1 / (1 + math.exp(min(h, 700))))
        elif kind == "hinge":
            loss, slope = max(0.0, 1 - h), -beta if h < 1 else 0.0
        else:
            away = lead - margin - 1 / (2 * beta)
            loss, slope = away ** 2, 2 * away
        out["loss"][p], out["rewards"][p] = loss, [beta * x for x in score]
        if dloss is not None and dloss[p] != 0:
            for sign, (toks, ws), m in zip((1, -1), members, norm):
                for t, a in zip(toks, ws):
                    out["dlogprob"][t] = sign * slope * float(dloss[p]) / m * a
    return out
