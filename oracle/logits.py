"""Operators over logits in float64 (oracle; test infrastructure only).

Token log probabilities with entropy and top alternatives, and distillation from a teacher's top
logits, each with its gradient, row by row from the definitions:

  d_i = c (x_i - max x),  L = log sum exp d,  log p_i = d_i - L

A logit of -inf has p = 0; a row of only -inf has p = 0 everywhere (statistics -inf, entropy 0,
gradient 0); a NaN or +inf makes a row's results NaN.  Nothing here is rounded to the logits' type.
"""

import math

import numpy as np


def _row(x, scale):
    """(state, m, L, log p) of one row; state is "ok", "empty" or "nan"."""
    x = np.asarray(x, np.float64)
    if np.isnan(x).any() or (x == np.inf).any():
        return "nan", np.nan, np.nan, np.full(x.size, np.nan)
    m = x.max() if x.size else -np.inf
    if m == -np.inf:
        return "empty", m, m, np.full(x.size, -np.inf)
    d = scale * (x - m)
    e = np.exp(d)
    e[int(np.argmax(x))] = 0.0
    L = math.log1p(math.fsum(e.tolist()))
    return "ok", m, L, d - L


def token_logprobs(x, ids, scale=1.0, top_k=0):
    """dict(logprob, entropy, stats, top_ids, top_logprobs) of the rows of ``x``."""
    x = np.asarray(x, np.float64)
    R, V = x.shape
    out = dict(logprob=np.zeros(R), entropy=np.zeros(R), stats=np.zeros((R, 2)),
               top_ids=np.full((R, top_k), -1, np.int64),
               top_logprobs=np.full((R, top_k), -np.inf))
    for r in range(R):
        state, m, L, logp = _row(x[r], scale)
        out["stats"][r] = m, L
        y = int(ids[r])
        out["logprob"][r] = 0.0 if y < 0 else (np.nan if y >= V else logp[y])
        if state == "nan":
            out["entropy"][r] = np.nan
            out["top_logprobs"][r] = np.nan
        elif state == "ok":
            some = logp > -np.inf
            out["entropy"][r] = -math.fsum((np.exp(logp[some]) * logp[some]).tolist())
            order = np.lexsort((np.arange(V), -x[r]))
            order = order[x[r][order] > -np.inf][:top_k]
            out["top_ids"][r, :order.size] = order
            out["top_logprobs"][r, :order.size] = logp[order]
    return out


def token_logprobs_grad(x, ids, g, h, scale=1.0):
    """Gradient of the logits for gradients g of the log probability and h of the entropy."""
    x = np.asarray(x, np.float64)
    R, V = x.shape
    out = np.zeros((R, V))
    for r in range(R):
        y = int(ids[r])
        gr = float(g[r]) if y >= 0 else 0.0
        hr = float(h[r])
        if gr == 0.0 and hr == 0.0:
            continue
        state, m, L, logp = _row(x[r], scale)
        if state == "nan" or y >= V:
            out[r] = np.nan
            continue
        if state == "empty":
            continue
        p = np.exp(logp)
        some = p > 0
        H = -math.fsum((p[some] * logp[some]).tolist())
        slope = np.zeros(V)
        slope[some] = p[some] * (logp[some] + H)
        dx = -gr * p - hr * slope
        if gr != 0.0:
            dx[y] = -gr * math.expm1(logp[y]) - hr * slope[y]
        out[r] = scale * dx
    return out


def _teacher(ids, values, scale, tail):
    """(places, log q, q, q_t, bad) of one row's list (Python lists; empty places left out); a
    list is bad when it holds a value of NaN or +inf."""
    places = [(int(i), float(v)) for i, v in zip(ids, values) if i >= 0]
    if not places:
        return [], [], [], 0.0, False
    v = [p[1] for p in places]
    if any(math.isnan(a) or a == math.inf for a in v):
        return [p[0] for p in places], v, v, 0.0, True
    if tail:
        logq = v
    else:
        top = max(scale * a for a in v)
        if top == -math.inf:
            logq = [-math.inf] * len(v)
        else:
            s = math.fsum(math.exp(scale * a - top) for a in v)
            logq = [scale * a - top - math.log(s) for a in v]
    q = [math.exp(a) for a in logq]
    rest = 1.0 - math.fsum(q) if tail else 0.0
    return [p[0] for p in places], logq, q, max(0.0, rest), False


def distill_topk(x, ids, values, scale=1.0, tail=False):
    """(loss, stats) of the rows."""
    x = np.asarray(x, np.float64)
    R, V = x.shape
    loss, stats = np.zeros(R), np.zeros((R, 4))
    for r in range(R):
        place, logq, q, rest, bad = _teacher(ids[r], values[r], scale, tail)
        if not place:
            continue
        state, m, L, logp = _row(x[r], scale)
        stats[r, :2] = m, L
        inside = np.zeros(V, bool)
        inside[[i for i in place if i < V]] = True
        if tail:
            tstate, mt, Lt, _ = _row(np.where(inside, -np.inf, x[r]), scale)
            if state == "nan":
                mt = Lt = np.nan
            if mt == -np.inf:
                rest = 0.0                      # nothing of the student's is outside the list
            stats[r, 2:] = mt, Lt
        if state == "nan" or bad or any(i >= V for i in place):
            loss[r] = np.nan
            continue
        terms = [a * (b - logp[i]) for i, a, b in zip(place, q, logq) if a > 0]
        if tail and rest > 0:
            logpt = scale * (mt - m) + Lt - L
            terms.append(rest * (math.log(rest) - logpt))
        loss[r] = math.inf if math.inf in terms else math.fsum(terms)
    return loss, stats


def distill_topk_grad(x, ids, values, g, scale=1.0, tail=False):
    x = np.asarray(x, np.float64)
    R, V = x.shape
    out = np.zeros((R, V))
    for r in range(R):
        place, logq, q, rest, bad = _teacher(ids[r], values[r], scale, tail)
        gr = float(g[r])
        if not place or gr == 0.0:
            continue
        state, m, L, logp = _row(x[r], scale)
        if state == "nan" or bad or any(i >= V for i in place):
            out[r] = np.nan
            continue
        if state == "empty":
            continue
        dense = np.zeros(V)
        for i, a in zip(place, q):
            dense[i] += a
        inside = np.zeros(V, bool)
        inside[place] = True
        outside = np.where(inside, -np.inf, x[r])
        if outside.max() == -np.inf:
            rest = 0.0
        dx = (math.fsum(q) + rest) * np.exp(logp) - dense
        if rest > 0:
            dx -= rest * np.exp(_row(outside, scale)[3])
        out[r] = gr * scale * dx
    return out
