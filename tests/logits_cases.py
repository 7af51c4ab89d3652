"""Inputs, error bounds and checks shared by the GPU tests of the operators over logits.

Error bounds.  With u = 2^-24 (half a step of float32) and d = c (x - m):
  * d is two float32 roundings of a value of size |d|, its exponential's argument one or two more
    and the exponential itself good to a step: exp d is off by at most u (4 |d| + 4), relatively;
    terms with |d| > 88 are below 1e-38 and do not count, and most of a row's sum comes from
    |d| < 32.
  * A float32 sum of n terms of one sign in which every partial sum is the result of at most a
    chain of a additions is off by at most a u, relatively; a = vocab / 256 + 64 covers one
    partial sum for each of 256 threads, a tree over them and a merge of splits.
  * So a row's sum, its log-sum L and everything built on them is off by at most
    unit(vocab) = u (256 + vocab / 256) times the sizes of the quantities that enter:
    1, |d|, |log p|, H, and for the entropy the sum of p (|d| + d^2).
  * A float32 value below 2^-126 is denormal: it has an absolute step, or is flushed to 0.  A few
    of them (times factors up to 4 here) make at most 2^-120, which every bound includes.
  * One rounding to the output's type comes last: eps / 2 relative, or half a denormal step.
"""

import numpy as np
import torch

import fsdp_sharded_optimizer_layout_amd as F
from oracle import logits as OL

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = np.inf


def unit(vocab):
    return 2.0 ** -24 * (256 + vocab / 256)


def to_dtype(x, dtype):
    """x (numpy) rounded to the type: (torch CPU tensor, the values held as float64)."""
    t = torch.from_numpy(np.asarray(x, np.float32)).to(DTYPES[dtype])
    return t, t.to(torch.float64).numpy()


def on_device(t, pad=0, shift=0):
    """The rows of ``t`` on the GPU, vocab + pad elements apart and ``shift`` elements past the
    start of an allocation; (view, whole buffer)."""
    rows, vocab = t.shape
    stride = vocab + pad
    buf = torch.full((shift + rows * stride + 8,), float("nan"), dtype=t.dtype)
    view = buf[shift:shift + rows * stride].view(rows, stride)[:, :vocab]
    view.copy_(t)
    dev = buf.cuda()
    return dev[shift:shift + rows * stride].view(rows, stride)[:, :vocab], dev


def filled_like(t, pad=0, shift=0):
    """A gradient buffer of t's shape and type filled with a pattern; (view, whole buffer)."""
    rows, vocab = t.shape
    stride = vocab + pad
    dev = torch.full((shift + rows * stride + 8,), 77.0, dtype=t.dtype, device="cuda")
    return dev[shift:shift + rows * stride].view(rows, stride)[:, :vocab], dev


def assert_between_rows_untouched(view, whole, what):
    """The elements of ``whole`` outside ``view`` still hold the pattern of filled_like."""
    inside = torch.zeros(whole.numel(), dtype=torch.bool)
    off = (view.data_ptr() - whole.data_ptr()) // whole.element_size()
    stride = view.stride(0) if view.shape[0] > 1 else view.shape[1]
    for r in range(view.shape[0]):
        inside[off + r * stride: off + r * stride + view.shape[1]] = True
    assert (whole.cpu()[~inside] == 77.0).all(), f"{what}: written outside the rows"


def close(got, want, tol, what):
    got, want, tol = np.broadcast_arrays(np.asarray(got, np.float64), want, tol)
    tol = tol + 2.0 ** -120
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        ok = same | (np.isfinite(want) & (np.abs(got - want) <= tol))
    if not ok.all():
        i = np.argwhere(~ok)[:5].tolist()
        at = [tuple(j) for j in i]
        raise AssertionError(f"{what}: {(~ok).sum()} of {ok.size} off, e.g. {at}: got "
                             f"{[got[j] for j in at]}, want {[want[j] for j in at]}, "
                             f"allowed {[tol[j] for j in at]}")


def _moments(x, scale):
    """(|d|, p, log p, H, sum p (|d| + d^2)) of the rows; zeros where a row has no numbers."""
    m = x.max(1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = scale * (x - m)
        e = np.exp(d)
        s = e.sum(1, keepdims=True)
        p = np.nan_to_num(e / s)
        ad = np.where(np.isfinite(d), np.abs(d), 0.0)
        lp = np.where(np.isfinite(d), d - np.log(s), 0.0)
        lp = np.nan_to_num(lp, posinf=0.0, neginf=0.0)
        wide = (p * (ad + np.where(p > 0, ad, 0.0) ** 2)).sum(1)
        H = -(p * lp).sum(1)
    return ad, p, np.abs(lp), np.abs(H), wide


def check_logprobs(x64, ids, scale, k, got, what):
    """got: dict of numpy arrays logprob, entropy, stats, top_ids, top_logprobs (any may be
    missing)."""
    R, V = x64.shape
    want = OL.token_logprobs(x64, ids, scale, k)
    U = unit(V)
    ad, p, lp, H, wide = _moments(x64, scale)
    if "logprob" in got:
        y = np.clip(ids, 0, V - 1)
        size = 1 + ad[np.arange(R), y] + lp[np.arange(R), y]
        rest = np.where(want["logprob"] == 0, 1, np.minimum(1, np.abs(want["logprob"])))
        # a row's most likely token: its log probability is -L, exact relative to its own size
        size = np.where(ad[np.arange(R), y] == 0, rest, size)
        close(got["logprob"], want["logprob"], U * size, what + " logprob")
    if "entropy" in got:
        close(got["entropy"], want["entropy"], U * (np.minimum(1, H) + H + wide),
              what + " entropy")
    if "stats" in got:
        assert np.array_equal(got["stats"][:, 0].astype(np.float64), want["stats"][:, 0],
                              equal_nan=True), what + " maximum"
        L = want["stats"][:, 1]
        close(got["stats"][:, 1], L, U * np.nan_to_num(np.minimum(1, np.abs(L)) + np.abs(L),
                                                       posinf=0), what + " log-sum")
    if k and "top_ids" in got:
        assert np.array_equal(got["top_ids"], want["top_ids"]), \
            f"{what} top ids: {got['top_ids']} want {want['top_ids']}"
        idx = np.clip(want["top_ids"], 0, V - 1)
        size = 1 + np.take_along_axis(ad, idx, 1) + np.take_along_axis(lp, idx, 1)
        close(got["top_logprobs"], want["top_logprobs"], U * size, what + " top logprobs")


def half_step(want, dtype):
    """The roundings of a gradient's last operations.  An entry is g c dx: dx, g c and their
    product are float32 values, each off by at most u = 2^-24 of itself, so the product is off by
    at most 3 u of itself (and terms of u^2, within the 1e-6 below) where dx itself is exact; then
    comes half a step of the type (its smallest step where the value is denormal)."""
    info = torch.finfo(DTYPES[dtype])
    size = np.abs(np.nan_to_num(want, posinf=0, neginf=0))
    return (np.maximum(size * info.eps / 2, info.tiny * info.eps / 2)
            + 3 * 2.0 ** -24 * size) * (1 + 1e-6)


def check_logprobs_grad(x64, ids, g, h, scale, dtype, got, what):
    R, V = x64.shape
    want = OL.token_logprobs_grad(x64, ids, g, h, scale)
    ad, p, lp, H, wide = _moments(x64, scale)
    ga, ha = np.abs(g)[:, None], np.abs(h)[:, None]
    size = p * (ga * (1 + ad) + ha * ((1 + ad) * (1 + lp + H[:, None]) + wide[:, None]))
    y = np.clip(ids, 0, V - 1)
    row = np.arange(R)
    # at the token itself: g (1 - p), where 1 - p keeps its relative precision
    size[row, y] += np.abs(g) * np.minimum(1 - p[row, y] + p[row, y] * ad[row, y], 1)
    close(got, want, scale * unit(V) * size + half_step(want, dtype), what)


def _teacher_arrays(ids, values):
    ids = np.asarray(ids)
    return ids, np.asarray(values, np.float32).astype(np.float64)


def check_distill(x64, ids, values, scale, tail, loss, stats, what):
    R, V = x64.shape
    ids, values = _teacher_arrays(ids, values)
    want, wstats = OL.distill_topk(x64, ids, values, scale, tail)
    ad, p, lp, H, wide = _moments(x64, scale)
    U = unit(V)
    tol = np.zeros(R)
    for r in range(R):
        place, logq, q, rest, bad = OL._teacher(ids[r], values[r], scale, tail)
        if bad or any(i >= V for i in place):
            continue
        tol[r] = sum(a * (1 + ad[r, i] + lp[r, i] + abs(b))
                     for i, a, b in zip(place, q, logq) if a > 0)
        if rest > 0 and np.isfinite(wstats[r]).all():
            tol[r] += rest * (2 + abs(scale * (wstats[r, 0] - wstats[r, 2])) + wstats[r, 3]
                              + wstats[r, 1] + abs(np.log(rest)))
    close(loss, want, U * tol, what + " loss")
    if stats is not None:
        for j in (0, 2):
            assert np.array_equal(stats[:, j].astype(np.float64), wstats[:, j], equal_nan=True), \
                f"{what} maximum: {stats[:, j]} want {wstats[:, j]}"
        for j in (1, 3):
            L = wstats[:, j]
            close(stats[:, j], L, U * np.nan_to_num(np.minimum(1, np.abs(L)) + np.abs(L),
                                                    posinf=0), what + " log-sum")
    return want


def check_distill_grad(x64, ids, values, g, scale, tail, dtype, got, what):
    R, V = x64.shape
    ids, values = _teacher_arrays(ids, values)
    want = OL.distill_topk_grad(x64, ids, values, g, scale, tail)
    ad, p, lp, H, wide = _moments(x64, scale)
    size = p * (1 + ad)
    for r in range(R):
        place, logq, q, rest, bad = OL._teacher(ids[r], values[r], scale, tail)
        if not place or bad:
            size[r] = 0
            continue
        if not tail:
            size[r] *= sum(q)
        elif rest > 0 and max(place) < V:
            size[r] *= sum(q) + rest
            outside = x64[r].copy()
            outside[place] = -INF
            if np.isfinite(outside).any():
                pad = _moments(outside[None], scale)
                size[r] += rest * (pad[1] * (1 + pad[0]))[0]
    close(got, want, np.abs(g)[:, None] * scale * unit(V) * size + half_step(want, dtype), what)


# ------------------------------------------------------------------------------------ inputs

def plain_rows(rng, rows, vocab, std=3.0):
    return rng.standard_normal((rows, vocab)) * std


def special_rows(rng, vocab, dtype):
    """One row of each kind that goes wrong easily."""
    low = float(torch.finfo(DTYPES[dtype]).min)
    x = [plain_rows(rng, 1, vocab)[0] for _ in range(16)]
    x[1][rng.random(vocab) < 0.7] = -INF                    # masked here and there
    x[2][:] = -INF                                          # nothing left
    x[3][:] = -INF
    x[3][vocab // 2] = 1.5                                  # one survivor
    x[4][:] = low                                           # masked by the lowest value
    x[5][rng.random(vocab) < 0.5] = low
    x[6][vocab - 1] = np.nan
    x[7][0] = INF
    x[8][:] = 0.25                                          # all equal
    x[9] = np.round(x[9])                                   # a few values, many ties
    x[10] = np.sort(x[10])
    x[11] = np.sort(x[11])[::-1].copy()
    x[12][:] = -30.0
    x[12][vocab // 3] = 10.0                                # almost sure of one token
    x[13] *= 1e3
    x[14][:] = np.where(rng.random(vocab) < 0.5, 0.0, -0.0)
    x[15][: vocab // 2] = -INF                              # the first half masked
    return np.stack(x)


def tokens(rng, rows, vocab):
    ids = rng.integers(0, vocab, rows)
    ids[rng.random(rows) < 0.2] = -100
    return ids


def teacher_lists(rng, x64, k, tail):
    """Lists drawn around the student's own likely tokens, values log probabilities (of a total
    below 1 for the tail), some places empty, some lists empty, some tokens twice."""
    R, V = x64.shape
    ids = np.zeros((R, k), np.int32)
    for r in range(R):
        ids[r] = rng.integers(0, V, k)
        best = np.argsort(-np.nan_to_num(x64[r], nan=0, posinf=0))[:max(1, k // 2)]
        ids[r, :best.size] = best
        if k <= V and rng.random() < 0.6:
            ids[r] = rng.permutation(V)[:k]
    w = rng.random((R, k)) ** 3 + 1e-6
    share = rng.uniform(0.3, 1.0, (R, 1)) if tail else 1.0
    values = np.log(w / w.sum(1, keepdims=True) * share).astype(np.float32)
    ids[rng.random((R, k)) < 0.1] = -1
    if R > 3:
        ids[rng.integers(0, R)] = -1
    if k > 1 and R > 1:
        ids[1, k - 1] = ids[1, 0]
        values[0, k - 1] = -INF                              # a place without mass
    return ids, values


# ------------------------------------------------------------------------------------- calls

def run_logprobs(dev, ids, scale, k, **kw):
    R = dev.shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(logprob=torch.full((R,), 55.0, **f), entropy=torch.full((R,), 55.0, **f),
               stats=torch.full((R, 2), 55.0, **f),
               top_ids=torch.full((R, k), 55, dtype=torch.int32, device="cuda"),
               top_logprobs=torch.full((R, k), 55.0, **f))
    F.token_logprobs(dev, torch.as_tensor(ids, dtype=torch.int64).cuda(), scale=scale, **out, **kw)
    return out


def host(out):
    return {n: t.float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()
            for n, t in out.items()}
