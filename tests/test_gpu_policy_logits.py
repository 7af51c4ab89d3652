"""The policy loss over logits on the GPU against the float64 oracles of the log probabilities and of
the loss.  Bounds: the log probability is off by E = unit(vocab) (1 + |d_y| + |log p_y|) (logits_cases),
which moves the ratio and exp(ref - lp) by E of themselves, on top of policy_cases' roundings; slope
errors move the gradient by c ([i = y] - p_i) of themselves, entropy errors by c p_i.  Ratios stay
1e-3 off the limits, where the last bit would decide."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say
from oracle import logits as OL
from oracle import policy as OP

pytestmark = pytest.mark.gpu
U = 2.0 ** -24

SHAPES = [(1, 1, 0, 0), (3, 2, 1, 1), (5, 7, 0, 3), (4, 63, 2, 0), (2, 257, 0, 1), (300, 33, 0, 0),
          (7, 1000, 24, 5), (2, 2048, 0, 0), (3, 4099, 0, 7), (5, 16384, 0, 0), (33, 8191, 0, 0),
          (2, 32000, 0, 0), (5, 50021, 0, 1), (3, 65536, 0, 0), (2, 65530, 0, 3),
          (1, 131077, 0, 2), (260, 9000, 0, 0), (2, 262144, 8, 0)]
TERMS = [OP.constants(0.2, 0.2, 0, 0, 0), OP.constants(0.2, 0.28, 1.5, 0.2, 0),
         OP.constants(0.1, 0.1, 0, 0.05, 0.3)]


def _seed(*key):
    return np.random.default_rng([int(v) for v in key] + [31])


def inputs(rng, x64, ids, scale, c):
    """old, ref, advantages and weights around the true log probabilities."""
    R, V = x64.shape
    lp = OL.token_logprobs(x64, ids, scale, 0)["logprob"]
    lp = np.where(np.isfinite(lp), lp, -1.0)
    d = rng.standard_normal(R) * 0.25
    borders = [np.log1p(c["clip_high"]), np.log1p(-c["clip_low"])]
    borders += [np.log(c["dual_clip"])] if c["dual_clip"] else []
    for b in borders:
        d = np.where(np.abs(d - b) < 2e-3, d + 5e-3, d)
    f = np.float32
    w = np.where(rng.random(R) < 0.15, 0, rng.random(R) + 0.2)
    return dict(old=(lp - d).astype(f), ref=(lp - rng.standard_normal(R) * 0.5).astype(f),
                A=rng.standard_normal(R).astype(f), w=w.astype(f))


def call(dev, ids, v, c, scale, out, entropy=True, **kw):
    R = dev.shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    got = dict(loss=torch.full((R,), 55.0, **f), logprob=torch.full((R,), 55.0, **f))
    if entropy:
        got["entropy"] = torch.full((R,), 55.0, **f)
    t = {k: None if x is None else torch.from_numpy(x).cuda() for k, x in v.items()}
    F.policy_logits_loss_grad(dev, torch.as_tensor(ids).cuda(), t["A"], t["w"], dlogits=out,
                              old_logprob=t["old"], ref_logprob=t["ref"], scale=scale, **got, **c,
                              **kw)
    return {k: x.cpu().numpy() for k, x in got.items()}


def check(x64, ids, v, c, scale, dtype, got, out, what):
    R, V = x64.shape
    counted = (ids >= 0) & (v["w"] != 0)
    past = counted & (ids >= V)
    first = OL.token_logprobs(x64, ids, scale, 0)
    lp = np.where(counted, first["logprob"], 0.0)
    H = np.where(counted, first["entropy"], 0.0)
    H[past] = np.nan
    ad, p, alp, aH, wide = C._moments(x64, scale)
    y, row = np.clip(ids, 0, V - 1), np.arange(R)
    unit = C.unit(V)
    size = 1 + ad[row, y] + alp[row, y]
    rest = np.where(lp == 0, 1, np.minimum(1, np.abs(np.nan_to_num(lp))))
    size = np.where(ad[row, y] == 0, rest, size)
    E = np.where(counted, unit * size, 0.0)
    C.close(got["logprob"], lp, E, what + " logprob")
    EH = unit * (np.minimum(1, aH) + aH + wide)
    if "entropy" in got:
        C.close(got["entropy"], H, np.where(counted, EH, 0), what + " entropy")
    # the loss, for rows whose log probability is a number
    fine = counted & np.isfinite(lp)
    w0 = np.where(fine, v["w"], 0)
    old = lp if v["old"] is None else v["old"].astype(np.float64)
    want = OP.policy(c, np.where(fine, lp, 0.0), v["A"], w0, np.where(fine, old, 0.0),
                     np.where(fine, v["ref"], 0.0), np.where(fine, H, 0.0))
    w, A = np.abs(w0).astype(np.float64), np.abs(v["A"].astype(np.float64))
    grow = np.abs(want["less1"]) + 1                    # exp(ref - lp) at most
    kl, eta = c["kl_coef"], abs(c["entropy_coef"])
    flow = np.where(want["cut"], 0, A * want["r"])
    move = flow * E + kl * grow * E
    S = np.abs(want["f"]) + kl * (want["k"] + np.abs(want["less1"])) + eta * np.abs(np.nan_to_num(H))
    loss = np.where(counted & ~fine, np.nan, want["loss"])
    C.close(got["loss"][~(counted & ~fine)], loss[~(counted & ~fine)],
            (w * (move + eta * EH + 20 * U * S))[~(counted & ~fine)], what + " loss")
    assert np.isnan(got["loss"][counted & np.isnan(lp)]).all(), what
    g = np.where(fine, want["dlogprob"], np.where(counted, np.nan, 0.0))
    h = np.where(counted, -c["entropy_coef"] * v["w"].astype(np.float64), 0.0)
    ok = ~counted | fine
    grad = np.zeros((R, V))
    grad[ok] = OL.token_logprobs_grad(x64[ok], np.where(counted, ids, -1)[ok], g[ok], h[ok], scale)
    grad[past | (counted & np.isnan(lp))] = np.nan
    ga, ha = np.abs(np.nan_to_num(g))[:, None], np.abs(h)[:, None]
    size = p * (ga * (1 + ad) + ha * ((1 + ad) * (1 + alp + aH[:, None]) + wide[:, None]))
    size[row, y] += ga[:, 0] * np.minimum(1 - p[row, y] + p[row, y] * ad[row, y], 1)
    dg = w * (move + 10 * U * (flow + kl * np.abs(want["less1"])))
    away = p.copy()
    away[row, y] = 1 - p[row, y]
    # The exponential flushes what is below 2^-126 to 0, and is then multiplied by c (g + h (log p + H))
    # with |log p| < 88 at that place: half of 2^-125 of that factor is lost.
    flushed = 2.0 ** -125 * (ga + ha * (88 + aH[:, None]))
    tol = scale * (unit * size + dg[:, None] * away + flushed) + C.half_step(grad, dtype)
    got_grad = out.double().cpu().numpy()
    settled = ok | past | (counted & np.isnan(lp))
    C.close(got_grad[settled], grad[settled], tol[settled], what + " dlogits")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, dtype):
    rows, vocab, pad, shift = shape
    rng = _seed(rows, vocab, pad, len(dtype))
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    dev, _ = C.on_device(t, pad, shift)
    ids = C.tokens(rng, rows, vocab)
    best = rng.random(rows) < 0.4
    ids[best] = np.argmax(x64[best], 1)
    scale = float(np.float32(0.8))
    for i, c in enumerate(TERMS):
        say(f"policy over logits {shape} {dtype} terms {i}")
        v = inputs(rng, x64, ids, scale, c)
        out, whole = C.filled_like(t, (pad + i) % 5, (shift + i) % 3)
        got = call(dev, ids, v, c, scale, out, entropy=i != 1)
        check(x64, ids, v, c, scale, dtype, got, out, f"{shape} {dtype} terms {i}")
        C.assert_between_rows_untouched(out, whole, f"{shape} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 9001, 70001])
def test_special_rows(vocab, dtype):
    rng = _seed(vocab, len(dtype), 5)
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    dev, _ = C.on_device(t, 0, 1)
    ids = rng.integers(0, vocab, 16)
    ids[[0, 9]] = -1, vocab                          # no token; past the vocabulary
    ids[12] = vocab // 3
    ids[3] = vocab // 2
    ids[1] = int(np.argmax(x64[1]))
    ids[15] = vocab - 1
    for i, c in enumerate(TERMS):
        say(f"policy over logits, special rows vocab={vocab} {dtype} terms {i}")
        v = inputs(rng, x64, ids, 1.0, c)
        v["w"][:] = 0.5
        v["w"][10] = 0
        out, whole = C.filled_like(t)
        got = call(dev, ids, v, c, 1.0, out)
        check(x64, ids, v, c, 1.0, dtype, got, out, f"special {vocab} {dtype} terms {i}")
        assert (out[2] == 0).all() and (out[0] == 0).all() and (out[10] == 0).all()
        assert out[[6, 7, 9]].isnan().all()


@pytest.mark.parametrize("vocab", [5000, 70001])
def test_rows_that_are_not_counted_are_not_read(vocab):
    rng = _seed(vocab, 6)
    x = C.plain_rows(rng, 8, vocab)
    t, x64 = C.to_dtype(x, "bf16")
    dev, _ = C.on_device(t)
    ids = rng.integers(0, vocab, 8)
    c = TERMS[2]
    v = inputs(rng, x64, ids, 1.0, c)
    ids[2], v["w"][5] = -1, 0
    dev[[2, 5]] = float("nan")
    for k in ("old", "ref", "A"):
        v[k][[2, 5]] = np.nan
    out, _ = C.filled_like(t)
    got = call(dev, ids, v, c, 1.0, out)
    assert (out[[2, 5]] == 0).all()
    for name in got:
        assert (got[name][[2, 5]] == 0).all() and np.isfinite(got[name]).all(), name


@pytest.mark.parametrize("dtype,rows,vocab", [("bf16", 9, 5003), ("fp32", 3, 50021),
                                              ("fp16", 5, 131077), ("bf16", 300, 9001)])
def test_in_place_and_without_old(dtype, rows, vocab):
    rng = _seed(rows, vocab, 7)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    ids, c = C.tokens(rng, rows, vocab), TERMS[2]
    v = inputs(rng, x64, ids, 1.0, c)
    for old in (v["old"], None):
        v = dict(v, old=old)
        dev, _ = C.on_device(t, 3, 1)
        apart, _ = C.filled_like(t, 3, 1)
        say(f"in place {dtype} {rows} x {vocab} old={old is not None}")
        a = call(dev, ids, v, c, 1.0, apart)
        check(x64, ids, v, c, 1.0, dtype, a, apart, "apart")
        b = call(dev, ids, v, c, 1.0, dev)
        check(x64, ids, v, c, 1.0, dtype, b, dev, "in place")


def test_matches_the_three_calls():
    """The joint call against token_logprobs, policy_loss and token_logprobs_grad."""
    rng = _seed(8)
    for dtype, rows, vocab in (("bf16", 700, 4001), ("fp32", 40, 40000)):
        t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
        dev = t.cuda()
        ids, c = C.tokens(rng, rows, vocab), TERMS[2]
        v = inputs(rng, x64, ids, 1.0, c)
        joint, _ = C.filled_like(t)
        got = call(dev, ids, v, c, 1.0, joint)
        f = dict(dtype=torch.float32, device="cuda")
        lp, H, g, h, loss = (torch.empty(rows, **f) for _ in range(5))
        stats = torch.empty(rows, 2, **f)
        idt = torch.from_numpy(ids).cuda()
        F.token_logprobs(dev, idt, logprob=lp, entropy=H, stats=stats)
        w = torch.from_numpy(v["w"]).cuda() * (idt >= 0)
        F.policy_loss(lp, torch.from_numpy(v["A"]).cuda(), w, g, loss=loss,
                      old_logprob=torch.from_numpy(v["old"]).cuda(),
                      ref_logprob=torch.from_numpy(v["ref"]).cuda(), entropy=H, dentropy=h, **c)
        out, _ = C.filled_like(t)
        F.token_logprobs_grad(dev, idt, stats, out, dlogprob=g, entropy=H, dentropy=h)
        check(x64, ids, v, c, 1.0, dtype, dict(got, loss=loss.cpu().numpy()), out, "three calls")
        check(x64, ids, v, c, 1.0, dtype, got, joint, "joint")


def test_far_from_zero():
    rng = _seed(41)
    for vocab in (700, 40001):
        x = 1e4 + 0.02 * rng.standard_normal((3, vocab))
        x[1] = -1e4 + 0.02 * rng.standard_normal(vocab)
        x[2] = 3.0 * rng.standard_normal(vocab)
        t, x64 = C.to_dtype(x, "fp32")
        dev, _ = C.on_device(t, 1, 1)
        ids = rng.integers(0, vocab, 3)
        v = inputs(rng, x64, ids, 300.0, TERMS[2])
        out, _ = C.filled_like(t)
        got = call(dev, ids, v, TERMS[2], 300.0, out)
        check(x64, ids, v, TERMS[2], 300.0, "fp32", got, out, f"far {vocab}")


def test_beyond_2_31_elements():
    rows, vocab = 66000, 32768
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    ids = torch.full((rows,), 5, device="cuda")
    loss = torch.empty(rows, **f)
    say("policy over logits beyond 2^31 elements, in place")
    F.policy_logits_loss_grad(x, ids, torch.ones(rows, **f), torch.ones(rows, **f), loss, x)
    assert (loss == -1).all()                            # ratio 1, advantage 1
    last = x[rows - 1].float()
    assert float(last[5]) == -1.0 and float(last[vocab - 1]) == 2.0 ** -15
