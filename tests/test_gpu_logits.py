"""Token log probabilities and top-k distillation on the GPU against the float64 oracle, with the
error bounds of logits_cases: sizes from one row and one token up, odd sizes, every type, strides
and phases, masks, empty and bad rows, ties, lists with empty and repeated places, in place, on
side streams, in a captured graph, and beyond 2^31 elements."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say
from oracle import logits as OL

pytestmark = pytest.mark.gpu

# (rows, vocab, pad between rows, shift of the base): one token, less than a vector, odd sizes,
# more than one work-group's tile, sizes around whole tiles, few rows of a large vocabulary.
SHAPES = [(1, 1, 0, 0), (3, 2, 1, 1), (5, 7, 0, 3), (4, 63, 2, 0), (2, 257, 0, 1),
          (300, 33, 0, 0), (7, 1000, 24, 5), (2, 2048, 0, 0), (3, 4099, 0, 7), (33, 8191, 0, 0),
          (2, 32000, 0, 0), (5, 50021, 0, 1), (1, 131077, 0, 2), (2, 262144, 8, 0)]


def _seed(*key):
    return np.random.default_rng([int(v) for v in key] + [17])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_logprobs_shapes(shape, dtype):
    rows, vocab, pad, shift = shape
    rng = _seed(rows, vocab, pad, len(dtype))
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    dev, _ = C.on_device(t, pad, shift)
    ids = C.tokens(rng, rows, vocab)
    for k, scale in ((0, 1.0), (1, 0.5), (20, 1.0), (128, 1 / 0.7)):
        say(f"logprobs {shape} {dtype} k={k}")
        got = C.host(C.run_logprobs(dev, ids, float(np.float32(scale)), k))
        C.check_logprobs(x64, ids, float(np.float32(scale)), k, got, f"{shape} {dtype} k={k}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 1003, 9000, 70001])
def test_logprobs_special_rows(vocab, dtype):
    rng = _seed(vocab, len(dtype), 3)
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    dev, _ = C.on_device(t, 0, 1)
    ids = rng.integers(0, vocab, 16)
    ids[[0, 9]] = -1, vocab                          # no token; past the vocabulary
    ids[12] = vocab // 3
    for k in (1, 5, 64, 128):
        say(f"logprobs special rows vocab={vocab} {dtype} k={k}")
        got = C.host(C.run_logprobs(dev, ids, 1.0, k))
        C.check_logprobs(x64, ids, 1.0, k, got, f"special {vocab} {dtype} k={k}")


@pytest.mark.parametrize("vocab", [2999, 40000])
def test_top_lists_where_the_best_stand_together(vocab):
    """The best values in one run of neighbours, in one residue class modulo a power of two, or
    all equal up to one: what a selection by partial maxima finds hardest."""
    rng = _seed(vocab, 9)
    x = C.plain_rows(rng, 6, vocab)
    x[0, 1000:1400] += 50
    x[1, 5::256] += 50
    x[2, 8::2048] += 50
    x[3] = 1.0
    x[3, vocab - 3] = 2.0
    x[4] = np.where(np.arange(vocab) % 3 == 0, 1.0, -1.0)
    x[5] = -np.inf
    x[5, vocab - 70:] = 0.5
    for dtype in ("bf16", "fp32"):
        t, x64 = C.to_dtype(x, dtype)
        dev, _ = C.on_device(t)
        for k in (3, 64, 128):
            say(f"top lists vocab={vocab} {dtype} k={k}")
            got = C.host(C.run_logprobs(dev, np.zeros(6, np.int64), 1.0, k))
            C.check_logprobs(x64, np.zeros(6, np.int64), 1.0, k, got, f"{vocab} {dtype} k={k}")


def test_logprobs_outputs_are_optional():
    rng = _seed(4, 4)
    t, x64 = C.to_dtype(C.plain_rows(rng, 4, 5000), "bf16")
    dev, _ = C.on_device(t)
    ids = C.tokens(rng, 4, 5000)
    full = C.run_logprobs(dev, ids, 1.0, 7)
    one = torch.empty(4, device="cuda")
    F.token_logprobs(dev, torch.as_tensor(ids).cuda(), logprob=one)
    assert torch.equal(one, full["logprob"])
    F.token_logprobs(dev, entropy=one)
    assert torch.equal(one, full["entropy"])
    st = torch.empty(4, 2, device="cuda")
    F.token_logprobs(dev, stats=st)
    assert torch.equal(st, full["stats"])
    i, v = torch.empty(4, 7, dtype=torch.int32, device="cuda"), torch.empty(4, 7, device="cuda")
    F.token_logprobs(dev, top_ids=i, top_logprobs=v)
    assert torch.equal(i, full["top_ids"]) and torch.equal(v, full["top_logprobs"])


def _forward_state(dev, ids, scale):
    out = C.run_logprobs(dev, ids, scale, 0)
    return out["stats"], out["entropy"]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_logprobs_grad_shapes(shape, dtype):
    rows, vocab, pad, shift = shape
    rng = _seed(rows, vocab, pad, len(dtype), 2)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    dev, _ = C.on_device(t, pad, shift)
    ids = C.tokens(rng, rows, vocab)
    g = rng.standard_normal(rows).astype(np.float32)
    h = rng.standard_normal(rows).astype(np.float32)
    g[rng.random(rows) < 0.2] = 0
    h[rng.random(rows) < 0.2] = 0
    scale = float(np.float32(0.8))
    stats, entropy = _forward_state(dev, ids, scale)
    idt = torch.as_tensor(ids).cuda()
    zero = np.zeros(rows, np.float32)
    for gg, hh, opad, oshift in ((g, None, pad, shift), (None, h, 0, 0), (g, h, 3, 1)):
        say(f"logprobs grad {shape} {dtype} g={gg is not None} h={hh is not None}")
        out, whole = C.filled_like(t, opad, oshift)
        F.token_logprobs_grad(dev, idt, stats, out, scale=scale,
                              dlogprob=None if gg is None else torch.from_numpy(gg).cuda(),
                              entropy=None if hh is None else entropy,
                              dentropy=None if hh is None else torch.from_numpy(hh).cuda())
        C.check_logprobs_grad(x64, ids, zero if gg is None else gg, zero if hh is None else hh,
                              scale, dtype, out.double().cpu().numpy(), f"{shape} {dtype}")
        C.assert_between_rows_untouched(out, whole, f"{shape} {dtype}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 9001])
def test_logprobs_grad_special_rows(vocab, dtype):
    rng = _seed(vocab, len(dtype), 5)
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    dev, _ = C.on_device(t)
    ids = rng.integers(0, vocab, 16)
    ids[[0, 9]] = -1, vocab
    ids[12] = vocab // 3
    ids[3] = vocab // 2
    stats, entropy = _forward_state(dev, ids, 1.0)
    for g, h in ((1.0, 0.0), (0.0, 1.0), (0.5, -0.25), (0.0, 0.0)):
        say(f"logprobs grad special rows vocab={vocab} {dtype} g={g} h={h}")
        out, whole = C.filled_like(t)
        gv, hv = np.full(16, g, np.float32), np.full(16, h, np.float32)
        F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), stats, out,
                              dlogprob=torch.from_numpy(gv).cuda(), entropy=entropy,
                              dentropy=torch.from_numpy(hv).cuda())
        C.check_logprobs_grad(x64, ids, gv, hv, 1.0, dtype, out.double().cpu().numpy(),
                              f"special {vocab} {dtype} g={g} h={h}")


def test_gradients_in_place():
    rng = _seed(8, 1)
    for dtype, pad, shift in (("bf16", 0, 1), ("fp32", 5, 0), ("fp16", 3, 2)):
        t, x64 = C.to_dtype(C.plain_rows(rng, 9, 5003), dtype)
        ids, ones = C.tokens(rng, 9, 5003), np.ones(9, np.float32)
        dev, _ = C.on_device(t, pad, shift)
        apart, _ = C.filled_like(t, pad, shift)
        stats, entropy = _forward_state(dev, ids, 1.0)
        kw = dict(dlogprob=torch.from_numpy(ones).cuda(), entropy=entropy,
                  dentropy=torch.from_numpy(ones).cuda())
        say(f"in place {dtype}")
        F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), stats, apart, **kw)
        F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), stats, dev, **kw)
        assert torch.equal(dev, apart)
        for tail in (False, True):
            tid, tv = C.teacher_lists(rng, x64, 20, tail)
            tid, tv = torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda()
            f = dict(dtype=torch.float32, device="cuda")
            loss, st, g = torch.empty(9, **f), torch.empty(9, 4, **f), torch.ones(9, **f)
            dev, _ = C.on_device(t, pad, shift)
            F.distill_topk(dev, tid, tv, loss, st, tail=tail)
            F.distill_topk_grad(dev, tid, tv, st, g, apart, tail=tail)
            F.distill_topk_grad(dev, tid, tv, st, g, dev, tail=tail)
            assert torch.equal(dev, apart)
            dev, _ = C.on_device(t, pad, shift)
            loss2, st2 = torch.empty(9, **f), torch.empty(9, 4, **f)
            F.distill_topk_loss_grad(dev, tid, tv, g, loss2, st2, apart, tail=tail)
            F.distill_topk_loss_grad(dev, tid, tv, g, loss, st, dev, tail=tail)
            assert torch.equal(dev, apart) and torch.equal(loss, loss2) and torch.equal(st, st2)


@pytest.mark.parametrize("dtype,rows,vocab", [("fp32", 3, 50021), ("bf16", 5, 131077),
                                              ("fp16", 2, 262144), ("bf16", 520, 70001)])
def test_gradients_in_place_of_long_rows(dtype, rows, vocab):
    """Rows that take two passes: in place, the second must not need what it has overwritten."""
    rng = _seed(rows, vocab, 31)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    f = dict(dtype=torch.float32, device="cuda")
    g = np.linspace(0.5, 1.5, rows).astype(np.float32)
    for tail in (False, True):
        tid, tv = C.teacher_lists(rng, x64, 60, tail)
        dev, whole = C.on_device(t, 3, 1)
        before = whole.clone()
        loss, st = torch.empty(rows, **f), torch.empty(rows, 4, **f)
        say(f"in place, long rows {dtype} {rows} x {vocab} tail={tail}")
        F.distill_topk_loss_grad(dev, torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda(),
                                 torch.from_numpy(g).cuda(), loss, st, dev, tail=tail)
        some = list(range(min(rows, 6)))
        C.check_distill(x64[some], tid[some], tv[some], 1.0, tail, loss.cpu().numpy()[some],
                        st.cpu().numpy()[some], "in place")
        C.check_distill_grad(x64[some], tid[some], tv[some], g[some], 1.0, tail, dtype,
                             dev[some].double().cpu().numpy(), "in place")
        between = torch.ones_like(whole, dtype=torch.bool)
        between[1:1 + rows * (vocab + 3)].view(rows, vocab + 3)[:, :vocab] = False
        assert torch.equal(whole[between].view(torch.uint8), before[between].view(torch.uint8))


def _distill_all(dev, t, x64, tid, tv, g, scale, tail, dtype, what, opad=0, oshift=0):
    """Forward, backward and the joint call, each against the oracle."""
    rows = t.shape[0]
    f = dict(dtype=torch.float32, device="cuda")
    ids, values, gd = tid.cuda(), tv.cuda(), torch.from_numpy(g).cuda()
    for joint in (False, True):
        say(f"{what} {'joint' if joint else 'apart'}")
        loss, stats = torch.full((rows,), 55.0, **f), torch.full((rows, 4), 55.0, **f)
        out, whole = C.filled_like(t, opad, oshift)
        if joint:
            F.distill_topk_loss_grad(dev, ids, values, gd, loss, stats, out, tail=tail,
                                     scale=scale)
        else:
            F.distill_topk(dev, ids, values, loss, stats, tail=tail, scale=scale)
            F.distill_topk_grad(dev, ids, values, stats, gd, out, tail=tail, scale=scale)
        C.check_distill(x64, tid.numpy(), tv.numpy(), scale, tail, loss.cpu().numpy(),
                        stats.cpu().numpy(), what)
        C.check_distill_grad(x64, tid.numpy(), tv.numpy(), g, scale, tail, dtype,
                             out.double().cpu().numpy(), what + (" joint" if joint else ""))
        C.assert_between_rows_untouched(out, whole, what)
    only = torch.full((rows,), 55.0, **f)
    F.distill_topk(dev, ids, values, only, tail=tail, scale=scale)       # without the statistics
    C.check_distill(x64, tid.numpy(), tv.numpy(), scale, tail, only.cpu().numpy(), None, what)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_distill_shapes(shape, dtype, tail):
    rows, vocab, pad, shift = shape
    rng = _seed(rows, vocab, pad, len(dtype), 4 + tail)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    dev, _ = C.on_device(t, pad, shift)
    for k in (1, 16, 128):
        tid, tv = C.teacher_lists(rng, x64, k, tail)
        g = rng.standard_normal(rows).astype(np.float32)
        g[rng.random(rows) < 0.15] = 0
        _distill_all(dev, t, x64, torch.from_numpy(tid), torch.from_numpy(tv), g,
                     float(np.float32(0.6)), tail, dtype, f"distill {shape} {dtype} k={k} {tail}",
                     opad=(k + pad) % 3, oshift=k % 2)


# Long rows at both sides of the size up to which the joint call's gradient joins a row's parts (32
# MiB), and rows that the loss by itself gives to one work-group each.
@pytest.mark.parametrize("dtype,rows", [("fp32", 119), ("fp32", 121), ("bf16", 241)])
def test_distill_few_long_rows(dtype, rows):
    vocab = 70001
    rng = _seed(rows, vocab, len(dtype))
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    dev, _ = C.on_device(t)
    tid, tv = C.teacher_lists(rng, x64, 16, True)
    g = rng.standard_normal(rows).astype(np.float32)
    _distill_all(dev, t, x64, torch.from_numpy(tid), torch.from_numpy(tv), g, 1.0, True, dtype,
                 f"distill {rows} x {vocab} {dtype}")


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 9001])
def test_distill_special_rows(vocab, dtype, tail):
    rng = _seed(vocab, len(dtype), 7 + tail)
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    dev, _ = C.on_device(t)
    for k in (3, 40):
        tid, tv = C.teacher_lists(rng, x64, k, tail)
        tid[12, 0] = vocab // 3
        tid[9, 1], tid[10, 0] = vocab, 2 ** 31 - 1      # past the vocabulary
        tid[11, 0], tv[11, 0] = 1, np.nan
        tid[8, 0], tv[8, 0] = 1, np.inf
        tv[14] = -np.inf                                  # places, but no mass on them
        g = np.ones(16, np.float32)
        g[1] = 0
        _distill_all(dev, t, x64, torch.from_numpy(tid), torch.from_numpy(tv), g, 1.0, tail,
                     dtype, f"distill special {vocab} {dtype} k={k} {tail}")


@pytest.mark.parametrize("vocab", [700, 40001, 150001])
def test_logits_far_from_zero(vocab):
    """|scale x| beyond 2^20 with neighbours that still share the mass: the difference to the
    maximum has to be taken before anything is rounded."""
    rng = _seed(vocab, 41)
    scale, rows = 300.0, 3
    x = 1e4 + 0.02 * rng.standard_normal((rows, vocab))
    x[1] = -1e4 + 0.02 * rng.standard_normal(vocab)
    x[2] = 3.0 * rng.standard_normal(vocab)                    # an ordinary row beside them
    t, x64 = C.to_dtype(x, "fp32")
    dev, _ = C.on_device(t, 1, 1)
    ids = rng.integers(0, vocab, rows)
    got = C.run_logprobs(dev, ids, scale, 20)
    C.check_logprobs(x64, ids, scale, 20, C.host(got), f"far {vocab}")
    g, h = np.ones(rows, np.float32), np.full(rows, 0.3, np.float32)
    out, _ = C.filled_like(t)
    F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), got["stats"], out, scale=scale,
                          dlogprob=torch.from_numpy(g).cuda(), entropy=got["entropy"],
                          dentropy=torch.from_numpy(h).cuda())
    C.check_logprobs_grad(x64, ids, g, h, scale, "fp32", out.double().cpu().numpy(), "far")
    for tail in (False, True):
        tid, tv = C.teacher_lists(rng, x64, 30, tail)
        tv = np.where(np.isfinite(tv), tv / (1 if tail else scale), tv).astype(np.float32)
        _distill_all(dev, t, x64, torch.from_numpy(tid), torch.from_numpy(tv), g, scale, tail,
                     "fp32", f"far {vocab} {tail}")


@pytest.mark.parametrize("scale", [3e38, 1e-30])
def test_extreme_scales(scale):
    """The largest scale leaves all mass on the maximum, the smallest spreads it evenly."""
    rng = _seed(43)
    x = rng.standard_normal((4, 5003)).astype(np.float32)
    dev = torch.from_numpy(x).cuda()
    best = torch.from_numpy(x.argmax(1)).cuda()
    got = C.run_logprobs(dev, best.cpu().numpy(), scale, 3)
    lp = 0.0 if scale > 1 else -np.log(5003)
    assert torch.allclose(got["logprob"].double(), torch.full((4,), lp, dtype=torch.float64,
                                                              device="cuda"), rtol=1e-4, atol=0)
    assert torch.allclose(got["entropy"].double(), torch.full((4,), -lp, dtype=torch.float64,
                                                              device="cuda"), rtol=1e-4, atol=0)
    assert torch.equal(got["top_ids"][:, 0].long(), best)


def test_distill_list_of_the_whole_vocabulary():
    """Nothing outside the list, every token in it (some twice)."""
    rng = _seed(11)
    t, x64 = C.to_dtype(C.plain_rows(rng, 4, 30), "fp32")
    dev, _ = C.on_device(t)
    tid = np.stack([np.concatenate([rng.permutation(30), rng.integers(0, 30, 10)])
                    for _ in range(4)]).astype(np.int32)
    w = rng.random((4, 40))
    tv = np.log(0.9 * w / w.sum(1, keepdims=True)).astype(np.float32)
    for tail in (False, True):
        _distill_all(dev, t, x64, torch.from_numpy(tid), torch.from_numpy(tv),
                     np.ones(4, np.float32), 1.0, tail, "fp32", f"whole vocabulary {tail}")


def test_teacher_lists_may_be_slices():
    rng = _seed(12)
    t, x64 = C.to_dtype(C.plain_rows(rng, 6, 3001), "bf16")
    dev, _ = C.on_device(t)
    tid, tv = C.teacher_lists(rng, x64, 50, False)
    wide_i, wide_v = torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda()
    loss = torch.empty(6, device="cuda")
    F.distill_topk(dev, wide_i[:, 5:25], wide_v[:, 5:25], loss)
    C.check_distill(x64, tid[:, 5:25], tv[:, 5:25], 1.0, False, loss.cpu().numpy(), None, "slice")


def test_results_repeat_bit_for_bit():
    rng = _seed(13)
    for rows, vocab in ((3, 131072), (600, 5000)):
        t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), "bf16")
        dev, _ = C.on_device(t)
        ids = C.tokens(rng, rows, vocab)
        tid, tv = (torch.from_numpy(a).cuda() for a in C.teacher_lists(rng, x64, 32, True))
        f = dict(dtype=torch.float32, device="cuda")
        g = torch.ones(rows, **f)

        def once():
            a = C.run_logprobs(dev, ids, 1.0, 40)
            a["loss"], a["st"] = torch.empty(rows, **f), torch.empty(rows, 4, **f)
            a["grad"] = torch.empty_like(dev)
            F.distill_topk_loss_grad(dev, tid, tv, g, a["loss"], a["st"], a["grad"], tail=True)
            return {n: v.view(torch.int16) if v.dtype == torch.bfloat16 else v.view(torch.int32)
                    for n, v in a.items()}

        first = once()
        for _ in range(3):
            again = once()
            for n in first:
                assert torch.equal(first[n], again[n]), n


def test_rows_beyond_2_to_31_elements():
    """Two rows more than 2^31 elements apart: 64-bit offsets of logits and gradient."""
    vocab, stride = 1201, (1 << 31) + 4096
    rng = _seed(14)
    t, x64 = C.to_dtype(C.plain_rows(rng, 2, vocab), "bf16")
    buf = torch.empty(stride + vocab, dtype=torch.bfloat16, device="cuda")
    dev = buf.as_strided((2, vocab), (stride, 1))
    dev.copy_(t)
    out = torch.empty(stride + vocab, dtype=torch.bfloat16, device="cuda").as_strided(
        (2, vocab), (stride, 1))
    ids = np.array([5, 1200])
    got = C.run_logprobs(dev, ids, 1.0, 9)
    C.check_logprobs(x64, ids, 1.0, 9, C.host(got), "far rows")
    one = np.ones(2, np.float32)
    F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), got["stats"], out,
                          dlogprob=torch.from_numpy(one).cuda())
    C.check_logprobs_grad(x64, ids, one, 0 * one, 1.0, "bf16", out.double().cpu().numpy(), "far")
    for tail in (False, True):
        tid, tv = C.teacher_lists(rng, x64, 8, tail)
        out.fill_(77.0)
        loss, st = torch.empty(2, device="cuda"), torch.empty(2, 4, device="cuda")
        F.distill_topk_loss_grad(dev, torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda(),
                                 torch.ones(2, device="cuda"), loss, st, out, tail=tail)
        C.check_distill(x64, tid, tv, 1.0, tail, loss.cpu().numpy(), st.cpu().numpy(), "far")
        C.check_distill_grad(x64, tid, tv, one, 1.0, tail, "bf16", out.double().cpu().numpy(),
                             "far")


def test_many_rows():
    """More rows than a launch has work-groups for one row each on the device at once."""
    rng = _seed(15)
    rows, vocab = 70001, 24
    x = C.plain_rows(rng, rows, vocab).astype(np.float32)
    t = torch.from_numpy(x)
    dev = t.cuda()
    ids = rng.integers(0, vocab, rows)
    got = C.host(C.run_logprobs(dev, ids, 1.0, 3))
    x64 = x.astype(np.float64)
    lp = x64 - x64.max(1, keepdims=True)
    lp -= np.log(np.exp(lp).sum(1, keepdims=True))
    assert np.abs(got["logprob"] - lp[np.arange(rows), ids]).max() < 1e-4
    want = np.argsort(-x64, 1, kind="stable")[:, :3]
    assert (got["top_ids"] == want).all()


def test_more_rows_than_one_launch_takes():
    """Rows beyond 2^20 go to further launches of the same kernels."""
    rows, vocab, k = (1 << 20) + 301, 5, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, vocab, generator=gen, device="cuda") * 2
    ids = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    lp, st = torch.full((rows,), 55.0, **f), torch.full((rows, 2), 55.0, **f)
    ti = torch.full((rows, k), 55, dtype=torch.int32, device="cuda")
    tl = torch.full((rows, k), 55.0, **f)
    F.token_logprobs(x, ids, logprob=lp, stats=st, top_ids=ti, top_logprobs=tl)
    want = torch.log_softmax(x.double(), 1)
    best = want.topk(k, 1)
    assert torch.equal(ti.long(), best.indices)
    # unit(5) is 1.6e-5; |d| and |log p| are below 25 here
    assert (lp - want.gather(1, ids[:, None])[:, 0]).abs().max() < 1e-3
    assert (tl - best.values).abs().max() < 1e-3
    g = torch.ones(rows, **f)
    d = torch.full_like(x, 55.0)
    F.token_logprobs_grad(x, ids, st, d, dlogprob=g)
    hot = torch.nn.functional.one_hot(ids, vocab)
    assert (d - (hot - want.exp())).abs().max() < 1e-3
    loss, ds = torch.full((rows,), 55.0, **f), torch.full((rows, 4), 55.0, **f)
    F.distill_topk_loss_grad(x, ti, tl, g, loss, ds, d)
    q = torch.softmax(tl.double(), 1)
    exact = (q * (q.log() - want.gather(1, ti.long()))).sum(1)
    assert (loss - exact).abs().max() < 1e-3
    assert (d - (want.exp() - torch.zeros_like(want).scatter(1, ti.long(), q))).abs().max() < 1e-3


def test_no_rows():
    x = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, device="cuda")
    F.token_logprobs(x, entropy=e)
    F.distill_topk(x, torch.empty(0, 4, dtype=torch.int32, device="cuda"),
                   torch.empty(0, 4, device="cuda"), e)
    F.token_logprobs_grad(x, None, torch.empty(0, 2, device="cuda"), torch.empty_like(x),
                          entropy=e, dentropy=e)
    torch.cuda.synchronize()


def test_binding_refusals_on_the_gpu():
    x = torch.zeros(4, 64, device="cuda")
    e = torch.empty(4, device="cuda")
    bad = [dict(logits=x.double(), entropy=e), dict(logits=x[0], entropy=e),
           dict(logits=x.t(), entropy=e), dict(logits=x, entropy=e[:3]),
           dict(logits=x, entropy=e.double()), dict(logits=x, logprob=e),
           dict(logits=x, ids=torch.zeros(4, dtype=torch.int32, device="cuda"), logprob=e),
           dict(logits=x, top_ids=torch.zeros(4, 2, dtype=torch.int32, device="cuda")),
           dict(logits=x, entropy=e.cpu()), dict(logits=x, stats=e)]
    for kw in bad:
        with pytest.raises(ValueError):
            F.token_logprobs(**kw)
    with pytest.raises(F.FsdpShardError):
        F.token_logprobs(x, entropy=e, scale=0.0)
    with pytest.raises(F.FsdpShardError):
        F.token_logprobs(x, entropy=x.view(-1)[:4])
    i, v = torch.zeros(4, 3, dtype=torch.int32, device="cuda"), torch.zeros(4, 3, device="cuda")
    for kw in (dict(teacher_ids=i.long(), teacher_values=v), dict(teacher_ids=i[:2],
               teacher_values=v), dict(teacher_ids=i, teacher_values=v[:, :2]),
               dict(teacher_ids=i, teacher_values=v.half())):
        with pytest.raises(ValueError):
            F.distill_topk(x, loss=e, **kw)
    with pytest.raises(ValueError):
        F.distill_topk_grad(x, i, v, torch.zeros(4, 4, device="cuda"), e, x.bfloat16())


def test_side_stream_with_its_own_workspace():
    rng = _seed(16)
    t, x64 = C.to_dtype(C.plain_rows(rng, 3, 100003), "bf16")
    dev, _ = C.on_device(t)
    ids = C.tokens(rng, 3, 100003)
    side = torch.cuda.Stream()
    idt = torch.as_tensor(ids).cuda()
    f = dict(dtype=torch.float32, device="cuda")
    out = dict(logprob=torch.empty(3, **f), top_ids=torch.empty(3, 20, dtype=torch.int32,
                                                                device="cuda"),
               top_logprobs=torch.empty(3, 20, **f))
    loss = torch.empty(3, **f)
    tid, tv = C.teacher_lists(rng, x64, 20, True)
    tid_d, tv_d = torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda()
    torch.cuda.synchronize()
    F.token_logprobs(dev, idt, stream=side, **out)
    F.distill_topk(dev, tid_d, tv_d, loss, tail=True, stream=side)
    junk = [torch.full((1 << 14,), float("nan"), device="cuda") for _ in range(64)]
    del junk
    side.synchronize()
    C.check_logprobs(x64, ids, 1.0, 20, C.host(out), "side stream")
    C.check_distill(x64, tid, tv, 1.0, True, loss.cpu().numpy(), None, "side stream")


@pytest.mark.parametrize("rows,vocab", [(2, 131072), (64, 4099)])
def test_graph_replays_match_eager(rows, vocab):
    rng = _seed(17, rows)
    f = dict(dtype=torch.float32, device="cuda")
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), "bf16")
    dev, _ = C.on_device(t)
    ids = torch.as_tensor(C.tokens(rng, rows, vocab)).cuda()
    tid, tv = (torch.from_numpy(a).cuda() for a in C.teacher_lists(rng, x64, 24, True))
    g, h = torch.ones(rows, **f), torch.full((rows,), -0.5, **f)

    def buffers():
        return dict(lp=torch.zeros(rows, **f), H=torch.zeros(rows, **f),
                    st=torch.zeros(rows, 2, **f),
                    ti=torch.zeros(rows, 24, dtype=torch.int32, device="cuda"),
                    tl=torch.zeros(rows, 24, **f), d1=torch.zeros_like(dev),
                    loss=torch.zeros(rows, **f), ds=torch.zeros(rows, 4, **f),
                    d2=torch.zeros_like(dev))

    def calls(b):
        F.token_logprobs(dev, ids, logprob=b["lp"], entropy=b["H"], stats=b["st"],
                         top_ids=b["ti"], top_logprobs=b["tl"])
        F.token_logprobs_grad(dev, ids, b["st"], b["d1"], dlogprob=g, entropy=b["H"], dentropy=h)
        F.distill_topk_loss_grad(dev, tid, tv, g, b["loss"], b["ds"], b["d2"], tail=True)

    eager, graphed, warm = buffers(), buffers(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls(warm)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls(graphed)
    for rep in range(4):
        # new logits in the captured buffer, unrelated eager work, then both
        dev.copy_(C.to_dtype(C.plain_rows(rng, rows, vocab), "bf16")[0])
        calls(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        torch.randn(1 << 20, device="cuda").sum()
        torch.cuda.synchronize()
        for n in eager:
            a, b = eager[n].cpu(), graphed[n].cpu()
            assert torch.equal(a, b), f"replay {rep}: {n}"
        say(f"  replay {rep} equals the eager calls")


def test_distillation_step_from_teacher_to_weights():
    """The operators in the order of use: a teacher's pass gives the lists, the student's step
    gives loss and gradient, the head's weight gradient of two micro-batches goes through the
    sharded update.  Every stage is checked against the oracle on the inputs it was given."""
    import workloads as W
    from oracle import step as OS
    rng = _seed(18)
    T, D, V, K, n = 48, 32, 1003, 16, 32 * 1003
    f = dict(dtype=torch.float32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(5)
    head = torch.randn(V, D, generator=gen, **f)
    teacher_head = head + 0.3 * torch.randn(V, D, generator=gen, **f)
    contribs = []
    for micro in range(2):
        hidden = torch.randn(T, D, generator=gen, **f)
        teacher = (hidden @ teacher_head.t()).bfloat16()
        student = (hidden @ head.t()).bfloat16()
        ti = torch.empty(T, K, dtype=torch.int32, device="cuda")
        tl = torch.empty(T, K, **f)
        F.token_logprobs(teacher, top_ids=ti, top_logprobs=tl)
        C.check_logprobs(teacher.double().cpu().numpy(), np.full(T, -1), 1.0, K,
                         C.host(dict(top_ids=ti, top_logprobs=tl)), "teacher")
        ti[:5] = -1                                   # prompt positions
        loss, st = torch.empty(T, **f), torch.empty(T, 4, **f)
        weight = torch.full((T,), 1.0 / T, **f)
        before = student.double().cpu().numpy()
        F.distill_topk_loss_grad(student, ti, tl, weight, loss, st, student, tail=True)
        C.check_distill(before, ti.cpu().numpy(), tl.cpu().numpy(), 1.0, True, loss.cpu().numpy(),
                        st.cpu().numpy(), "student")
        C.check_distill_grad(before, ti.cpu().numpy(), tl.cpu().numpy(),
                             weight.cpu().numpy(), 1.0, True, "bf16",
                             student.double().cpu().numpy(), "student")
        assert (student[:5] == 0).all() and (loss[:5] == 0).all()
        contribs.append((student.float().t() @ hidden).bfloat16().reshape(-1).contiguous())
    master, m, v = head.reshape(-1).clone(), torch.zeros(n, **f), torch.zeros(n, **f)
    flat = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    hp = dict(W.ADAMW)
    F.adamw_shard_step(master, m, v, contribs, step=1, flat=flat, **hp)
    want = OS.shard_step(head.reshape(-1).cpu().numpy(), np.zeros(n, np.float32),
                         np.zeros(n, np.float32),
                         [c.view(torch.int16).cpu().numpy().view(np.uint16) for c in contribs],
                         np.full(n, 1), hp, 1)
    assert np.array_equal(master.cpu().numpy(), want[0])
    assert np.array_equal(flat.view(torch.int16).cpu().numpy().view(np.uint16), want[3])


def test_policy_gradient_from_logits_to_logits():
    """Scoring, a clipped-ratio objective in torch, and the gradient of the logits, against the
    same in float64 on the CPU.  dlogprob is computed once, on the GPU, and given to both."""
    rng = _seed(19)
    t, x64 = C.to_dtype(C.plain_rows(rng, 40, 2999), "bf16")
    dev, _ = C.on_device(t)
    ids = C.tokens(rng, 40, 2999)
    out = C.run_logprobs(dev, ids, 1.0, 0)
    old = out["logprob"] + 0.1 * torch.randn(40, device="cuda")
    lp = out["logprob"].clone().requires_grad_()
    adv = torch.randn(40, device="cuda")
    ratio = (lp - old).exp()
    torch.min(ratio * adv, ratio.clamp(0.8, 1.2) * adv).mean().neg().backward()
    dent = torch.full((40,), -0.01 / 40, device="cuda")
    grad, _ = C.filled_like(t)
    F.token_logprobs_grad(dev, torch.as_tensor(ids).cuda(), out["stats"], grad, dlogprob=lp.grad,
                          entropy=out["entropy"], dentropy=dent)
    C.check_logprobs_grad(x64, ids, lp.grad.cpu().numpy(), dent.cpu().numpy(), 1.0, "bf16",
                          grad.double().cpu().numpy(), "policy")
