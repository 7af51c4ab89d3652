"""The kernels that matrices of logits of real sizes take, by value against the float64 oracle: rows of
odd vocabularies in every type, as many as the CUs and more, below and beyond 128 MiB (where rows are
loaded without keeping them in a cache), in one work-group a row and in parts, and the largest
vocabulary.

A sample of rows goes to the oracle, with the error bounds of logits_cases: one row of each kind of
special_rows, spread over the matrix, and 8 ordinary ones between them.  All rows are checked for
having been written, and what lies between them for not having been."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# (dtype, rows, vocab, pad between rows, shift of the base).  Vectors a row decide the joint call's
# kernel: up to 4096 one work-group of 256 threads, up to 8192 one of 512, beyond that two passes.
MATRICES = [
    # few rows: a row has a CU to itself up to 256 of them; the loss alone holds rows in registers up
    # to 128 rows beyond 81,920 elements of 16 bits
    ("bf16", 256, 32003, 0, 1), ("fp16", 257, 32003, 0, 1), ("bf16", 128, 90001, 1, 0),
    ("fp16", 129, 90001, 0, 1), ("fp32", 128, 50021, 0, 1), ("fp32", 400, 16001, 0, 1),
    ("bf16", 300, 100003, 0, 0),
    # more
    ("bf16", 600, 5003, 0, 1), ("fp16", 600, 31999, 1, 0), ("fp32", 600, 16001, 3, 1),
    ("bf16", 530, 50021, 0, 3), ("fp32", 530, 32003, 0, 1),
    ("fp16", 520, 100003, 5, 0),                                  # two passes, whole rows
    # 128 MiB and more
    ("bf16", 2100, 32003, 0, 1), ("fp16", 2100, 32000, 0, 0), ("fp32", 2200, 16001, 0, 1),
    ("fp16", 1400, 50021, 0, 0), ("fp32", 1100, 32003, 5, 0),
    ("bf16", 530, 131071, 0, 1),                                  # two passes, whole rows
    ("bf16", 600, 140001, 0, 1), ("fp32", 600, 70001, 0, 0),      # parts
    ("fp16", 1000, 140001, 0, 1),                                 # beyond 256 MiB
]


def _matrix(dtype, rows, vocab, pad, shift):
    """(logits on the GPU, sampled rows, their values as float64)."""
    rng = np.random.default_rng([rows, vocab, len(dtype)])
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + vocab)
    stride = vocab + pad
    buf = torch.full((shift + rows * stride + 8,), float("nan"), dtype=C.DTYPES[dtype],
                     device="cuda")
    x = buf[shift:shift + rows * stride].view(rows, stride)[:, :vocab]
    for r in range(0, rows, 256):
        n = min(256, rows - r)
        x[r:r + n] = torch.randn(n, vocab, generator=gen, device="cuda") * 3
    odd, _ = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    spread = np.linspace(0, rows - 1, 24).round().astype(np.int64)
    special = spread[np.arange(16) * 3 // 2]
    x[torch.from_numpy(special).cuda()] = odd.cuda()
    return x, spread, x[torch.from_numpy(spread).cuda()].double().cpu().numpy(), special


def _gradient_like(x, pad, shift):
    rows, vocab = x.shape
    whole = torch.full((shift + rows * (vocab + pad) + 8,), 77.0, dtype=x.dtype, device="cuda")
    return whole[shift:shift + rows * (vocab + pad)].view(rows, -1)[:, :vocab], whole


def _check_written(out, whole, pad, shift, what):
    """Gradients here are below 77, so no element of the rows still holds it, and all others do."""
    rows, vocab = out.shape
    assert not (out == 77).any(), f"{what}: elements not written"
    end = shift + rows * (vocab + pad)
    assert (whole[:shift] == 77).all() and (whole[end:] == 77).all(), f"{what}: written outside"
    if pad:
        between = whole[shift:end].view(rows, vocab + pad)[:, vocab:]
        assert (between == 77).all(), f"{what}: written between the rows"


def _pick(t, rows):
    return t[torch.from_numpy(rows).to(t.device)]


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("dtype,rows,vocab,pad,shift", MATRICES)
def test_logprobs_of_large_matrices(dtype, rows, vocab, pad, shift):
    x, some, x64, special = _matrix(dtype, rows, vocab, pad, shift)
    rng = np.random.default_rng([rows, vocab, 1])
    ids = C.tokens(rng, rows, vocab)
    ids[special[[0, 9]]] = -1, vocab
    ids[special[3]], ids[special[12]] = vocab // 2, vocab // 3
    got = None
    for k in (0, 20, 128):
        what = f"logprobs {dtype} {rows} x {vocab} k={k}"
        say(what)
        got = C.run_logprobs(x, ids, 1.0, k)
        for name, t in got.items():
            assert name == "top_ids" or not (t == 55).any(), f"{what}: {name} not written"
        C.check_logprobs(x64, ids[some], 1.0, k, C.host({n: _pick(t, some)
                                                         for n, t in got.items()}), what)
    g, h = (rng.standard_normal(rows).astype(np.float32) for _ in range(2))
    g[rng.random(rows) < 0.2] = 0
    h[rng.random(rows) < 0.2] = 0
    idt, gd, hd = torch.as_tensor(ids).cuda(), torch.from_numpy(g).cuda(), torch.from_numpy(h).cuda()
    for hh in (None, hd):
        what = f"logprobs grad {dtype} {rows} x {vocab} h={hh is not None}"
        say(what)
        out, whole = _gradient_like(x, pad, shift)
        F.token_logprobs_grad(x, idt, got["stats"], out, dlogprob=gd, entropy=got["entropy"],
                              dentropy=hh)
        C.check_logprobs_grad(x64, ids[some], g[some], (0 * h if hh is None else h)[some], 1.0,
                              dtype, _np(_pick(out, some)), what)
        _check_written(out, whole, pad, shift, what)


def _lists(x, k, tail, special):
    """Half of each list the row's best tokens, half drawn (so that some stand in it twice); a tenth
    of the places empty, every ninth list, and what test_distill_special_rows gives its rows."""
    rows, vocab = x.shape
    gen = torch.Generator(device="cuda").manual_seed(k)
    ids = torch.randint(0, vocab, (rows, k), generator=gen, device="cuda")
    ids[:, :(k + 1) // 2] = x.topk((k + 1) // 2, 1).indices
    w = torch.rand(rows, k, generator=gen, device="cuda") ** 3 + 1e-6
    share = torch.rand(rows, 1, generator=gen, device="cuda") * 0.7 + 0.3 if tail else 1.0
    values = (w / w.sum(1, keepdim=True) * share).log()
    ids[torch.rand(rows, k, generator=gen, device="cuda") < 0.1] = -1
    ids[4::9] = -1
    sp = special.tolist()
    ids[sp[12], 0] = vocab // 3
    ids[sp[9], 1], ids[sp[10], 0] = vocab, 2 ** 31 - 1
    ids[sp[11], 0], values[sp[11], 0] = 1, float("nan")
    ids[sp[8], 0], values[sp[8], 0] = 1, float("inf")
    values[sp[14]] = -float("inf")
    return ids.int(), values


@pytest.mark.parametrize("k,tail", [(64, False), (100, True)])
@pytest.mark.parametrize("dtype,rows,vocab,pad,shift", MATRICES)
def test_distill_of_large_matrices(dtype, rows, vocab, pad, shift, k, tail):
    x, some, x64, special = _matrix(dtype, rows, vocab, pad, shift)
    rng = np.random.default_rng([rows, vocab, k])
    tid, tv = _lists(x, k, tail, special)
    g = rng.uniform(0.5, 1.5, rows).astype(np.float32)
    g[rng.random(rows) < 0.1] = 0
    gd = torch.from_numpy(g).cuda()
    si, sv = _pick(tid, some).cpu().numpy(), _pick(tv, some).cpu().numpy()
    f = dict(dtype=torch.float32, device="cuda")
    for form in ("apart", "joint", "joint, in place"):
        what = f"distill {dtype} {rows} x {vocab} k={k} tail={tail} {form}"
        say(what)
        loss, stats = torch.full((rows,), 55.0, **f), torch.full((rows, 4), 55.0, **f)
        if form == "joint, in place":
            out, whole = x, None
        else:
            out, whole = _gradient_like(x, pad, shift)
        if form == "apart":
            F.distill_topk(x, tid, tv, loss, stats, tail=tail)
            F.distill_topk_grad(x, tid, tv, stats, gd, out, tail=tail)
        else:
            F.distill_topk_loss_grad(x, tid, tv, gd, loss, stats, out, tail=tail)
        assert not (loss == 55).any() and not (stats == 55).any(), f"{what}: not written"
        C.check_distill(x64, si, sv, 1.0, tail, _np(_pick(loss, some)), _np(_pick(stats, some)),
                        what)
        C.check_distill_grad(x64, si, sv, g[some], 1.0, tail, dtype, _np(_pick(out, some)), what)
        if whole is not None:
            _check_written(out, whole, pad, shift, what)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_largest_vocabulary(dtype):
    """Hundreds of parts a row, each with its own list of alternatives: an ordinary row, one masked in
    large part, and one of many ties."""
    rows, vocab, k = 3, (1 << 21) - 3, 128
    rng = np.random.default_rng([vocab, len(dtype)])
    v = C.plain_rows(rng, rows, vocab)
    v[1, rng.random(vocab) < 0.7] = -np.inf
    v[2] = np.round(v[2])
    t, x64 = C.to_dtype(v, dtype)
    x, _ = C.on_device(t, 2, 1)
    ids = np.array([vocab - 1, int(np.argmax(x64[1])), 0])
    say(f"logprobs {dtype} {rows} x {vocab}")
    got = C.run_logprobs(x, ids, 1.0, k)
    C.check_logprobs(x64, ids, 1.0, k, C.host(got), f"largest vocabulary {dtype}")
    g, h = np.ones(rows, np.float32), np.full(rows, -0.5, np.float32)
    gd = torch.from_numpy(g).cuda()
    say("logprobs grad")
    out, whole = C.filled_like(t, 1, 3)
    F.token_logprobs_grad(x, torch.as_tensor(ids).cuda(), got["stats"], out, dlogprob=gd,
                          entropy=got["entropy"], dentropy=torch.from_numpy(h).cuda())
    C.check_logprobs_grad(x64, ids, g, h, 1.0, dtype, _np(out), f"largest vocabulary {dtype}")
    C.assert_between_rows_untouched(out, whole, dtype)
    tid, tv = C.teacher_lists(rng, x64, k, True)
    tid[0, :2] = vocab - 1, 0
    tid_d, tv_d = torch.from_numpy(tid).cuda(), torch.from_numpy(tv).cuda()
    for joint in (False, True):
        say(f"distill {'joint' if joint else 'apart'}")
        loss, stats = torch.full((rows,), 55.0).cuda(), torch.full((rows, 4), 55.0).cuda()
        out, whole = C.filled_like(t, 1, 3)
        if joint:
            F.distill_topk_loss_grad(x, tid_d, tv_d, gd, loss, stats, out, tail=True)
        else:
            F.distill_topk(x, tid_d, tv_d, loss, stats, tail=True)
            F.distill_topk_grad(x, tid_d, tv_d, stats, gd, out, tail=True)
        C.check_distill(x64, tid, tv, 1.0, True, _np(loss), _np(stats), dtype)
        C.check_distill_grad(x64, tid, tv, g, 1.0, True, dtype, _np(out), dtype)
        C.assert_between_rows_untouched(out, whole, dtype)


# Vectors a row, at both sides of five for each alternative: the number of threads changes there, and
# short rows have fewer maxima than alternatives.
@pytest.mark.parametrize("dtype,vocab,k", [("bf16", 5106, 128), ("bf16", 5098, 128),
                                           ("fp16", 2554, 64), ("bf16", 2546, 64),
                                           ("fp32", 2557, 128), ("fp32", 2553, 128),
                                           ("bf16", 801, 20), ("bf16", 769, 128),
                                           ("fp32", 900, 128)])
def test_lists_of_short_rows(dtype, vocab, k):
    rng = np.random.default_rng([vocab, k])
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    ids = np.where(np.arange(16) % 3 == 0, -1, np.arange(16) % vocab)
    for pad, shift in ((0, 0), (3, 1)):
        x, _ = C.on_device(t, pad, shift)
        say(f"lists of short rows {dtype} {vocab} k={k} shift={shift}")
        got = C.run_logprobs(x, ids, 1.0, k)
        C.check_logprobs(x64, ids, 1.0, k, C.host(got), f"{dtype} {vocab} k={k} shift={shift}")
