"""The policy loss over logits of rows too long for a work-group's registers, in matrices of many rows
and in place, against the oracles within the bounds of test_gpu_policy_logits; which side of a limit a
token falls on, whatever way its row takes; and rows that do not count."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say
from oracle import policy as OP
from test_gpu_policy_logits import TERMS, call, check, inputs

pytestmark = pytest.mark.gpu


def _rng(*key):
    return np.random.default_rng([int(v) for v in key] + [41])


# dtype, rows, vocab, in place; the first ones fit the registers or join their parts
FORMS = [("bf16", 3, 30001, False), ("bf16", 300, 30001, True), ("bf16", 3, 70001, False),
         ("bf16", 3, 70001, True), ("bf16", 300, 70001, False), ("fp32", 4, 40001, False),
         ("fp32", 4, 40001, True), ("fp32", 260, 40001, False), ("fp16", 2, 500001, True),
         ("fp16", 270, 140001, False)]


@pytest.mark.parametrize("dtype,rows,vocab,in_place", FORMS)
@pytest.mark.parametrize("above", [False, True])
def test_the_side_of_a_limit_is_decided_in_64_bits(dtype, rows, vocab, in_place, above):
    """Rows of equal logits have the log probability -log(vocab), from a sum that float32 holds
    exactly.  The limit lies halfway between it and its rounding to float32."""
    lp = -np.log(np.float64(vocab))
    old = np.float32(lp - (0.1 if above else -0.1))
    exact, rounded = lp - np.float64(old), np.float64(np.float32(lp)) - np.float64(old)
    assert 2e-8 < abs(exact - rounded) < 1e-6
    limit = (exact + rounded) / 2
    c = OP.constants(clip_high=float(np.expm1(limit))) if above else \
        OP.constants(clip_low=float(-np.expm1(limit)))
    cut = exact > np.log1p(c["clip_high"]) if above else exact < np.log1p(-c["clip_low"])
    f = dict(dtype=torch.float32, device="cuda")
    x = torch.zeros(rows, vocab, dtype=C.DTYPES[dtype], device="cuda")
    out = x if in_place else torch.full_like(x, 7)
    ids = torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(1)).cuda()
    loss, sign = torch.empty(rows, **f), 1.0 if above else -1.0
    say(f"{dtype} {rows} x {vocab} in place {in_place}, clipped {cut}")
    F.policy_logits_loss_grad(x, ids, torch.full((rows,), sign, **f), torch.ones(rows, **f), loss,
                              out, old_logprob=torch.full((rows,), float(old), **f), **c)
    at = out.gather(1, ids[:, None])[:, 0].float()
    if cut:
        assert (out == 0).all()
    else:
        assert (at * -sign > 0).all() and int((out != 0).all(1).sum()) == rows


@pytest.mark.parametrize("dtype,rows,vocab,pad,shift", [("bf16", 258, 70001, 1, 3),
                                                        ("fp16", 257, 66000, 0, 0),
                                                        ("fp32", 257, 33000, 3, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_rows(dtype, rows, vocab, pad, shift, in_place):
    rng = _rng(rows, vocab, in_place)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), dtype)
    ids = C.tokens(rng, rows, vocab)
    best = rng.random(rows) < 0.4
    ids[best] = np.argmax(x64[best], 1)
    ids[7], ids[8] = vocab, vocab                        # past the vocabulary; one of no weight
    scale = float(np.float32(0.8))
    c = TERMS[2] if in_place else TERMS[1]
    v = inputs(rng, x64, ids, scale, c)
    v["w"][7], v["w"][8] = 0.5, 0
    dev, whole = C.on_device(t, pad, shift)
    say(f"{dtype} {rows} x {vocab} in place {in_place}")
    if in_place:
        got = call(dev, ids, v, c, scale, dev)
        out = dev
    else:
        out, whole = C.filled_like(t, pad + 1, shift)
        got = call(dev, ids, v, c, scale, out, entropy=False)
        C.assert_between_rows_untouched(out, whole, dtype)
    check(x64, ids, v, c, scale, dtype, got, out, f"{dtype} {rows} x {vocab}")
    assert (out[8] == 0).all() and got["loss"][8] == 0 and got["logprob"][8] == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("vocab", [70001, 140003])
def test_special_rows_in_place(dtype, vocab):
    rng = _rng(vocab, len(dtype), 5)
    t, x64 = C.to_dtype(C.special_rows(rng, vocab, dtype), dtype)
    ids = rng.integers(0, vocab, 16)
    ids[[0, 9]] = -1, vocab
    ids[12], ids[3] = vocab // 3, vocab // 2
    ids[1] = int(np.argmax(x64[1]))
    ids[15] = vocab - 1
    for i, c in enumerate(TERMS):
        say(f"special rows in place vocab={vocab} {dtype} terms {i}")
        v = inputs(rng, x64, ids, 1.0, c)
        v["w"][:] = 0.5
        v["w"][10] = 0
        dev, _ = C.on_device(t, 0, 1)
        got = call(dev, ids, v, c, 1.0, dev)
        check(x64, ids, v, c, 1.0, dtype, got, dev, f"special {vocab} {dtype} terms {i}")
        assert (dev[2] == 0).all() and (dev[0] == 0).all() and (dev[10] == 0).all()
        assert dev[[6, 7, 9]].isnan().all()


@pytest.mark.parametrize("rows,vocab,in_place", [(8, 70001, True), (300, 70001, False)])
def test_rows_that_do_not_count_may_hold_anything(rows, vocab, in_place):
    rng = _rng(rows, vocab, 6)
    t, x64 = C.to_dtype(C.plain_rows(rng, rows, vocab), "bf16")
    ids = rng.integers(0, vocab, rows)
    c = TERMS[2]
    v = inputs(rng, x64, ids, 1.0, c)
    v["w"][:] = 0.5
    none = [2, 5, rows - 1]
    ids[2], v["w"][5], v["w"][rows - 1] = -1, 0, 0
    clean, _ = C.on_device(t)
    want_out, _ = C.filled_like(t)
    want = call(clean, ids, v, c, 1.0, clean if in_place else want_out)
    if in_place:
        want_out = clean
    dev, _ = C.on_device(t)
    dev[none] = float("nan")
    for k in ("old", "ref", "A"):
        v[k][none] = np.nan
    out = dev if in_place else C.filled_like(t)[0]
    got = call(dev, ids, v, c, 1.0, out)
    assert (out[none] == 0).all() and torch.equal(out, want_out)
    for name in got:
        assert (got[name][none] == 0).all() and np.array_equal(got[name], want[name]), name


def test_captured_and_repeated():
    """Every replay, with eager work between, gives the eager call's bits."""
    rows, vocab = 300, 70001
    g = torch.Generator(device="cuda").manual_seed(3)
    f = dict(generator=g, device="cuda")
    x = torch.randn(rows, vocab, **f).bfloat16()
    ids = torch.randint(0, vocab, (rows,), **f)
    A, old = torch.randn(rows, **f), torch.randn(rows, **f) - 11
    w = (torch.rand(rows, **f) > 0.3).float()
    out, loss = torch.empty_like(x), torch.empty(rows, device="cuda")
    ws = torch.empty(F.policy_logits_loss_grad_workspace_bytes(rows, vocab), dtype=torch.uint8,
                     device="cuda")

    def run():
        F.policy_logits_loss_grad(x, ids, A, w, loss, out, old_logprob=old, workspace=ws)

    ws.fill_(255)
    run()
    torch.cuda.synchronize()
    want = out.clone(), loss.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for rep in range(3):
        out.fill_(3)
        loss.fill_(3)
        ws.fill_(rep)
        torch.cuda.synchronize()
        say(f"replay {rep}")
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16))
        assert torch.equal(loss, want[1])


def test_long_rows_beyond_2_31_elements():
    rows, vocab = 16500, 131072
    x = torch.zeros(rows, vocab, dtype=torch.bfloat16, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    ids = torch.full((rows,), 5, device="cuda")
    loss = torch.empty(rows, **f)
    say("long rows beyond 2^31 elements, in place")
    F.policy_logits_loss_grad(x, ids, torch.ones(rows, **f), torch.ones(rows, **f), loss, x)
    assert (loss == -1).all()                            # ratio 1, advantage 1
    last = x[rows - 1].float()
    assert float(last[5]) == -1.0 and float(last[vocab - 1]) == 2.0 ** -17
