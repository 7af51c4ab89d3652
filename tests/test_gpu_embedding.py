"""Embedding lookup and its gradient on the GPU.  The lookup is one float32 product and one rounding,
so it is compared bit for bit.  The gradient's bound: with u = 2^-24 a row's float32 sums are chains of
at most 2 chunk additions of terms of total size S (a chunk is at most max(32, tokens / 2048) tokens, rounded up
to 8, and a run's sum goes on into the next one), their float64 sum is rounded once, and the product with
the scale, the sum with what was there and the rounding to the type come last: u S (2 chunk + 1) + u |d| +
u |result| + half a step of the type."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say
from oracle import embedding as OE

pytestmark = pytest.mark.gpu
T = C.DTYPES
U = 2.0 ** -24


def _seed(*key):
    return np.random.default_rng([int(v) for v in key] + [29])


def _ids(rng, tokens, vocab, skew=2.0, outside=True):
    """Tokens of which some are frequent; some positions without a token, some past the table."""
    ids = (vocab * rng.random(tokens) ** skew).astype(np.int64)
    if outside:
        ids[rng.random(tokens) < 0.15] = -100
        if tokens > 4:
            ids[tokens // 2] = vocab
            ids[tokens // 3] = 1 << 40
    return ids


# tokens, vocab, dim, pad between rows, shift of the base
SHAPES = [(1, 1, 1, 0, 0), (1, 5, 7, 0, 1), (3, 2, 8, 1, 0), (33, 100, 9, 0, 3), (17, 50, 64, 8, 0),
          (200, 37, 250, 5, 1), (65, 129, 1000, 0, 0), (9, 300, 2048, 0, 5), (130, 64, 4096, 0, 0),
          (5, 40, 4100, 3, 2), (4, 30, 12345, 0, 0)]


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_lookup(shape, dtype, out):
    tokens, vocab, dim, pad, shift = shape
    rng = _seed(*shape)
    t, _ = C.to_dtype(rng.standard_normal((vocab, dim)), dtype)
    dev, _ = C.on_device(t, pad, shift)
    ids = _ids(rng, tokens, vocab)
    like = torch.zeros(tokens, dim, dtype=T[out])
    for scale in (1.0, 64.0, -0.3):
        say(f"lookup {shape} {dtype} -> {out} scale={scale}")
        got, whole = C.filled_like(like, (pad + 1) % 7, shift // 2)
        F.embedding_lookup(dev, torch.from_numpy(ids).cuda(), got, scale=scale)
        rows = t[torch.from_numpy(np.clip(ids, 0, vocab - 1))].float() * np.float32(scale)
        rows[torch.from_numpy(ids < 0)] = 0
        rows[torch.from_numpy(ids >= vocab)] = float("nan")
        want = rows.to(T[out])
        assert torch.equal(torch.nan_to_num(got.cpu().float(), nan=-7e4),
                           torch.nan_to_num(want.float(), nan=-7e4))
        C.assert_between_rows_untouched(got, whole, f"{shape}")


def test_lookup_special_values():
    x = torch.tensor([[float("inf"), -float("inf"), float("nan"), -0.0, 1e-40, 3e38, 65504.0, 1.0]])
    for dtype in T.values():
        table = x.to(dtype).cuda()
        out = torch.empty(2, 8, dtype=dtype, device="cuda")
        F.embedding_lookup(table, torch.tensor([0, -1]).cuda(), out)
        got, want = out[0].cpu(), x[0].to(dtype)
        assert torch.equal(got.isnan(), want.isnan())
        ints = torch.int32 if dtype == torch.float32 else torch.int16
        ok = ~want.isnan()
        assert torch.equal(got.view(ints)[ok], want.view(ints)[ok])     # signs of zero, denormals
        assert (out[1] == 0).all()


def _chunk(tokens):
    return max(32, (-(-tokens // 2048) + 7) // 8 * 8)


def _check_grad(ids, dev, vocab, dtype, scale, got, what, before=None):
    tokens = len(ids)
    d, size, count = OE.grad(ids, dev.double().cpu().numpy(), vocab, scale)
    got = got.double().cpu().numpy()
    want = d if before is None else before + d
    if before is not None:
        untouched = count == 0
        assert np.array_equal(got[untouched], before[untouched]), what + ": rows without a token"
    tol = U * (size * (2 * _chunk(tokens) + 1) + np.abs(d) + np.abs(want))
    info = torch.finfo(T[dtype])
    tol += np.maximum((np.abs(want) + tol) * info.eps / 2, info.tiny * info.eps / 2)
    C.close(got, want, tol, what)


@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_grad(shape, dtype, out):
    tokens, vocab, dim, pad, shift = shape
    rng = _seed(*shape, 2)
    t, _ = C.to_dtype(rng.standard_normal((tokens, dim)), dtype)
    dev, _ = C.on_device(t, pad, shift)
    ids = _ids(rng, tokens, vocab)
    idt = torch.from_numpy(ids).cuda()
    like = torch.zeros(vocab, dim, dtype=T[out])
    for scale in (1.0, -0.3):
        say(f"grad {shape} {dtype} -> {out} scale={scale}")
        scale = float(np.float32(scale))
        got, whole = C.filled_like(like, (pad + 1) % 7, shift // 2)
        F.embedding_grad(idt, dev, got, scale=scale)
        _check_grad(ids, dev, vocab, out, scale, got, f"set {shape} {dtype} -> {out}")
        C.assert_between_rows_untouched(got, whole, f"{shape}")
        old, before = C.to_dtype(rng.standard_normal((vocab, dim)), out)
        got.copy_(old)
        F.embedding_grad(idt, dev, got, scale=scale, accumulate=True)
        _check_grad(ids, dev, vocab, out, scale, got, f"add {shape} {dtype} -> {out}", before)
        C.assert_between_rows_untouched(got, whole, f"{shape}")


# Around a chunk of 32 tokens, chunks of more than 32 tokens (65,537 and up), tokens sorted in one
# launch by smaller and larger work-groups (up to 16,384 and 131,072 tokens, or fewer for a large
# vocabulary) and by digits, around a sorting work-group's
# 4096, the largest digits, rows narrower and wider than a wave.
@pytest.mark.parametrize("tokens,vocab,dim", [(31, 9, 16), (32, 9, 16), (33, 9, 16), (4097, 300, 8),
                                              (16384, 32000, 24), (16385, 32000, 24), (65537, 1000, 8), (20001, 700, 520),
                                              (131072, 32000, 8), (131073, 300, 8),
                                              (135168, 131072, 8), (135169, 70000, 8),
                                              (3000, 1 << 21, 8), (4097, 1 << 21, 8)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grad_of_many_tokens(tokens, vocab, dim, accumulate):
    rng = _seed(tokens, vocab)
    t, _ = C.to_dtype(rng.standard_normal((tokens, dim)), "bf16")
    dev = t.cuda()
    ids = _ids(rng, tokens, vocab, skew=4.0)
    got = torch.full((vocab, dim), 3.0, device="cuda")
    say(f"grad tokens={tokens} vocab={vocab} accumulate={accumulate}")
    F.embedding_grad(torch.from_numpy(ids).cuda(), dev, got, accumulate=accumulate)
    _check_grad(ids, dev, vocab, "fp32", 1.0, got, f"{tokens} {vocab}",
                np.full((vocab, dim), 3.0) if accumulate else None)


@pytest.mark.parametrize("kind", ["one token", "two", "sorted", "reversed", "none", "past", "every"])
@pytest.mark.parametrize("tokens", [1, 100, 9000, 70000])
def test_grad_of_special_tokens(kind, tokens):
    rng = _seed(tokens, len(kind))
    vocab, dim = 200, 40
    ids = {"one token": np.full(tokens, 7), "two": rng.integers(0, 2, tokens) * 199,
           "sorted": np.sort(rng.integers(0, vocab, tokens)),
           "reversed": np.sort(rng.integers(0, vocab, tokens))[::-1].copy(),
           "none": np.full(tokens, -1), "past": np.full(tokens, vocab),
           "every": np.arange(tokens) % vocab}[kind].astype(np.int64)
    t, _ = C.to_dtype(rng.standard_normal((tokens, dim)), "fp16")
    dev = t.cuda()
    dev[torch.from_numpy((ids < 0) | (ids >= vocab))] = float("nan")      # never read
    for out in ("bf16", "fp32"):
        got = torch.full((vocab, dim), 3.0, dtype=T[out], device="cuda")
        say(f"grad {kind} tokens={tokens} {out}")
        F.embedding_grad(torch.from_numpy(ids).cuda(), dev, got)
        clean = torch.nan_to_num(dev.float())
        _check_grad(ids, clean, vocab, out, 1.0, got, f"{kind} {tokens} {out}")


def test_grad_without_tokens_sets_zeros():
    got = torch.full((300, 70), 3.0, dtype=torch.bfloat16, device="cuda")
    F.embedding_grad(torch.empty(0, dtype=torch.int64, device="cuda"),
                     torch.empty(0, 70, dtype=torch.bfloat16, device="cuda"), got)
    assert (got == 0).all()
    got.fill_(3)
    F.embedding_grad(torch.empty(0, dtype=torch.int64, device="cuda"),
                     torch.empty(0, 70, dtype=torch.bfloat16, device="cuda"), got, accumulate=True)
    assert (got == 3).all()


def test_grad_repeats_bit_for_bit():
    rng = _seed(91)
    ids = torch.from_numpy(_ids(rng, 30011, 500, skew=6.0)).cuda()
    dev = torch.randn(30011, 136, device="cuda")
    a, b = (torch.empty(500, 136, device="cuda") for _ in range(2))
    F.embedding_grad(ids, dev, a)
    ws = torch.full((F.embedding_grad_workspace_bytes(30011, 500, 136),), 255, dtype=torch.uint8,
                    device="cuda")
    F.embedding_grad(ids, dev, b, workspace=ws)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))


def test_lookup_and_gradient_are_adjoint():
    """<lookup(table), dout> = <table, grad(dout)>, and a difference quotient of the former."""
    rng = _seed(93)
    table, dout = rng.standard_normal((50, 24)), rng.standard_normal((90, 24))
    ids = _ids(rng, 90, 50, outside=False)
    idt = torch.from_numpy(ids).cuda()
    tt, dd = (torch.from_numpy(x.astype(np.float32)).cuda() for x in (table, dout))
    out, grad = torch.empty(90, 24, device="cuda"), torch.empty(50, 24, device="cuda")
    F.embedding_lookup(tt, idt, out, scale=1.5)
    F.embedding_grad(idt, dd, grad, scale=1.5)
    a, b = (out.double() * dd.double()).sum(), (tt.double() * grad.double()).sum()
    size = (out.double() * dd.double()).abs().sum()
    assert abs(a - b) <= 40 * U * size
    h = 2.0 ** -6
    for v, j in ((0, 0), (int(ids[5]), 3), (49, 23)):
        up = tt.clone()
        up[v, j] += h
        two = torch.empty(90, 24, device="cuda")
        F.embedding_lookup(up, idt, two, scale=1.5)
        step = float(up[v, j].double() - tt[v, j].double())
        num = ((two.double() - out.double()) * dd.double()).sum() / step
        assert abs(num - grad[v, j]) <= 8 * U * (out.abs().max() * dd.abs().sum()) / h


@pytest.mark.parametrize("tokens,dim", [(3, 1 << 18), (1, (1 << 20) - 3)])
def test_wide_rows(tokens, dim):
    rng = _seed(tokens, dim)
    t, _ = C.to_dtype(rng.standard_normal((4, dim)), "bf16")
    ids = torch.tensor([2, 0, 2][:tokens]).cuda()
    out = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    F.embedding_lookup(t.cuda(), ids, out)
    assert torch.equal(out.cpu(), t[ids.cpu()])
    got = torch.empty(4, dim, device="cuda")
    F.embedding_grad(ids, out, got)
    want = torch.zeros(4, dim).index_add_(0, ids.cpu(), out.cpu().float())
    assert torch.equal(got.cpu(), want)                  # two terms at most: one rounding


def test_table_beyond_2_31_elements():
    """Offsets of rows and of the gradient's rows pass 32 bits."""
    vocab, dim = 140000, 16384                           # 2.29e9 elements, 4.6 GB
    table = torch.zeros(vocab, dim, dtype=torch.bfloat16, device="cuda")
    table[vocab - 1] = 3.0
    table[vocab - 2] = 2.0
    ids = torch.tensor([vocab - 1, 0, vocab - 2, vocab - 1]).cuda()
    out = torch.empty(4, dim, dtype=torch.bfloat16, device="cuda")
    say("lookup beyond 2^31 elements")
    F.embedding_lookup(table, ids, out)
    assert [float(x) for x in out[:, dim - 1]] == [3.0, 0.0, 2.0, 3.0]
    say("grad beyond 2^31 elements")
    F.embedding_grad(ids, out, table)
    assert float(table[vocab - 1].float().mean()) == 6.0
    assert float(table[vocab - 2].float().mean()) == 2.0
    assert float(table[:vocab - 2].float().abs().max()) == 0.0


def test_tokens_beyond_2_31_elements():
    """Offsets of the tokens' rows pass 32 bits, written and read."""
    tokens, dim = 140000, 16384                          # 2.29e9 elements, 4.6 GB
    table = torch.arange(4, device="cuda", dtype=torch.bfloat16)[:, None].expand(4, dim).contiguous()
    ids = torch.zeros(tokens, dtype=torch.int64, device="cuda")
    ids[-2:] = torch.tensor([3, -1]).cuda()
    ids[-70000] = 2
    out = torch.full((tokens, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    say("lookup of 2.29e9 elements")
    F.embedding_lookup(table, ids, out)
    assert float(out[-2].float().min()) == 3.0 and float(out[-1].float().abs().max()) == 0.0
    assert float(out[-70000].float().min()) == 2.0
    assert float(out.sum(dtype=torch.float64)) == (3.0 + 2.0) * dim
    ids[ids == 0] = -1
    say("grad of 2.29e9 elements")
    got = torch.empty(4, dim, device="cuda")
    F.embedding_grad(ids, out, got)
    assert [float(x) for x in got.sum(1)] == [0.0, 0.0, 2.0 * dim, 3.0 * dim]
