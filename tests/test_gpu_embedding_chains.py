"""The embedding gradient's float32 sums stay short however many tokens there are.  With u = 2^-24 and S
the sizes of a row's terms: a float32 sum of at most 64 of them is off by at most 63 u S, at most n =
tokens / 2^17 + 2 such sums added up by another n u S, a part of a run kept in float32 by u S, and the
result by a rounding of the float64 sum, of the product with the scale and, added to what was there, of
that sum: (64 + n) u S + 3 u |d| + u |before|, for results in float32."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
from gpu_helpers import say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _check(ids, dout, vocab, got, before=0.0):
    n = len(ids) // (1 << 17) + 2
    want, size = np.zeros((vocab, dout.shape[1])), np.zeros((vocab, dout.shape[1]))
    host = dout.double().cpu().numpy()
    for v in np.unique(ids):
        rows = host[ids == v]
        want[v], size[v] = rows.sum(0), np.abs(rows).sum(0)
    want += before
    tol = U * ((64 + n) * size + 3 * np.abs(want) + 4 * abs(before))
    bad = np.abs(got.double().cpu().numpy() - want) > tol
    assert not bad.any(), (bad.sum(), np.argwhere(bad)[:3])


# Terms are summed in parts of at least 32 tokens, 1 / 4096 of them all; a lone 1 starts a part.
@pytest.mark.parametrize("tokens,vocab,dim", [(65536, 3, 8), (200000, 5, 72), (1 << 20, 2, 8),
                                              ((1 << 20) + 77, 700, 520), (3 << 20, 1, 16)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_small_terms_after_a_large_one_are_not_lost(tokens, vocab, dim, accumulate):
    """A part starts with 1, and goes on with terms of three quarters of half its step, each of
    which a float32 sum rounds away."""
    ids = np.sort(np.random.default_rng([tokens, vocab]).integers(0, vocab, tokens))
    dout = torch.full((tokens, dim), 0.75 * U, device="cuda")
    part = max(32, (-(-tokens // 4096) + 7) // 8 * 8)
    dout[::part] = 1.0
    got = torch.full((vocab, dim), 0.5, device="cuda")
    say(f"{tokens} tokens of {vocab} rows, accumulate={accumulate}")
    F.embedding_grad(torch.from_numpy(ids).cuda(), dout, got, accumulate=accumulate)
    _check(ids, dout, vocab, got, 0.5 if accumulate else 0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_frequent_token_among_a_million(dtype):
    tokens, vocab, dim = (1 << 20) + 5, 1000, 40
    rng = np.random.default_rng(5)
    ids = (vocab * rng.random(tokens) ** 6).astype(np.int64)
    dout = torch.randn(tokens, dim, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    a, b = (torch.empty(vocab, dim, device="cuda") for _ in range(2))
    F.embedding_grad(torch.from_numpy(ids).cuda(), dout, a)
    _check(ids, dout, vocab, a)
    F.embedding_grad(torch.from_numpy(ids).cuda(), dout, b)
    assert torch.equal(a.view(torch.int32), b.view(torch.int32))


@pytest.mark.parametrize("lengths", [(64,), (65,), (66, 64), (95, 33, 97), (96,), (128, 1, 64), (63, 65)])
@pytest.mark.parametrize("first", [0, 1, 31])
def test_long_runs_next_to_each_other(lengths, first):
    """Runs of about two and three parts of 32 tokens, one after the other, at every place in a part;
    each part's sums have a place of their own."""
    runs, dim = 300, 72
    rows = np.repeat(np.arange(runs), np.resize(lengths, runs))
    ids = np.concatenate([np.full(first, runs), rows]).astype(np.int64)
    rng = np.random.default_rng([first, *lengths])
    ids = ids[rng.permutation(len(ids))]
    dout = torch.from_numpy(rng.standard_normal((len(ids), dim)).astype(np.float32)).cuda()
    got = torch.full((runs + 1, dim), 3.0, device="cuda")
    say(f"runs of {lengths} after {first}")
    F.embedding_grad(torch.from_numpy(ids).cuda(), dout, got)
    _check(ids, dout, runs + 1, got)
