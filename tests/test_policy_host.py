"""Refusals of the policy and preference losses and of the embedding, without a GPU: every call here
stops in the argument checks, before anything is enqueued (or has nothing to do)."""

import ctypes
import os
import subprocess

import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F

OK, INVALID, OVERFLOW, CAPACITY, ALIGN, UNSUP, HIPERR = range(7)
BASE = 1 << 40                       # addresses are only compared, never read
NAN, INF = float("nan"), float("inf")


def _at(i):
    return BASE + (i << 36)


def _terms(**kw):
    a = dict(clip_low=0.2, clip_high=0.2, dual_clip=0.0, kl_coef=0.1, entropy_coef=0.01)
    a.update(kw)
    return F._Policy(*(a[n] for n, _ in F._Policy._fields_))


def policy(terms=None, tokens=100, logprob=_at(0), old=_at(1), ref=_at(2), entropy=_at(3),
           advantage=_at(4), weight=_at(5), sequences=3, offsets=_at(6), loss=_at(7),
           dlogprob=_at(8), dentropy=_at(9), totals=_at(10), counts=_at(11), ws=_at(12),
           wbytes=1 << 30):
    t = _terms() if terms is None else terms
    return F.lib().policy_loss(ctypes.byref(t), tokens, logprob, old, ref, entropy, advantage,
                               weight, sequences, offsets, loss, dlogprob, dentropy, totals, counts,
                               ws, wbytes, None)


def _pref(**kw):
    a = dict(kind=0, length_normalised=0, beta=0.1, margin=0.0, label_smoothing=0.0)
    a.update(kw)
    return F._Preference(*(a[n] for n, _ in F._Preference._fields_))


def preference(terms=None, tokens=100, pairs=3, offsets=_at(6), logprob=_at(0), ref=_at(2),
               weight=_at(5), dloss=_at(4), loss=_at(7), rewards=_at(9), dlogprob=_at(8),
               ws=_at(12), wbytes=1 << 30):
    t = _pref() if terms is None else terms
    return F.lib().preference_loss(ctypes.byref(t), tokens, pairs, offsets, logprob, ref, weight,
                                   dloss, loss, rewards, dlogprob, ws, wbytes, None)


def _logits(**kw):
    a = dict(data=_at(20), rows=4, vocab=100, row_stride=100, dtype=0, scale=1.0)
    a.update(kw)
    return F._Logits(*(a[n] for n, _ in F._Logits._fields_))


def over_logits(x=None, ids=_at(21), terms=None, old=_at(1), ref=_at(2), advantage=_at(4),
                weight=_at(5), loss=_at(7), logprob=_at(8), entropy=_at(9), out=_at(22), stride=100,
                ws=_at(12), wbytes=1 << 30):
    x, t = _logits() if x is None else x, _terms() if terms is None else terms
    return F.lib().policy_logits_loss_grad(ctypes.byref(x), ids, ctypes.byref(t), old, ref,
                                           advantage, weight, loss, logprob, entropy, out, stride,
                                           ws, wbytes, None)


def _matrix(**kw):
    a = dict(data=_at(30), rows=50, cols=64, row_stride=64, dtype=0)
    a.update(kw)
    return F._Matrix(*(a[n] for n, _ in F._Matrix._fields_))


def lookup(table=None, ids=_at(31), out=None, scale=1.0):
    table = _matrix() if table is None else table
    out = _matrix(data=_at(32), rows=7) if out is None else out
    return F.lib().embedding_lookup(ctypes.byref(table), ids, ctypes.byref(out), scale, None)


def grad(ids=_at(31), dout=None, table=None, scale=1.0, accumulate=0, ws=_at(12),
         wbytes=1 << 30):
    table = _matrix() if table is None else table
    dout = _matrix(data=_at(32), rows=7) if dout is None else dout
    return F.lib().embedding_grad(ids, ctypes.byref(dout), ctypes.byref(table), scale, accumulate,
                                  ws, wbytes, None)


@pytest.mark.parametrize("call", [policy, over_logits])
def test_bad_policy_constants_are_refused(call):
    for bad in (dict(clip_low=-0.1), dict(clip_low=NAN), dict(clip_high=-0.1), dict(clip_high=NAN),
                dict(dual_clip=0.5), dict(dual_clip=-1.0), dict(dual_clip=INF), dict(dual_clip=NAN),
                dict(kl_coef=-0.1), dict(kl_coef=INF), dict(kl_coef=NAN), dict(entropy_coef=INF),
                dict(entropy_coef=NAN)):
        assert call(terms=_terms(**bad)) == INVALID, bad
    assert call(ref=None) == INVALID                       # a KL term without a reference


def test_policy_refusals():
    assert policy(tokens=-1) == INVALID and policy(sequences=-1) == INVALID
    assert policy(tokens=(1 << 40) + 1) == UNSUP
    assert policy(sequences=1 << 31) == UNSUP
    assert policy(offsets=None) == INVALID and policy(sequences=0) == INVALID
    assert policy(entropy=None) == INVALID
    for name in ("logprob", "advantage", "weight"):
        assert policy(**{name: None}) == INVALID, name
    for name in ("logprob", "old", "ref", "entropy", "advantage", "weight", "loss", "dlogprob",
                 "dentropy", "totals"):
        assert policy(**{name: _at(15) + 2}) == ALIGN, name
    assert policy(offsets=_at(15) + 4) == ALIGN and policy(counts=_at(15) + 4) == ALIGN
    for name in ("loss", "dlogprob", "dentropy", "totals", "counts", "ws"):
        for where in range(7):
            assert policy(**{name: _at(where)}) == INVALID, (name, where)
    assert policy(loss=_at(8) + 396) == INVALID            # two outputs share an element
    assert policy(totals=_at(11) + 8) == INVALID
    assert policy(ws=None) == INVALID and policy(wbytes=-1) == INVALID
    assert policy(ws=_at(12) + 8) == ALIGN


def test_preference_refusals():
    for bad in (dict(kind=-1), dict(kind=3), dict(length_normalised=2), dict(beta=0.0),
                dict(beta=-1.0), dict(beta=INF), dict(beta=NAN), dict(margin=INF), dict(margin=NAN),
                dict(label_smoothing=-0.1), dict(label_smoothing=0.6), dict(label_smoothing=NAN),
                dict(kind=1, label_smoothing=0.1)):
        assert preference(terms=_pref(**bad)) == INVALID, bad
    assert preference(tokens=-1) == INVALID and preference(pairs=-1) == INVALID
    assert preference(tokens=(1 << 40) + 1) == UNSUP and preference(pairs=1 << 30) == UNSUP
    for name in ("offsets", "logprob", "loss", "dloss", "dlogprob"):
        assert preference(**{name: None}) == INVALID, name
    for name in ("logprob", "ref", "weight", "dloss", "loss", "rewards", "dlogprob"):
        assert preference(**{name: _at(15) + 2}) == ALIGN, name
    assert preference(offsets=_at(15) + 4) == ALIGN
    for name in ("loss", "rewards", "dlogprob", "ws"):
        for where in (0, 2, 4, 5, 6):
            assert preference(**{name: _at(where)}) == INVALID, (name, where)
    assert preference(loss=_at(9) + 20) == INVALID
    assert preference(ws=None) == INVALID and preference(ws=_at(12) + 4) == ALIGN


def test_policy_over_logits_refusals():
    for bad in (dict(rows=-1), dict(vocab=0), dict(row_stride=99), dict(dtype=3), dict(scale=0.0),
                dict(scale=NAN), dict(data=None)):
        assert over_logits(x=_logits(**bad)) == INVALID, bad
    assert over_logits(x=_logits(data=_at(20) + 1)) == ALIGN
    assert over_logits(x=_logits(vocab=(1 << 21) + 1, row_stride=1 << 22)) == UNSUP
    assert over_logits(x=_logits(rows=1 << 40, row_stride=1 << 40)) == OVERFLOW
    for name in ("ids", "advantage", "weight", "loss", "out"):
        assert over_logits(**{name: None}) == INVALID, name
    assert over_logits(stride=99) == INVALID and over_logits(out=_at(22) + 1) == ALIGN
    assert over_logits(ids=_at(15) + 4) == ALIGN
    for name in ("old", "ref", "advantage", "weight", "loss", "logprob", "entropy"):
        assert over_logits(**{name: _at(15) + 2}) == ALIGN, name
    for name in ("loss", "logprob", "entropy", "out", "ws"):
        for where in (1, 2, 4, 5, 21):
            assert over_logits(**{name: _at(where)}) == INVALID, (name, where)
    assert over_logits(out=_at(20) + 200) == INVALID       # overlaps the logits, not in place
    assert over_logits(out=_at(20), stride=101) == INVALID
    assert over_logits(loss=_at(20)) == INVALID
    assert over_logits(loss=_at(8) + 12) == INVALID        # two outputs share an element
    assert over_logits(ws=None) == INVALID and over_logits(ws=_at(12) + 8) == ALIGN


def test_embedding_refusals():
    for bad in (dict(rows=-1), dict(cols=0), dict(cols=-1), dict(row_stride=63), dict(dtype=3),
                dict(dtype=-1), dict(data=None)):
        assert lookup(table=_matrix(**bad)) == INVALID, bad
        assert lookup(out=_matrix(**{"data": _at(32), **bad})) == INVALID, bad
        assert grad(table=_matrix(**bad)) == INVALID, bad
        assert grad(dout=_matrix(**{"data": _at(32), **bad})) == INVALID, bad
    for call in (lookup, grad):
        assert call(table=_matrix(cols=65, row_stride=65)) == INVALID       # another width
        assert call(ids=None) == INVALID and call(ids=_at(31) + 4) == ALIGN
        assert call(scale=INF) == INVALID and call(scale=NAN) == INVALID
        assert call(table=_matrix(data=_at(30) + 1)) == ALIGN
        assert call(table=_matrix(data=_at(30) + 2, dtype=2)) == ALIGN
        assert call(table=_matrix(cols=(1 << 20) + 1, row_stride=1 << 21)) == UNSUP
        assert call(table=_matrix(rows=(1 << 21) + 1)) == UNSUP
        assert call(table=_matrix(row_stride=1 << 60)) == OVERFLOW
    assert grad(dout=_matrix(data=_at(32), rows=(1 << 24) + 1), wbytes=1 << 40) == UNSUP
    assert grad(accumulate=2) == INVALID and grad(accumulate=-1) == INVALID
    assert lookup(out=_matrix(data=_at(30) + 128, rows=7)) == INVALID
    assert lookup(out=_matrix(data=_at(31), rows=7)) == INVALID
    assert grad(table=_matrix(data=_at(32))) == INVALID
    assert grad(table=_matrix(data=_at(31))) == INVALID
    for where in (30, 31, 32):
        assert grad(ws=_at(where)) == INVALID, where
    assert grad(ws=None) == INVALID and grad(wbytes=-1) == INVALID and grad(ws=_at(12) + 8) == ALIGN


def test_nothing_to_do_is_a_no_op():
    assert lookup(out=_matrix(data=None, rows=0), ids=None) == OK
    assert grad(dout=_matrix(data=None, rows=0), ids=None, accumulate=1) == OK
    assert grad(table=_matrix(data=None, rows=0)) == OK
    assert policy(tokens=0, totals=None, counts=None) == OK
    assert preference(pairs=0) == OK
    assert over_logits(x=_logits(rows=0, data=None)) == OK


def test_workspaces():
    assert F.policy_loss_workspace_bytes(-1, 0) == -1
    assert F.policy_loss_workspace_bytes(1, -1) == -1
    assert F.policy_loss_workspace_bytes((1 << 40) + 1, 0) == -1
    assert F.policy_loss_workspace_bytes(1, 1 << 31) == -1
    assert F.policy_loss_workspace_bytes(100, 0) == 0
    assert F.preference_loss_workspace_bytes(-1, 1) == -1
    assert F.preference_loss_workspace_bytes(1, 1 << 30) == -1
    assert F.policy_logits_loss_grad_workspace_bytes(-1, 5) == -1
    assert F.policy_logits_loss_grad_workspace_bytes(5, (1 << 21) + 1) == -1
    assert F.embedding_grad_workspace_bytes(-1, 5, 5) == -1
    assert F.embedding_grad_workspace_bytes(5, (1 << 21) + 1, 5) == -1
    assert F.embedding_grad_workspace_bytes(5, 5, 0) == -1
    assert F.embedding_grad_workspace_bytes((1 << 24) + 1, 5, 5) == -1
    for tokens, seqs in ((100, 3), (1 << 20, 0), (1 << 20, 3), (100, 5000)):
        need = F.policy_loss_workspace_bytes(tokens, seqs)
        kw = dict(tokens=tokens, sequences=seqs, offsets=_at(6) if seqs else None)
        assert need > 0 and policy(wbytes=need - 1, **kw) == CAPACITY
    for tokens, pairs in ((100, 3), (1 << 20, 3)):
        need = F.preference_loss_workspace_bytes(tokens, pairs)
        assert need > 0 and preference(tokens=tokens, pairs=pairs, wbytes=need - 1) == CAPACITY
    for tokens, vocab, dim in ((7, 50, 64), (100000, 1 << 21, 5)):
        need = F.embedding_grad_workspace_bytes(tokens, vocab, dim)
        assert need > 0 and grad(dout=_matrix(data=_at(32), rows=tokens, cols=dim, row_stride=dim),
                                 table=_matrix(rows=vocab, cols=dim, row_stride=dim),
                                 wbytes=need - 1) == CAPACITY
    need = F.policy_logits_loss_grad_workspace_bytes(4, 140001)
    assert need > 0 and over_logits(x=_logits(vocab=140001, row_stride=140001), stride=140001,
                                    wbytes=need - 1) == CAPACITY


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="device tensor"):
        F.policy_loss(x[0], x[0], x[0], x[0])
    with pytest.raises(ValueError, match="device tensor"):
        F.preference_loss(x[0], i, x[0])
    with pytest.raises(ValueError, match="device tensor"):
        F.policy_logits_loss_grad(x, i, x[0], x[0], x[0], x)
    with pytest.raises(ValueError, match="device tensor"):
        F.embedding_lookup(x, i, x)
    with pytest.raises(ValueError, match="device tensor"):
        F.embedding_grad(i, x, x)


@pytest.mark.parametrize("header,use", [
    ("fsdpshard_policy.h", "int use(const fsdpshard_policy* p, const fsdpshard_preference* q, "
     "float* f) { return policy_loss(p, 0, f, 0, 0, 0, f, f, 0, 0, f, f, f, f, 0, 0, 0, 0) + "
     "preference_loss(q, 0, 0, 0, f, 0, 0, 0, f, 0, 0, 0, 0, 0) + FSDPSHARD_SQUARED; }"),
    ("fsdpshard_embedding.h", "int use(const fsdpshard_matrix* m, const int64_t* i) { return "
     "embedding_lookup(m, i, m, 1, 0) + embedding_grad(i, m, m, 1, 0, 0, 0, 0); }")])
def test_headers_are_plain_c(tmp_path, header, use):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "use.c"
    src.write_text(f'#include "{header}"\n{use}\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-fsyntax-only",
                    f"-I{os.path.join(root, 'include')}", str(src)], check=True)
