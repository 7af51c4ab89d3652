"""Refusals of the operators over logits, without a GPU: every call here stops in the argument
checks, before anything is enqueued (or has no rows)."""

import ctypes

import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F

OK, INVALID, OVERFLOW, CAPACITY, ALIGN, UNSUP, HIPERR = range(7)
BASE = 1 << 40                       # addresses are only compared, never read


def _at(i):
    return BASE + (i << 32)


def _logits(**kw):
    a = dict(data=_at(0), rows=4, vocab=100, row_stride=100, dtype=0, scale=1.0)
    a.update(kw)
    return F._Logits(a["data"], a["rows"], a["vocab"], a["row_stride"], a["dtype"], a["scale"])


def _teacher(**kw):
    a = dict(ids=_at(1), values=_at(2), row_stride=8, k=8, tail=0)
    a.update(kw)
    return F._Teacher(a["ids"], a["values"], a["row_stride"], a["k"], a["tail"])


def logprobs(x=None, ids=_at(3), logprob=_at(4), entropy=_at(5), stats=_at(6), k=2,
             top_ids=_at(7), top_logprobs=_at(8), ws=_at(9), wbytes=1 << 24):
    x = _logits() if x is None else x
    return F.lib().token_logprobs(ctypes.byref(x), ids, logprob, entropy, stats, k, top_ids,
                                  top_logprobs, ws, wbytes, None)


def logprobs_grad(x=None, ids=_at(3), stats=_at(6), entropy=_at(5), g=_at(4), h=_at(7),
                  out=_at(10), stride=100):
    x = _logits() if x is None else x
    return F.lib().token_logprobs_grad(ctypes.byref(x), ids, stats, entropy, g, h, out, stride,
                                       None)


def distill(x=None, t=None, loss=_at(4), stats=_at(6), ws=_at(9), wbytes=1 << 24):
    x, t = _logits() if x is None else x, _teacher() if t is None else t
    return F.lib().distill_topk(ctypes.byref(x), ctypes.byref(t), loss, stats, ws, wbytes, None)


def distill_grad(x=None, t=None, stats=_at(6), g=_at(5), out=_at(10), stride=100):
    x, t = _logits() if x is None else x, _teacher() if t is None else t
    return F.lib().distill_topk_grad(ctypes.byref(x), ctypes.byref(t), stats, g, out, stride, None)


def distill_loss_grad(x=None, t=None, g=_at(5), loss=_at(4), stats=_at(6), out=_at(10),
                      stride=100, ws=_at(9), wbytes=1 << 24):
    x, t = _logits() if x is None else x, _teacher() if t is None else t
    return F.lib().distill_topk_loss_grad(ctypes.byref(x), ctypes.byref(t), g, loss, stats, out,
                                          stride, ws, wbytes, None)


CALLS = [logprobs, logprobs_grad, distill, distill_grad, distill_loss_grad]


@pytest.mark.parametrize("call", CALLS)
def test_bad_logits_are_refused(call):
    for bad in (dict(rows=-1), dict(vocab=0), dict(vocab=-3), dict(row_stride=99), dict(dtype=3),
                dict(dtype=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(data=None)):
        assert call(x=_logits(**bad)) == INVALID, bad
    assert call(x=_logits(vocab=(1 << 30) + 1, row_stride=1 << 31)) == UNSUP
    assert call(x=_logits(data=_at(0) + 1)) == ALIGN
    assert call(x=_logits(data=_at(0) + 2, dtype=2)) == ALIGN
    assert call(x=_logits(rows=1 << 40, row_stride=1 << 40)) == OVERFLOW
    assert call(x=_logits(rows=1 << 62, row_stride=100)) == OVERFLOW


@pytest.mark.parametrize("call", CALLS)
def test_no_rows_is_a_no_op(call):
    assert call(x=_logits(rows=0, data=None)) == OK


@pytest.mark.parametrize("call", [distill, distill_grad, distill_loss_grad])
def test_bad_lists_are_refused(call):
    for bad in (dict(k=0), dict(k=-1), dict(row_stride=7), dict(tail=2), dict(tail=-1),
                dict(ids=None), dict(values=None)):
        assert call(t=_teacher(**bad)) == INVALID, bad
    assert call(t=_teacher(k=129, row_stride=129)) == UNSUP
    assert call(t=_teacher(ids=_at(1) + 2)) == ALIGN
    assert call(t=_teacher(values=_at(2) + 1)) == ALIGN
    assert call(t=_teacher(row_stride=1 << 62)) == OVERFLOW


def test_logprobs_refusals():
    assert logprobs(ids=None) == INVALID and logprobs(logprob=None) == INVALID
    assert logprobs(k=-1) == INVALID and logprobs(k=129) == UNSUP
    assert logprobs(top_ids=None) == INVALID and logprobs(top_logprobs=None) == INVALID
    assert logprobs(k=0) == INVALID                        # lists without places
    for name in ("logprob", "entropy", "stats", "top_ids", "top_logprobs"):
        assert logprobs(**{name: _at(11) + 2}) == ALIGN, name
        assert logprobs(**{name: _at(0) + 16}) == INVALID, name       # inside the logits
        assert logprobs(**{name: _at(3)}) == INVALID, name            # the tokens
    assert logprobs(ids=_at(3) + 4) == ALIGN
    assert logprobs(entropy=_at(4) + 12) == INVALID        # two outputs share an element
    assert logprobs(ws=_at(9) + 8) == ALIGN
    assert logprobs(ws=None) == INVALID and logprobs(wbytes=-1) == INVALID
    assert logprobs(ws=_at(0) - 64) == INVALID


def test_logprobs_grad_refusals():
    assert logprobs_grad(stats=None) == INVALID and logprobs_grad(out=None) == INVALID
    assert logprobs_grad(g=None, h=None) == INVALID
    assert logprobs_grad(ids=None) == INVALID              # g without tokens
    assert logprobs_grad(entropy=None) == INVALID          # h without entropies
    assert logprobs_grad(stride=99) == INVALID
    assert logprobs_grad(out=_at(0) + 200) == INVALID      # overlaps the logits, not in place
    assert logprobs_grad(out=_at(0), stride=101) == INVALID
    for name in ("stats", "entropy", "g", "h"):
        assert logprobs_grad(**{name: _at(11) + 2}) == ALIGN, name
        assert logprobs_grad(**{name: _at(10) + 64}) == INVALID, name
    assert logprobs_grad(ids=_at(10) + 64) == INVALID
    assert logprobs_grad(out=_at(10) + 1) == ALIGN
    assert logprobs_grad(out=_at(10), stride=1 << 62) == OVERFLOW


@pytest.mark.parametrize("call", [distill, distill_loss_grad])
def test_distill_loss_refusals(call):
    assert call(loss=None) == INVALID
    assert call(loss=_at(11) + 2) == ALIGN and call(stats=_at(11) + 1) == ALIGN
    for where in (_at(0) + 16, _at(1) + 16, _at(2) + 16):
        assert call(loss=where) == INVALID and call(stats=where) == INVALID
    assert call(loss=_at(6) + 60) == INVALID               # the last element of the statistics
    assert call(ws=None) == INVALID and call(wbytes=-1) == INVALID and call(ws=_at(9) + 4) == ALIGN
    assert call(ws=_at(1) - 64) == INVALID


def test_distill_grad_refusals():
    for call in (distill_grad, distill_loss_grad):
        assert call(stats=None) == INVALID and call(g=None) == INVALID
        assert call(out=None) == INVALID and call(stride=99) == INVALID
        assert call(g=_at(11) + 2) == ALIGN
        assert call(out=_at(0) + 200) == INVALID and call(out=_at(0), stride=104) == INVALID
        for where in (_at(1) - 200, _at(2) - 200, _at(6) - 200, _at(5) - 200):
            assert call(out=where) == INVALID
    assert distill_loss_grad(loss=_at(10) + 64) == INVALID
    assert distill_loss_grad(x=_logits(), out=_at(0), loss=_at(0) + 64) == INVALID


def test_workspace_sizes():
    assert F.token_logprobs_workspace_bytes(0, 1, 0) >= 0
    assert F.token_logprobs_workspace_bytes(-1, 1, 0) == -1
    assert F.token_logprobs_workspace_bytes(1, 0, 0) == -1
    assert F.token_logprobs_workspace_bytes(1, 5, 129) == -1
    assert F.token_logprobs_workspace_bytes(1, 5, -1) == -1
    assert F.distill_topk_workspace_bytes(-1, 5) == -1
    assert F.distill_topk_workspace_bytes(1, (1 << 30) + 1) == -1
    for rows, vocab in ((1, 32000), (1, 131072), (16, 131072), (100000, 32000)):
        need = F.token_logprobs_workspace_bytes(rows, vocab, 128)
        if need:
            assert logprobs(x=_logits(rows=rows, vocab=vocab, row_stride=vocab), k=128,
                            wbytes=need - 1) == CAPACITY
        need = F.distill_topk_workspace_bytes(rows, vocab)
        if need:
            x = _logits(rows=rows, vocab=vocab, row_stride=vocab)
            assert distill(x=x, wbytes=need - 1) == CAPACITY


def test_binding_refuses_host_tensors_and_wrong_shapes():
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        F.token_logprobs(x, entropy=torch.zeros(2))
    with pytest.raises(ValueError, match="device tensor"):
        F.token_logprobs_grad(x, None, torch.zeros(2, 2), x, dlogprob=torch.zeros(2))
    with pytest.raises(ValueError, match="device tensor"):
        F.distill_topk(x, torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1), torch.zeros(2))


def test_header_is_plain_c(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "use.c"
    src.write_text('#include "fsdpshard_logits.h"\n'
                   'int use(const fsdpshard_logits* x, const fsdpshard_teacher* t, float* f) {\n'
                   '    return distill_topk(x, t, f, f, 0, 0, 0) + (FSDPSHARD_MAX_VOCAB > 0);\n}\n')
    subprocess.run(["gcc", "-std=c99", "-pedantic", "-Wall", "-Wextra", "-Werror", "-fsyntax-only",
                    f"-I{os.path.join(root, 'include')}", str(src)], check=True)


MOST = 1 << 21                       # the largest vocabulary that the header promises


@pytest.mark.parametrize("call", CALLS)
def test_vocabulary_limit(call):
    wide = dict(row_stride=1 << 22, rows=0)
    assert call(x=_logits(vocab=MOST, **wide)) == OK
    assert call(x=_logits(vocab=MOST + 1, **wide)) == UNSUP
    assert call(x=_logits(vocab=MOST + 1, row_stride=1 << 22, rows=1)) == UNSUP


def test_vocabulary_limit_of_the_workspaces():
    for rows in (1, 4, 1000):
        need = F.token_logprobs_workspace_bytes(rows, MOST, 128)
        assert need > 0 and F.token_logprobs_workspace_bytes(rows, MOST + 1, 128) == -1
        x = _logits(rows=rows, vocab=MOST, row_stride=MOST)
        assert logprobs(x=x, k=128, wbytes=need - 1) == CAPACITY
        need = F.distill_topk_workspace_bytes(rows, MOST)
        assert need > 0 and F.distill_topk_workspace_bytes(rows, MOST + 1) == -1
        assert distill(x=x, wbytes=need - 1) == CAPACITY
        assert distill_loss_grad(x=x, stride=MOST, wbytes=need - 1) == CAPACITY
