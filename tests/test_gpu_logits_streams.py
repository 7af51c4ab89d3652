"""Operators over logits, two calls at once: on two streams, each with the workspace that the binding
allocates for its call, and in two captured graphs that are replayed side by side.  The results are
compared bit for bit with the same calls made one after the other."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say

pytestmark = pytest.mark.gpu

# Rows in parts, which go through the workspace: a few rows in two launches, many parts a row.
SIZES = [("bf16", 16, 131072), ("fp32", 64, 100003), ("bf16", 700, 140001)]


class _Work:
    """One caller's inputs, and its calls."""

    def __init__(self, dtype, rows, vocab, seed):
        rng = np.random.default_rng([rows, vocab, seed])
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.x = (torch.randn(rows, vocab, generator=gen, device="cuda") * 3).to(C.DTYPES[dtype])
        self.ids = torch.as_tensor(C.tokens(rng, rows, vocab)).cuda()
        # the teacher's list: the student's best tokens, with weights of their own
        self.tid = self.x.topk(16, 1).indices.int()
        w = torch.rand(rows, 16, generator=gen, device="cuda") + 0.01
        self.tv = (0.9 * w / w.sum(1, keepdim=True)).log()
        self.g = torch.ones(rows, device="cuda")

    def buffers(self):
        rows, f = self.x.shape[0], dict(dtype=torch.float32, device="cuda")
        return dict(lp=torch.full((rows,), 55.0, **f), H=torch.full((rows,), 55.0, **f),
                    st=torch.full((rows, 2), 55.0, **f),
                    ti=torch.full((rows, 16), 55, dtype=torch.int32, device="cuda"),
                    tl=torch.full((rows, 16), 55.0, **f),
                    loss=torch.full((rows,), 55.0, **f), ds=torch.full((rows, 4), 55.0, **f),
                    d=torch.full_like(self.x, 77.0))

    def calls(self, b, stream=None):
        F.token_logprobs(self.x, self.ids, logprob=b["lp"], entropy=b["H"], stats=b["st"],
                         top_ids=b["ti"], top_logprobs=b["tl"], stream=stream)
        F.distill_topk_loss_grad(self.x, self.tid, self.tv, self.g, b["loss"], b["ds"], b["d"],
                                 tail=True, stream=stream)


def _same(a, b, what):
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), f"{what}: {n}"


@pytest.mark.parametrize("dtype,rows,vocab", SIZES)
def test_two_streams_at_once(dtype, rows, vocab):
    work = [_Work(dtype, rows, vocab, s) for s in (1, 2)]
    want = []
    for w in work:
        want.append(w.buffers())
        w.calls(want[-1])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    for rep in range(3):
        got = [w.buffers() for w in work]
        torch.cuda.synchronize()
        for _ in range(4):                     # in turn, so that both streams have work waiting
            for w, b, s in zip(work, got, streams):
                w.calls(b, stream=s)
        torch.cuda.synchronize()
        for i in range(2):
            _same(got[i], want[i], f"{dtype} {rows} x {vocab}, repeat {rep}, stream {i}")
        say(f"two streams {dtype} {rows} x {vocab}, repeat {rep}")


@pytest.mark.parametrize("dtype,rows,vocab", SIZES[:2])
def test_two_graphs_at_once(dtype, rows, vocab):
    work = [_Work(dtype, rows, vocab, s) for s in (3, 4)]
    want, got, graphs = [], [], []
    for w in work:
        want.append(w.buffers())
        w.calls(want[-1])
    torch.cuda.synchronize()
    for w in work:
        got.append(w.buffers())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w.calls(got[-1])
    streams = [torch.cuda.Stream() for _ in work]
    for rep in range(4):
        for b in got:
            for t in b.values():
                t.fill_(33)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            _same(got[i], want[i], f"{dtype} {rows} x {vocab}, replay {rep}, graph {i}")
        say(f"two graphs {dtype} {rows} x {vocab}, replay {rep}")
