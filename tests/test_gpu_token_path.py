"""The token path's operators as a training step uses them: a run from the embedding to the sharded
update, two calls at once on two streams and in two graphs, a captured and replayed call, and a call on
another stream than the current one.  Results are compared bit for bit with the same calls made one
after the other; the run, with the float64 oracles."""

import numpy as np
import pytest
import torch

import fsdp_sharded_optimizer_layout_amd as F
import logits_cases as C
from gpu_helpers import say
from oracle import policy as OP
from test_gpu_policy_logits import check

pytestmark = pytest.mark.gpu


class _Work:
    """One caller's inputs, and its calls: every operator, in sizes that go through workspaces."""

    def __init__(self, seed, tokens=9001, vocab=4001, dim=72, rows=40, classes=70001):
        g = torch.Generator(device="cuda").manual_seed(seed)
        f = dict(generator=g, device="cuda")
        self.ids = (torch.rand(tokens, **f) ** 3 * vocab).long()
        self.ids[torch.rand(tokens, **f) < 0.1] = -1
        self.table = torch.randn(vocab, dim, **f).bfloat16()
        self.dout = torch.randn(tokens, dim, **f).bfloat16()
        self.lp = -torch.rand(tokens, **f) * 4
        self.old = self.lp + torch.randn(tokens, **f) * 0.2
        self.ref = self.lp + torch.randn(tokens, **f) * 0.3
        self.H, self.A = torch.rand(tokens, **f), torch.randn(tokens, **f)
        self.w = (torch.rand(tokens, **f) > 0.3).float()
        cuts = torch.randint(0, tokens + 1, (41,), **f).sort().values
        cuts[0], cuts[-1] = 0, tokens
        self.offsets = cuts
        self.g = torch.randn(20, **f)
        self.x = torch.randn(rows, classes, **f).bfloat16()
        self.y = torch.randint(0, classes, (rows,), **f)
        self.row_A, self.row_w = torch.randn(rows, **f), torch.ones(rows, device="cuda")
        self.row_old, self.row_ref = (torch.randn(rows, **f) - 11 for _ in range(2))

    def buffers(self):
        n, f = self.lp.numel(), dict(dtype=torch.float32, device="cuda")
        b = dict(out=torch.empty_like(self.dout), d=torch.empty_like(self.table),
                 acc=torch.empty(self.table.shape, **f), loss=torch.empty(n, **f),
                 g=torch.empty(n, **f), h=torch.empty(n, **f), totals=torch.empty(4, **f),
                 counts=torch.empty(2, dtype=torch.int64, device="cuda"), g2=torch.empty(n, **f),
                 totals2=torch.empty(4, **f), pair=torch.empty(20, **f), won=torch.empty(20, 2, **f),
                 g3=torch.empty(n, **f), row=torch.empty(self.x.shape[0], **f),
                 dx=torch.empty_like(self.x))
        for t in b.values():
            t.fill_(7)
        return b

    def calls(self, b, stream=None):
        terms = dict(old_logprob=self.old, ref_logprob=self.ref, kl_coef=0.1, stream=stream)
        F.embedding_lookup(self.table, self.ids, b["out"], scale=2.0, stream=stream)
        F.embedding_grad(self.ids, self.dout, b["d"], scale=2.0, stream=stream)
        F.embedding_grad(self.ids, self.dout, b["acc"], stream=stream)
        F.embedding_grad(self.ids, self.dout, b["acc"], accumulate=True, stream=stream)
        F.policy_loss(self.lp, self.A, self.w, b["g"], loss=b["loss"], totals=b["totals"],
                      counts=b["counts"], entropy=self.H, dentropy=b["h"], entropy_coef=0.01,
                      **terms)
        F.policy_loss(self.lp, self.A, self.w, b["g2"], totals=b["totals2"], offsets=self.offsets,
                      **terms)
        F.preference_loss(self.lp, self.offsets, b["pair"], rewards=b["won"],
                          ref_logprob=self.ref, weight=self.w, dloss=self.g, dlogprob=b["g3"],
                          stream=stream)
        F.policy_logits_loss_grad(self.x, self.y, self.row_A, self.row_w, b["row"], b["dx"],
                                  old_logprob=self.row_old, ref_logprob=self.row_ref,
                                  kl_coef=0.01, stream=stream)


def _same(a, b, what):
    for n in a:
        assert torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)), f"{what}: {n}"


def _results(w):
    b = w.buffers()
    w.calls(b)
    torch.cuda.synchronize()
    return b


def test_two_streams_at_once():
    work = [_Work(s) for s in (1, 2)]
    want = [_results(w) for w in work]
    streams = [torch.cuda.Stream() for _ in work]
    for rep in range(3):
        got = [w.buffers() for w in work]
        torch.cuda.synchronize()
        for _ in range(3):                     # in turn, so that both streams have work waiting
            for w, b, s in zip(work, got, streams):
                with torch.cuda.stream(s):
                    w.calls(b)
        torch.cuda.synchronize()
        for i in range(2):
            _same(got[i], want[i], f"repeat {rep}, stream {i}")
        say(f"two streams, repeat {rep}")


def test_a_stream_that_is_not_the_current_one():
    """The binding's own workspaces stay with the stream that the call runs on."""
    w = _Work(3)
    want = _results(w)
    side = torch.cuda.Stream()
    got = w.buffers()
    torch.cuda.synchronize()
    for _ in range(3):
        w.calls(got, stream=side)
    torch.cuda.synchronize()
    _same(got, want, "side stream")


def test_two_graphs_at_once():
    work = [_Work(s) for s in (4, 5)]
    want, got, graphs = [_results(w) for w in work], [], []
    for w in work:
        got.append(w.buffers())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            w.calls(got[-1])
    streams = [torch.cuda.Stream() for _ in work]
    for rep in range(4):
        for b in got:
            for t in b.values():
                t.fill_(3)
        extra = work[0].x.float().sum()        # the program's own work between the replays
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
                g.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(extra)
        for i in range(2):
            _same(got[i], want[i], f"replay {rep}, graph {i}")
        say(f"two graphs, replay {rep}")


def _head(hidden, weight):
    """Logits of a linear head, in float64 on the CPU."""
    return hidden.double().cpu().numpy() @ weight.double().cpu().numpy().T


def test_a_policy_step_from_the_embedding_to_the_sharded_update():
    """Lookup from the flat parameter vector, a linear head, log probabilities, policy loss, gradients
    back to the embedding in the flat gradient, and the fused update of a rank's slice; in the joint
    call over logits, too."""
    vocab, dim, tokens = 300, 64, 200
    rng = np.random.default_rng(11)
    sizes = [7, vocab * dim, vocab * dim]               # a tensor before them: an odd place
    offsets = np.concatenate([[0], np.cumsum(sizes)])
    flat = torch.from_numpy(rng.standard_normal(offsets[-1]).astype(np.float32) * 0.3).bfloat16().cuda()
    table = flat[offsets[1]:offsets[2]].view(vocab, dim)
    head = flat[offsets[2]:].view(vocab, dim)
    prompt = torch.from_numpy(rng.integers(0, vocab, tokens)).cuda()
    answer = torch.from_numpy(C.tokens(rng, tokens, vocab)).cuda()
    f = dict(dtype=torch.float32, device="cuda")
    hidden = torch.empty(tokens, dim, dtype=torch.bfloat16, device="cuda")
    F.embedding_lookup(table, prompt, hidden, scale=dim ** 0.5)
    logits = torch.from_numpy(_head(hidden, head)).float().cuda()
    lp, H, stats = torch.empty(tokens, **f), torch.empty(tokens, **f), torch.empty(tokens, 2, **f)
    F.token_logprobs(logits, answer, logprob=lp, entropy=H, stats=stats)
    old = lp - 0.15 * torch.randn(tokens, generator=torch.Generator().manual_seed(1)).cuda()
    ref = lp - 0.3 * torch.randn(tokens, generator=torch.Generator().manual_seed(2)).cuda()
    A = torch.randn(tokens, generator=torch.Generator().manual_seed(3)).cuda()
    w = (answer >= 0).float() / (answer >= 0).sum()
    terms = dict(old_logprob=old, ref_logprob=ref, kl_coef=0.1, entropy_coef=0.01)
    g, h, dlogits = torch.empty(tokens, **f), torch.empty(tokens, **f), torch.empty_like(logits)
    loss = torch.empty(tokens, **f)
    F.policy_loss(lp, A, w, g, loss=loss, entropy=H, dentropy=h, **terms)
    F.token_logprobs_grad(logits, answer, stats, dlogits, dlogprob=g, entropy=H, dentropy=h)
    joint, jloss, jH = torch.empty_like(logits), torch.empty(tokens, **f), torch.empty(tokens, **f)
    F.policy_logits_loss_grad(logits, answer, A, w, jloss, joint, entropy=jH, **terms)
    c = OP.constants(kl_coef=0.1, entropy_coef=0.01)
    ids, host = answer.cpu().numpy(), lambda t: t.cpu().numpy()
    v = dict(old=host(old), ref=host(ref), A=host(A), w=host(w))
    x64 = logits.double().cpu().numpy()
    counted = (answer >= 0).float()
    for how, l, ent, d in (("apart", loss, H * counted, dlogits), ("joint", jloss, jH, joint)):
        check(x64, ids, v, c, 1.0, "fp32", dict(loss=host(l), logprob=host(lp), entropy=host(ent)), d,
              how)
    # back to the embedding: a bf16 contribution in the flat gradient, at the same odd place
    dhidden = (dlogits.double() @ head.double()).float()
    grad = torch.zeros_like(flat)
    dtable = grad[offsets[1]:offsets[2]].view(vocab, dim)
    F.embedding_grad(prompt, dhidden, dtable, scale=dim ** 0.5)
    want = torch.zeros(vocab, dim, dtype=torch.float64, device="cuda")
    want.index_add_(0, prompt, dhidden.double())
    want *= float(np.float32(dim ** 0.5))
    size = torch.zeros_like(want).index_add_(0, prompt, dhidden.double().abs()) * dim ** 0.5
    assert ((dtable.double() - want).abs() <= want.abs() * 2.0 ** -8 + size * 2.0 ** -18
            + 2.0 ** -133).all()
    # and the same gradient by autograd, in float64
    t = table.double().requires_grad_()
    z = (t[prompt] * float(np.float32(dim ** 0.5))) @ head.double().T
    logp = torch.log_softmax(z, 1)
    y = answer.clamp_min(0)
    at = logp.gather(1, y[:, None])[:, 0]
    r = (at - old.double()).exp()
    obj = torch.minimum(r * A, r.clamp(0.8, 1.2) * A.double())
    kl = (ref.double() - at).expm1() - (ref.double() - at)
    ent = -(logp.exp() * logp).sum(1)
    (w.double() * (-obj + 0.1 * kl - 0.01 * ent)).sum().backward()
    # The hidden state was rounded to bf16 before the head: 2^-8 of it, over the head's sum.
    assert (t.grad - want).norm() <= 0.05 * t.grad.norm()
    # the rank's slice of the update takes it as its contribution
    L, segs = F.shard_layout([int(s) for s in sizes], 2, 0)
    master = flat[:L.n].float().clone()
    m, v = torch.zeros(L.n, **f), torch.zeros(L.n, **f)
    before = master.clone()
    mine = grad[:L.n].clone()
    F.adamw_shard_step(master, m, v, [mine], step=1, lr=1e-3,
                       segs=F.segments_to_device(segs), n_segments=L.n_segments, flat=flat.clone(),
                       flat_index0=0, lo=0)
    moved = master - before
    some = mine.float().abs() > 1e-6
    assert some.any() and (moved[some].sign() == -mine[some].float().sign()).all()
