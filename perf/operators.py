"""Measured cases of the operators over logits: token log probabilities and top-k distillation.

Five kinds of pass, each over a matrix of logits [rows, vocab] in bf16, fp16 or fp32:

  logprobs       log probability of a given token, entropy of the row and its top alternatives
  logprobs_grad  gradient of the logits for gradients of the log probability and the entropy
  distill        divergence from a teacher known by its top logits (loss for each row)
  distill_grad   its gradient of the logits
  distill_step   loss and gradient in one call, as a training step that knows its loss weights

With `own` false, run() computes a pass in elementary torch operations; with `own` true it calls
the framework.  Both take the same state, made by prepare() from a seed.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_NO_TOKEN = -100          # a position without a token: a prompt or padding position


def _case(name, op, dtype, rows, vocab, k=0, scale=1.0, pad=0, masked=0.0, ignored=0.0,
          tail=False, entropy=True):
    return dict(name=name, op=op, dtype=dtype, rows=rows, vocab=vocab, k=k, scale=scale, pad=pad,
                masked=masked, ignored=ignored, tail=tail, entropy=entropy)


def listed():
    return [
        # One new token of one sequence, sampled at temperature 0.7, reported with five
        # alternatives: the smallest call, where latency counts.
        _case("next_token_top", "logprobs", "bf16", 1, 32000, k=5, scale=1 / 0.7),
        # One decoding step of 16 sequences under a grammar that forbids a third of a large
        # vocabulary, 20 alternatives each.
        _case("decode_batch_top", "logprobs", "bf16", 16, 131072, k=20, masked=0.33),
        # Scoring a prompt with an odd vocabulary (rows start at any 2-byte phase).
        _case("score_prompt_odd", "logprobs", "fp16", 1021, 50021, k=1, ignored=0.1),
        # A teacher's pass over a batch with a large vocabulary: its 64 best tokens for each
        # position, stored as distillation targets.  The largest case.
        _case("teacher_top", "logprobs", "bf16", 4096, 131072, k=64),
        # Scoring a rollout for policy training: log probabilities and entropies only.
        _case("score_rollout", "logprobs", "bf16", 8192, 32000, ignored=0.2),
        # The policy loss's backward with an entropy bonus.
        _case("policy_grad", "logprobs_grad", "bf16", 8192, 32000, ignored=0.1),
        # The backward alone of a log probability in 32 bits, odd vocabulary, a quarter of the
        # positions without a token.
        _case("token_grad_odd", "logprobs_grad", "fp32", 515, 50021, ignored=0.25,
              entropy=False),
        # Evaluation of a distillation loss at temperature 2 on stored targets.
        _case("distill_loss", "distill", "bf16", 4096, 32000, k=32, scale=0.5),
        # The same with the mass outside the teacher's list in one bucket, odd sizes.
        _case("distill_loss_tail_odd", "distill", "fp16", 777, 100003, k=100, tail=True,
              ignored=0.1),
        # Backward of that loss where the weights come from a later computation.
        _case("distill_grad_tail", "distill_grad", "bf16", 4096, 32000, k=32, tail=True,
              ignored=0.1),
        # The training step's call: loss and gradient together.
        _case("distill_step", "distill_step", "bf16", 8192, 32000, k=64, scale=0.5, ignored=0.1),
        # A few positions of a large vocabulary in 32 bits.
        _case("distill_step_few", "distill_step", "fp32", 64, 131072, k=16, tail=True),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "logprobs_grad", "distill", "distill_grad",
                     "distill_step"])
    vocab = _log_uniform(rng, 1000, 131072)
    rows = _log_uniform(rng, 1, min(8192, (1 << 28) // vocab))
    if op == "logprobs":
        k = rng.choice([0, 1, rng.randint(2, 20), rng.randint(21, 128)])
    elif op == "logprobs_grad":
        k = 0
    else:
        k = _log_uniform(rng, 1, 128)
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows=rows, vocab=vocab,
                k=k, scale=rng.choice([1.0, 1.0, 0.5, 0.25, 1 / 0.7]),
                pad=rng.choice([0, 0, rng.randint(1, 64)]),
                masked=rng.choice([0.0, 0.0, rng.uniform(0.05, 0.9)]),
                ignored=rng.choice([0.0, rng.uniform(0.0, 0.5)]),
                tail=rng.random() < 0.5, entropy=rng.random() < 0.6)


def work(case):
    r, v, k = case["rows"], case["vocab"], case["k"]
    e = _DTYPES[case["dtype"]].itemsize
    read, op = r * v * e, case["op"]
    if op == "logprobs":
        return {"bytes": read + r * (8 + 4 + 4 + 8) + r * k * 8, "flops": 7 * r * v}
    if op == "logprobs_grad":
        return {"bytes": 2 * read + r * (8 + 8 + 4 + (8 if case["entropy"] else 0)),
                "flops": 7 * r * v}
    if op == "distill":
        return {"bytes": read + r * k * 8 + r * (4 + 16), "flops": 5 * r * v}
    if op == "distill_grad":
        return {"bytes": 2 * read + r * k * 8 + r * (4 + 16), "flops": 5 * r * v}
    return {"bytes": 2 * read + r * k * 8 + r * (4 + 4 + 16), "flops": 9 * r * v}


# ------------------------------------------------------------------------------------- inputs

def _strided(rows, vocab, pad, dtype):
    """A [rows, vocab] matrix whose rows are vocab + pad elements apart."""
    return torch.zeros(rows, vocab + pad, dtype=dtype, device="cuda")[:, :vocab]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    rows, vocab, k, dtype = case["rows"], case["vocab"], case["k"], _DTYPES[case["dtype"]]
    dev = dict(generator=gen, device="cuda")

    # Logits as a language model gives them: a broad bulk and a few likely tokens in each row.
    x = torch.randn(rows, vocab, **dev).mul_(2.5)
    likely = torch.randint(0, vocab, (rows, 6), **dev)
    x.scatter_add_(1, likely, torch.rand(rows, 6, **dev).mul_(12).add_(2))
    logits = _strided(rows, vocab, case["pad"], dtype)
    state = dict(op=case["op"], logits=logits, scale=case["scale"], k=k, tail=case["tail"])

    ignored = torch.rand(rows, **dev) < case["ignored"]
    if case["op"].startswith("logprobs"):
        ids = torch.where(torch.rand(rows, **dev) < 0.7, likely[:, 0],
                          torch.randint(0, vocab, (rows,), **dev))
        if case["masked"] > 0:
            forbidden = torch.rand(rows, vocab, **dev) < case["masked"]
            forbidden.scatter_(1, ids[:, None], False)
            x.masked_fill_(forbidden, -math.inf)
            del forbidden
        logits.copy_(x)
        state["ids"] = ids.masked_fill(ignored, _NO_TOKEN)
    else:
        logits.copy_(x)
        # The teacher agrees with the student up to noise; its list holds its best tokens.
        teacher = x.add_(torch.randn(rows, vocab, **dev).mul_(0.7))
        if case["tail"]:
            teacher = torch.log_softmax(teacher * case["scale"], 1)
        values, places = teacher.topk(k, 1)
        del teacher
        places = places.to(torch.int32)
        short = torch.randint(0, 2 * k + 1, (rows, 1), **dev)      # some lists are not full
        places.masked_fill_(torch.arange(k, device="cuda")[None] > short, -1)
        places.masked_fill_(ignored[:, None], -1)
        state["teacher_ids"] = places.contiguous()
        state["teacher_values"] = values.float().contiguous()
    del x

    f32 = dict(dtype=torch.float32, device="cuda")
    # A mean over the rows; gradients in fp16 are kept in range by a loss scale.
    weight = 1.0 if dtype == torch.float16 else 1.0 / rows
    if case["op"] == "logprobs":
        state.update(logprob=torch.empty(rows, **f32), entropy=torch.empty(rows, **f32),
                     stats=torch.empty(rows, 2, **f32),
                     top_ids=torch.empty(rows, k, dtype=torch.int32, device="cuda"),
                     top_logprobs=torch.empty(rows, k, **f32))
    elif case["op"] == "logprobs_grad":
        # What the forward pass left: the row's maximum, log-sum and entropy.
        peak, logsum, entropy = (torch.empty(rows, **f32) for _ in range(3))
        for i in range(0, rows, 512):
            z = logits[i:i + 512].double()
            m = z.amax(1, keepdim=True)
            logp = torch.log_softmax(z * case["scale"], 1)
            peak[i:i + 512] = m[:, 0]
            logsum[i:i + 512] = -logp.amax(1)
            entropy[i:i + 512] = -torch.special.xlogy(logp.exp(), logp.exp()).sum(1)
        state["stats"] = torch.stack([peak, logsum], 1).contiguous()
        state["dlogprob"] = torch.randn(rows, **dev) * weight
        if case["entropy"]:
            state["entropy"] = entropy
            state["dentropy"] = torch.rand(rows, **dev) * (-0.01 * weight)
            state["dentropy"][ignored] = 0.0
    else:
        state["dloss"] = torch.rand(rows, **dev) * weight
        if case["op"] == "distill_grad":
            loss, stats = _plain_distill(state)
            state["stats"] = stats
        else:
            state.update(loss=torch.empty(rows, **f32), stats=torch.empty(rows, 4, **f32))
    if case["op"] in ("logprobs_grad", "distill_grad", "distill_step"):
        state["dlogits"] = _strided(rows, vocab, case["pad"], dtype)
    if own:
        import fsdp_sharded_optimizer_layout_amd as F
        if case["op"] == "logprobs":
            need = F.token_logprobs_workspace_bytes(rows, vocab, k)
        else:
            need = F.distill_topk_workspace_bytes(rows, vocab)
        state["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        state["F"] = F
    return state


# --------------------------------------------------------------------------------- plain forms

def _plain_top(z, k):
    """The k largest values of each row, equal ones by lower index: (values, indices).

    A float's bits, read as an integer that grows with the value, are joined with the reversed
    index to one 64-bit key, so that no two keys of a row are equal."""
    vocab = z.shape[1]
    bits = (z + 0.0).view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).to(torch.int64) << 32
    key += torch.arange(vocab - 1, -1, -1, device=z.device)
    idx = (vocab - 1) - (key.topk(k, 1).values & 0xFFFFFFFF)
    return z.gather(1, idx), idx


def _plain_row(z, scale):
    """(maximum, scaled distance to it, its exponential, log-sum) of each row.  The maximum's own
    term is left out of the sum and comes back in log1p: the log-sum of a row that is almost sure
    of one token is small, and would be lost next to 1 in 32 bits."""
    m, at = z.max(1, keepdim=True)
    d = (z - m) * scale
    e = d.exp()
    logsum = e.scatter(1, at, 0.0).sum(1, keepdim=True).log1p()
    return m, d, e, logsum


def _plain_logprobs(st):
    z, scale, ids, k = st["logits"].float(), st["scale"], st["ids"], st["k"]
    m, d, e, logsum = _plain_row(z, scale)
    weighted = torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True)
    entropy = logsum - weighted * (-logsum).exp()
    at = d.gather(1, ids.clamp_min(0)[:, None]) - logsum
    logprob = torch.where(ids >= 0, at[:, 0], 0.0)
    top, idx = _plain_top(z, k)
    top_logprobs = (top - m) * scale - logsum
    top_ids = torch.where(top > -math.inf, idx, -1).to(torch.int32)
    return logprob, entropy[:, 0], torch.cat([m, logsum], 1), top_ids, top_logprobs


def _plain_logprobs_grad(st):
    z, scale = st["logits"].float(), st["scale"]
    ids, g = st["ids"][:, None], st["dlogprob"][:, None]
    logp = (z - st["stats"][:, :1]) * scale - st["stats"][:, 1:]
    p = logp.exp()
    g = torch.where(ids >= 0, g, 0.0)
    grad = p * -g
    at = ids.clamp_min(0)
    own_entry = -g * logp.gather(1, at).expm1()            # g (1 - p), also where p is near 1
    if "dentropy" in st:
        slope = torch.where(p > 0, logp + st["entropy"][:, None], 0.0)
        slope = p * slope * st["dentropy"][:, None]
        grad -= slope
        own_entry -= slope.gather(1, at)
    grad.scatter_(1, at, own_entry)
    return (grad * scale).to(st["logits"].dtype)


def _plain_teacher(st):
    """(valid, index, q, log q, mass outside) of the teacher's places, in 64 bits: the mass
    outside a list is what is left of 1.  A list's tokens are distinct; empty places come after
    them and repeat the first one's index."""
    ids, y = st["teacher_ids"], st["teacher_values"].double()
    valid = ids >= 0
    idx = torch.where(valid, ids, ids[:, :1]).clamp_min(0).long()
    y = torch.where(valid, y, -math.inf)
    if st["tail"]:
        logq = y
    else:
        y = y * st["scale"]
        y = y - y[:, :1].clamp_min(-1e300)
        logq = y - y.exp().sum(1, keepdim=True).clamp_min(1e-300).log()
    q = logq.exp()
    rest = (1 - q.sum(1, keepdim=True)).clamp_min(0) if st["tail"] else torch.zeros_like(q[:, :1])
    return valid, idx, q, logq, rest


def _plain_distill(st):
    z, scale = st["logits"].float(), st["scale"]
    valid, idx, q, logq, rest = _plain_teacher(st)
    m, d, e, logsum = _plain_row(z, scale)
    logp = d.gather(1, idx).double() - logsum
    loss = torch.where(q > 0, q * (logq - logp), 0.0).sum(1)
    if st["tail"]:
        zt = z.scatter(1, idx, -math.inf)
        mt, _, _, lt = _plain_row(zt, scale)
        outside = (mt - m).double() * scale + lt - logsum
        loss = loss + torch.where(rest > 0, rest * (rest.log() - outside), 0.0)[:, 0]
        stats = torch.cat([m, logsum, mt, lt], 1)
    else:
        stats = torch.cat([m, logsum, torch.zeros_like(m), torch.zeros_like(m)], 1)
    some = valid[:, :1]
    return torch.where(some[:, 0], loss, 0.0).float(), torch.where(some, stats, 0.0)


def _plain_distill_grad(st, stats):
    z, scale = st["logits"].float(), st["scale"]
    valid, idx, q, logq, rest = _plain_teacher(st)
    mass = q.sum(1, keepdim=True) + rest
    logp = (z - stats[:, 0:1]) * scale - stats[:, 1:2]
    grad = logp.exp() * mass.float()
    if st["tail"]:
        grad -= ((z - stats[:, 2:3]) * scale - stats[:, 3:4]).exp() * rest.float()
    listed_entries = logp.gather(1, idx).double().exp() * mass - q
    listed_entries = torch.where(valid, listed_entries, listed_entries[:, :1])
    grad.scatter_(1, idx, listed_entries.float())
    factor = torch.where(valid[:, :1], st["dloss"][:, None] * scale, 0.0)
    return torch.where(factor != 0, grad * factor, 0.0).to(st["logits"].dtype)


# ----------------------------------------------------------------------------------- one pass

def run(state):
    st, op = state, state["op"]
    if not own:
        if op == "logprobs":
            return _plain_logprobs(st)
        if op == "logprobs_grad":
            return _plain_logprobs_grad(st)
        if op == "distill":
            return _plain_distill(st)
        if op == "distill_grad":
            return _plain_distill_grad(st, st["stats"])
        loss, stats = _plain_distill(st)
        return loss, stats, _plain_distill_grad(st, stats)
    F, scale, ws = st["F"], st["scale"], st["workspace"]
    if op == "logprobs":
        F.token_logprobs(st["logits"], st["ids"], logprob=st["logprob"], entropy=st["entropy"],
                         stats=st["stats"], top_ids=st["top_ids"],
                         top_logprobs=st["top_logprobs"], scale=scale, workspace=ws)
        return st["logprob"], st["entropy"], st["stats"], st["top_ids"], st["top_logprobs"]
    if op == "logprobs_grad":
        F.token_logprobs_grad(st["logits"], st["ids"], st["stats"], st["dlogits"],
                              dlogprob=st["dlogprob"], entropy=st.get("entropy"),
                              dentropy=st.get("dentropy"), scale=scale)
        return st["dlogits"]
    teacher = (st["teacher_ids"], st["teacher_values"])
    if op == "distill":
        F.distill_topk(st["logits"], *teacher, loss=st["loss"], stats=st["stats"],
                       tail=st["tail"], scale=scale, workspace=ws)
        return st["loss"], st["stats"]
    if op == "distill_grad":
        F.distill_topk_grad(st["logits"], *teacher, stats=st["stats"], dloss=st["dloss"],
                            dlogits=st["dlogits"], tail=st["tail"], scale=scale)
        return st["dlogits"]
    F.distill_topk_loss_grad(st["logits"], *teacher, dloss=st["dloss"], loss=st["loss"],
                             stats=st["stats"], dlogits=st["dlogits"], tail=st["tail"],
                             scale=scale, workspace=ws)
    return st["loss"], st["stats"], st["dlogits"]


# ------------------------------------------------------------------------------ in 64 bits

def _exact_top(z, k):
    """Indices of the k largest of each row of z (float64), equal ones by lower index."""
    least = torch.topk(z, k, 1).values[:, -1:]
    above, level = z > least, z == least
    room = k - above.sum(1, keepdim=True)
    chosen = above | (level & (level.cumsum(1) <= room))
    idx = chosen.nonzero()[:, 1].view(z.shape[0], k)          # by rising index
    order = torch.sort(z.gather(1, idx), dim=1, descending=True, stable=True).indices
    return idx.gather(1, order)


def _exact_rows(case, st, lo, hi):
    z, scale, op = st["logits"][lo:hi].double(), case["scale"], case["op"]
    n = z.shape[0]
    peak = z.max(1, keepdim=True).values
    logsum = torch.logsumexp((z - peak) * scale, 1, keepdim=True)
    logp = (z - peak) * scale - logsum
    p = logp.exp()
    if op.startswith("logprobs"):
        ids = st["ids"][lo:hi]
        has = ids >= 0
        each = torch.arange(n, device=z.device)
        entropy = -torch.special.xlogy(p, p).sum(1)
        if op == "logprobs":
            logprob = torch.where(has, logp[each, ids * has], 0.0)
            out = [logprob, entropy, torch.cat([peak, logsum], 1)]
            k = case["k"]
            if k:
                idx = _exact_top(z, k)
                real = z.gather(1, idx) > -math.inf
                out += [torch.where(real, idx, -1).to(torch.int32), logp.gather(1, idx)]
            else:
                out += [torch.empty(n, 0, dtype=torch.int32, device=z.device),
                        torch.empty(n, 0, dtype=torch.float64, device=z.device)]
            return out
        g = st["dlogprob"][lo:hi].double() * has
        grad = -g[:, None] * p
        grad[each, ids * has] += g
        if case["entropy"]:
            h = st["dentropy"][lo:hi].double()[:, None]
            grad -= h * (torch.special.xlogy(p, p) + p * entropy[:, None])
        return [grad * scale]
    ids, y = st["teacher_ids"][lo:hi].long(), st["teacher_values"][lo:hi].double()
    valid = ids >= 0
    some = valid.any(1, keepdim=True)
    row, place = valid.nonzero(as_tuple=True)
    inside = torch.zeros_like(z, dtype=torch.bool)
    inside[row, ids[row, place]] = True
    y = torch.where(valid, y, -math.inf)
    q = y.exp() if case["tail"] else torch.nan_to_num(torch.softmax(y * scale, 1), nan=0.0)
    dense = torch.zeros_like(z)
    dense[row, ids[row, place]] = q[row, place]
    rest = (1 - q.sum(1, keepdim=True)).clamp_min(0) if case["tail"] else torch.zeros_like(peak)
    zt = torch.where(inside, -math.inf, z)
    peak_t = zt.max(1, keepdim=True).values
    logsum_t = torch.logsumexp((zt - peak_t) * scale, 1, keepdim=True)
    outside = (peak_t - peak) * scale + logsum_t - logsum
    loss = (torch.special.xlogy(dense, dense) - dense * logp).sum(1)
    stats = torch.cat([peak, logsum, torch.zeros_like(peak), torch.zeros_like(peak)], 1)
    mass = q.sum(1, keepdim=True) + rest
    grad = p * mass - dense
    if case["tail"]:
        loss += (torch.special.xlogy(rest, rest) - rest * outside)[:, 0]
        stats[:, 2:3], stats[:, 3:4] = peak_t, logsum_t
        grad -= rest * ((zt - peak_t) * scale - logsum_t).exp()
    loss, stats = loss * some[:, 0], stats * some
    grad = grad * (st["dloss"][lo:hi].double()[:, None] * scale * some)
    if op == "distill":
        return [loss, stats]
    if op == "distill_grad":
        return [grad]
    return [loss, stats, grad]


def exact(case, seed):
    st = prepare(case, seed)
    step = max(1, (1 << 26) // case["vocab"])
    parts = [_exact_rows(case, st, lo, min(lo + step, case["rows"]))
             for lo in range(0, case["rows"], step)]
    out = [torch.cat(cols) for cols in zip(*parts)]
    return out[0] if len(out) == 1 else tuple(out)
