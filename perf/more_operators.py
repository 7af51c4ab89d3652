"""Measured cases of the token path's two ends: embedding, and policy and preference losses.

Five kinds of pass:

  lookup        rows of an embedding table for given tokens, scaled
  embed_grad    the table's gradient: rows of equal tokens added up, set or added to a table
  policy        clipped policy loss with a KL term over log probabilities, and its gradients
  preference    loss over pairs of packed sequences, and its gradient
  policy_step   the policy loss straight over logits [rows, vocab], with the logits' gradient

With `own` false, run() computes a pass in elementary torch operations; with `own` true it calls
the framework.  Both take the same state, made by prepare() from a seed.
"""

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_NO_TOKEN = -100          # a position without a token: a prompt or padding position


def _embed(name, op, dtype, out, tokens, vocab, dim, scale=1.0, ignored=0.0, pad=0,
           accumulate=False):
    return dict(name=name, op=op, dtype=dtype, out=out, tokens=tokens, vocab=vocab, dim=dim,
                scale=scale, ignored=ignored, pad=pad, accumulate=accumulate)


def _policy(name, tokens, sequences=0, ignored=0.0, low=0.2, high=0.2, dual=0.0, kl=0.0,
            entropy=0.0):
    return dict(name=name, op="policy", tokens=tokens, sequences=sequences, ignored=ignored,
                low=low, high=high, dual=dual, kl=kl, entropy=entropy)


def _preference(name, pairs, tokens, kind="logistic", beta=0.1, margin=0.0, smoothing=0.0,
                normalised=False, reference=True, prompt=0.0):
    return dict(name=name, op="preference", pairs=pairs, tokens=tokens, kind=kind, beta=beta,
                margin=margin, smoothing=smoothing, normalised=normalised, reference=reference,
                prompt=prompt)


def _step(name, dtype, rows, vocab, scale=1.0, pad=0, ignored=0.0, low=0.2, high=0.2, dual=0.0,
          kl=0.0, entropy=0.0):
    return dict(name=name, op="policy_step", dtype=dtype, rows=rows, vocab=vocab, scale=scale,
                pad=pad, ignored=ignored, low=low, high=high, dual=dual, kl=kl, entropy=entropy)


def listed():
    return [
        # One new token of one sequence: the smallest lookup, where latency counts.
        _embed("lookup_next_token", "lookup", "bf16", "bf16", 1, 32000, 4096, scale=64.0),
        # The tokens of a training micro-batch in a wide model.
        _embed("lookup_batch", "lookup", "bf16", "bf16", 16384, 32000, 8192, scale=8192 ** 0.5),
        # A micro-batch's contribution to the flat gradient: every row of the table is written.
        _embed("embed_grad_set", "embed_grad", "bf16", "bf16", 16384, 32000, 4096,
               scale=64.0, ignored=0.05),
        # The next micro-batch, larger and in a wide model, added to a gradient kept in 32 bits.
        _embed("embed_grad_add", "embed_grad", "bf16", "fp32", 65536, 32000, 8192,
               accumulate=True),
        # One short sequence in 32 bits, odd sizes, a fifth of the positions without a token.
        _embed("embed_grad_odd", "embed_grad", "fp32", "fp32", 1021, 50021, 771, ignored=0.2,
               pad=5),
        # One rollout's tokens, clipped with a KL term to the reference policy.
        _policy("policy_rollout", 733, ignored=0.2, kl=0.05),
        # A packed batch of rollouts with one ratio for each sequence, KL and entropy terms.
        _policy("policy_sequences", 1000003, sequences=1024, ignored=0.25, low=0.01, high=0.015,
                kl=0.02, entropy=0.001),
        # A few pairs of short answers.
        _preference("preference_few", 4, 2311, prompt=0.3),
        # A large packed batch of pairs, half of it prompts, with smoothed labels.
        _preference("preference_batch", 512, 2000003, beta=0.2, smoothing=0.1, prompt=0.5),
        # A policy update's step over logits: loss and gradient together, a tenth of the
        # positions prompts.
        _step("policy_step", "bf16", 8192, 32000, ignored=0.1, kl=0.05),
        # An odd vocabulary in rows that start at any 2-byte phase, with an entropy bonus.
        _step("policy_step_odd", "fp16", 1021, 50021, scale=1 / 0.7, pad=3, ignored=0.25,
              low=0.2, high=0.28, dual=3.0, entropy=0.01),
        # A few positions of a large vocabulary in 32 bits.
        _step("policy_step_few", "fp32", 64, 131072, kl=0.1, entropy=0.001),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lookup", "embed_grad", "embed_grad", "policy", "preference", "policy_step"])
    ignored = rng.choice([0.0, rng.uniform(0.0, 0.5)])
    clip = dict(low=rng.choice([0.2, 0.1, 0.3]), high=rng.choice([0.2, 0.28, 0.4]),
                dual=rng.choice([0.0, 0.0, 3.0]), kl=rng.choice([0.0, 0.05, rng.uniform(0, 0.5)]),
                entropy=rng.choice([0.0, 0.0, 0.001, 0.01]))
    if op in ("lookup", "embed_grad"):
        vocab, dim = _log_uniform(rng, 1000, 131072), _log_uniform(rng, 64, 8192)
        dim = min(dim, (1 << 28) // vocab)
        if rng.random() < 0.6:
            dim = max(8, dim // 8 * 8)
        tokens = _log_uniform(rng, 1, min(65536, (1 << 27) // dim))
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        out = dtype if rng.random() < 0.6 else "fp32"
        accumulate = op == "embed_grad" and out == "fp32" and rng.random() < 0.5
        return dict(op=op, dtype=dtype, out=out, tokens=tokens, vocab=vocab, dim=dim,
                    scale=rng.choice([1.0, dim ** 0.5, rng.uniform(0.1, 4.0)]), ignored=ignored,
                    pad=rng.choice([0, 0, rng.randint(1, 64)]), accumulate=accumulate)
    if op == "policy":
        tokens = _log_uniform(rng, 1, 1 << 20)
        sequences = rng.choice([0, _log_uniform(rng, 1, min(tokens, 4096))])
        if sequences:
            clip.update(low=rng.uniform(0.005, 0.05), high=rng.uniform(0.005, 0.05))
        return dict(op=op, tokens=tokens, sequences=sequences, ignored=ignored, **clip)
    if op == "preference":
        pairs = _log_uniform(rng, 1, 1024)
        return dict(op=op, pairs=pairs, tokens=_log_uniform(rng, 8 * pairs, 1 << 21),
                    kind=rng.choice(["logistic", "logistic", "hinge", "squared"]),
                    beta=rng.choice([0.1, 0.5, 2.0]), margin=rng.choice([0.0, 0.0, 0.5]),
                    smoothing=rng.choice([0.0, 0.1]), normalised=rng.random() < 0.4,
                    reference=rng.random() < 0.7, prompt=rng.choice([0.0, rng.uniform(0, 0.6)]))
    vocab = _log_uniform(rng, 1000, 131072)
    rows = _log_uniform(rng, 1, min(8192, (1 << 28) // vocab))
    return dict(op=op, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), rows=rows, vocab=vocab,
                scale=rng.choice([1.0, 1.0, 0.5, 1 / 0.7]),
                pad=rng.choice([0, 0, rng.randint(1, 64)]), ignored=ignored, **clip)


def _distinct(case):
    """Rows of the table that prepare()'s tokens are expected to name."""
    i = torch.arange(1, case["vocab"] + 1, dtype=torch.float64)
    p = torch.log1p(1 / i) / math.log(case["vocab"] + 1)
    kept = case["tokens"] * (1 - case["ignored"])
    return float((1 - torch.exp(kept * torch.log1p(-p))).sum())


def work(case):
    op = case["op"]
    if op in ("lookup", "embed_grad"):
        t, d = case["tokens"], case["dim"]
        e, eo = _DTYPES[case["dtype"]].itemsize, _DTYPES[case["out"]].itemsize
        if op == "lookup":
            return {"bytes": 8 * t + d * (_distinct(case) * e + t * eo), "flops": t * d}
        kept = t * (1 - case["ignored"])
        written = 2 * _distinct(case) if case["accumulate"] else case["vocab"]
        return {"bytes": 8 * t + d * (kept * e + written * eo), "flops": kept * d}
    if op == "policy":
        t = case["tokens"]
        arrays = 4 + 2 + (case["kl"] > 0) + 2 * (case["entropy"] > 0)
        return {"bytes": 4 * arrays * t + 8 * (case["sequences"] + 1) + 32, "flops": 40 * t}
    if op == "preference":
        t, b = case["tokens"], case["pairs"]
        return {"bytes": 4 * (3 + case["reference"]) * t + 16 * b + 16 * b, "flops": 5 * t}
    r, v = case["rows"], case["vocab"]
    kept = r * (1 - case["ignored"])
    arrays = 8 + 3 * 4 + 4 * (case["kl"] > 0) + 8 + 4 * (case["entropy"] > 0)
    return {"bytes": (kept + r) * v * _DTYPES[case["dtype"]].itemsize + r * arrays,
            "flops": 9 * kept * v}


# ------------------------------------------------------------------------------------- inputs

def _strided(rows, cols, pad, dtype):
    """A [rows, cols] matrix whose rows are cols + pad elements apart."""
    return torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")[:, :cols]


def _prepare_embed(case, dev):
    tokens, vocab, dim = case["tokens"], case["vocab"], case["dim"]
    dtype, out = _DTYPES[case["dtype"]], _DTYPES[case["out"]]
    # Tokens as a text has them: the i-th most frequent one with a share of about 1 / i.
    rank = torch.exp(torch.rand(tokens, dtype=torch.float64, **dev) * math.log(vocab + 1)) - 1
    ids = torch.randperm(vocab, **dev)[rank.long().clamp_(0, vocab - 1)]
    ids[torch.rand(tokens, **dev) < case["ignored"]] = _NO_TOKEN
    st = dict(op=case["op"], ids=ids, scale=case["scale"], accumulate=case["accumulate"])
    if case["op"] == "lookup":
        st["table"] = _strided(vocab, dim, case["pad"], dtype)
        st["table"].copy_(torch.randn(vocab, dim, **dev).mul_(0.02))
        st["result"] = _strided(tokens, dim, case["pad"], out)
        return st
    st["dout"] = _strided(tokens, dim, case["pad"], dtype)
    st["dout"].copy_(torch.randn(tokens, dim, **dev).mul_(1e-3))
    st["dtable"] = _strided(vocab, dim, case["pad"], out)
    if case["accumulate"]:
        st["dtable"].copy_(torch.randn(vocab, dim, **dev).mul_(1e-3))
    return st


def _apart_from_borders(delta, case):
    """Log ratios moved off the clipping borders by 1e-3 where they are nearer than 5e-4: right
    at a border the gradient jumps, and there the last bit of a log probability decides."""
    borders = [math.log1p(case["high"]), math.log1p(-case["low"])]
    borders += [math.log(case["dual"])] if case["dual"] else []
    for b in borders:
        delta = torch.where((delta - b).abs() < 5e-4, delta + 1e-3, delta)
    return delta


def _prepare_policy(case, dev):
    tokens, sequences = case["tokens"], case["sequences"]
    f32 = dict(dtype=torch.float32, device="cuda")
    logprob = torch.rand(tokens, **dev).clamp_min_(1e-6).log_().mul_(1.5)
    # The policy that sampled the tokens is a few updates older.  Noise of a token, and a drift
    # of its whole sequence where one ratio counts for the sequence.
    old = logprob - torch.randn(tokens, **dev) * 0.15
    st = dict(op="policy", logprob=logprob, case=case)
    if sequences:
        # Packed sequences of uneven length, 2 % of the batch behind the last one.
        end = max(1, tokens - tokens // 50)
        cuts = torch.randint(0, end + 1, (sequences + 1,), **dev).sort().values
        cuts[0], cuts[-1] = 0, end
        at = torch.searchsorted(cuts, torch.arange(tokens, device="cuda"), right=True) - 1
        at = at.clamp_(0, sequences - 1)
        old = old + (torch.randn(sequences, **dev) * 0.02)[at]
        st["offsets"] = cuts
        st["advantage"] = torch.randn(sequences, **dev)[at]
    else:
        old = logprob - _apart_from_borders(logprob - old, case)
        st["advantage"] = torch.randn(tokens, **dev)
    weight = (torch.rand(tokens, **dev) >= case["ignored"]).float()
    st["weight"] = weight / weight.sum().clamp_min(1)
    st["old"] = old
    if case["kl"]:
        st["ref"] = logprob - torch.randn(tokens, **dev) * 0.2
    if case["entropy"]:
        st["entropy"] = torch.rand(tokens, **dev) * 4
        st["dentropy"] = torch.zeros(tokens, **f32)
    st.update(loss=torch.zeros(tokens, **f32), dlogprob=torch.zeros(tokens, **f32),
              totals=torch.zeros(4, **f32),
              counts=torch.zeros(2, dtype=torch.int64, device="cuda"))
    return st


def _prepare_preference(case, dev):
    tokens, pairs = case["tokens"], case["pairs"]
    f32 = dict(dtype=torch.float32, device="cuda")
    cuts = torch.randint(0, tokens + 1, (2 * pairs + 1,), **dev).sort().values
    cuts[0], cuts[-1] = 0, tokens
    logprob = torch.rand(tokens, **dev).clamp_min_(1e-6).log_().mul_(1.5)
    st = dict(op="preference", case=case, logprob=logprob, offsets=cuts)
    if case["reference"]:
        # The policy has moved by a little in each token, and away from or to each sequence.
        at = torch.searchsorted(cuts, torch.arange(tokens, device="cuda"), right=True) - 1
        at = at.clamp_(0, 2 * pairs - 1)
        length = (cuts[1:] - cuts[:-1]).clamp_min(1)
        drift = torch.randn(2 * pairs, **dev) * 4 / length
        st["ref"] = logprob - torch.randn(tokens, **dev) * 0.05 - drift[at]
    st["weight"] = (torch.rand(tokens, **dev) >= case["prompt"]).float()
    st["dloss"] = torch.full((pairs,), 1.0 / pairs, **f32)
    st.update(loss=torch.zeros(pairs, **f32), rewards=torch.zeros(pairs, 2, **f32),
              dlogprob=torch.zeros(tokens, **f32))
    return st


def _prepare_step(case, dev):
    rows, vocab, dtype, scale = case["rows"], case["vocab"], _DTYPES[case["dtype"]], case["scale"]
    # Logits as a language model gives them: a broad bulk and a few likely tokens in each row.
    x = torch.randn(rows, vocab, **dev).mul_(2.5)
    likely = torch.randint(0, vocab, (rows, 6), **dev)
    x.scatter_add_(1, likely, torch.rand(rows, 6, **dev).mul_(12).add_(2))
    logits = _strided(rows, vocab, case["pad"], dtype)
    logits.copy_(x)
    del x
    ids = torch.where(torch.rand(rows, **dev) < 0.8, likely[:, 0],
                      torch.randint(0, vocab, (rows,), **dev))
    logprob = torch.empty(rows, dtype=torch.float64, device="cuda")
    for i in range(0, rows, 512):
        z = torch.log_softmax(logits[i:i + 512].double() * scale, 1)
        logprob[i:i + 512] = z.gather(1, ids[i:i + 512, None])[:, 0]
    delta = _apart_from_borders(torch.randn(rows, **dev).double() * 0.2, case)
    st = dict(op="policy_step", case=case, logits=logits, scale=scale,
              old=(logprob - delta).float(), advantage=torch.randn(rows, **dev))
    if case["kl"]:
        st["ref"] = (logprob - torch.randn(rows, **dev).double() * 0.2).float()
    st["ids"] = ids.masked_fill(torch.rand(rows, **dev) < case["ignored"], _NO_TOKEN)
    f32 = dict(dtype=torch.float32, device="cuda")
    # A mean over the rows; gradients in fp16 are kept in range by a loss scale.
    st["weight"] = torch.full((rows,), 1.0 if dtype == torch.float16 else 1.0 / rows, **f32)
    st.update(loss=torch.zeros(rows, **f32), logprob=torch.zeros(rows, **f32),
              dlogits=_strided(rows, vocab, case["pad"], dtype))
    if case["entropy"]:
        st["entropy"] = torch.zeros(rows, **f32)
    return st


_PREPARE = dict(lookup=_prepare_embed, embed_grad=_prepare_embed, policy=_prepare_policy,
                preference=_prepare_preference, policy_step=_prepare_step)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 29)
    op = case["op"]
    state = _PREPARE[op](case, dict(generator=gen, device="cuda"))
    if own:
        import fsdp_sharded_optimizer_layout_amd as F
        need = 0
        if op == "embed_grad":
            need = F.embedding_grad_workspace_bytes(case["tokens"], case["vocab"], case["dim"])
        elif op == "policy":
            need = F.policy_loss_workspace_bytes(case["tokens"], case["sequences"])
        elif op == "preference":
            need = F.preference_loss_workspace_bytes(case["tokens"], case["pairs"])
        elif op == "policy_step":
            need = F.policy_logits_loss_grad_workspace_bytes(case["rows"], case["vocab"])
        state["workspace"] = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
        state["F"] = F
    return state


# --------------------------------------------------------------------------------- plain forms

def _plain_lookup(st):
    ids = st["ids"]
    rows = st["table"][ids.clamp_min(0)].float() * st["scale"]
    return torch.where(ids[:, None] >= 0, rows, 0.0).to(st["result"].dtype)


def _plain_embed_grad(st):
    ids, table = st["ids"], st["dtable"]
    # A row past the table takes the positions without a token.
    total = torch.zeros(table.shape[0] + 1, table.shape[1], device="cuda")
    total.index_add_(0, torch.where(ids >= 0, ids, table.shape[0]), st["dout"].float())
    total = total[:-1] * st["scale"]
    table.copy_(table + total if st["accumulate"] else total)
    return table


def _plain_policy_tokens(case, delta, logprob, st, entropy, mass=None):
    """(policy part, KL, loss, slope in the log probability, slope in the entropy, cut) of each
    token, each slope and the loss times the token's weight.  The log ratio comes in 64 bits, so
    that a token next to a clipping border falls on its side of it.  `mass`: the function that
    gives each token the sum of its sequence, and the sequence's share for one token."""
    a, w, beta, eta = st["advantage"], st["weight"], case["kl"], case["entropy"]
    high, low = math.log1p(case["high"]), math.log1p(-case["low"])
    dual = math.log(case["dual"]) if case["dual"] else math.inf
    cut = torch.where(a > 0, delta > high, (a < 0) & ((delta < low) | (delta > dual)))
    ratio = delta.exp().float()
    limited = torch.where(a > 0, ratio.clamp_max(1 + case["high"]),
                          ratio.clamp_min(1 - case["low"]))
    if case["dual"]:
        limited = torch.where(a < 0, limited.clamp_max(case["dual"]), limited)
    gain = a * limited
    flow = torch.where(cut, 0.0, a)
    if mass is None:
        slope = -w * flow * ratio
    else:
        total, share = mass((w * flow).double())
        slope = -(ratio.double() * total * share).float()
    kl = torch.zeros_like(gain)
    if beta:
        gap = st["ref"] - logprob
        kl = (gap.double().expm1() - gap.double()).float()      # tiny where the gap is small
        slope = slope - w * beta * gap.expm1()
    loss = beta * kl - gain
    if eta:
        loss = loss - eta * entropy
    return -gain, kl, w * loss, slope, -eta * w, cut


def _plain_policy(st):
    case, w, logprob = st["case"], st["weight"], st["logprob"]
    counted = w != 0
    delta = logprob.double() - st["old"].double()
    mass = None
    if "offsets" in st:
        cuts = st["offsets"]
        at = torch.searchsorted(cuts, torch.arange(w.numel(), device="cuda"), right=True) - 1
        inside = (at >= 0) & (at < cuts.numel() - 1)
        at = at.clamp(0, cuts.numel() - 2)
        counted = counted & inside

        def mass(x):
            run_ = torch.cat([torch.zeros_like(x[:1]),
                              torch.where(counted, x, 0.0).cumsum(0)])
            total = run_[cuts[1:]] - run_[cuts[:-1]]
            return total[at], share

        share = 1.0
        count = mass(torch.ones_like(delta))[0]
        share = 1 / count.clamp_min(1)
        total, share = mass(delta)
        delta = total * share
    part, kl, loss, slope, bonus, cut = _plain_policy_tokens(case, delta, logprob, st,
                                                             st.get("entropy"), mass)
    loss = torch.where(counted, loss, 0.0)
    slope = torch.where(counted, slope, 0.0)
    weighed = torch.where(counted, w, 0.0).double()
    h = st["entropy"].double() if "entropy" in st else torch.zeros_like(weighed)
    totals = torch.stack([loss.double().sum(), (weighed * part).sum(), (weighed * kl).sum(),
                          (weighed * h).sum()]).float()
    counts = torch.stack([counted.sum(), (counted & cut).sum()])
    out = [loss, slope, totals, counts]
    if "entropy" in st:
        out.append(torch.where(counted, bonus, 0.0))
    return tuple(out)


def _plain_preference(st):
    case, cuts, w = st["case"], st["offsets"], st["weight"]
    gap = st["logprob"].double()
    if "ref" in st:
        gap = gap - st["ref"].double()

    def sums(x):
        run_ = torch.cat([torch.zeros_like(x[:1]), x.cumsum(0)])
        return run_[cuts[1:]] - run_[cuts[:-1]]

    # Long sums, and the logistic loss of far margins, in 64 bits.
    mass = sums(w.double())
    total = sums(torch.where(w != 0, w * gap, 0.0))
    share = 1 / mass.clamp_min(1e-300) if case["normalised"] else torch.ones_like(mass)
    there = (sums((w != 0).double()) > 0).view(-1, 2).all(1)
    score = (total * share).view(-1, 2)
    lead, beta = score[:, 0] - score[:, 1], case["beta"]
    h = beta * lead - case["margin"]
    if case["kind"] == "logistic":
        loss = (-h.abs()).exp().log1p() + (-h).clamp_min(0) + case["smoothing"] * h
        slope = beta * (case["smoothing"] - 1 / (1 + h.exp()))
    elif case["kind"] == "hinge":
        loss, slope = (1 - h).clamp_min(0), torch.where(h < 1, -beta, 0.0)
    else:
        away = lead - case["margin"] - 1 / (2 * beta)
        loss, slope = away * away, 2 * away
    slope = torch.where(there, slope * st["dloss"], 0.0)
    factor = torch.stack([slope, -slope], 1).view(-1) * share
    at = torch.searchsorted(cuts, torch.arange(w.numel(), device="cuda"), right=True) - 1
    factor = factor.float()[at.clamp(0, cuts.numel() - 2)]
    return (torch.where(there, loss, 0.0).float(),
            torch.where(there[:, None], beta * score, 0.0).float(),
            torch.where(w != 0, factor * w, 0.0))


def _plain_step(st):
    case, z, scale, ids = st["case"], st["logits"].float(), st["scale"], st["ids"]
    m, top = z.max(1, keepdim=True)
    d = (z - m) * scale
    e = d.exp()
    # The maximum's own term comes back in log1p: a row almost sure of one token has a small
    # log-sum, which would be lost next to 1 in 32 bits.
    logsum = e.scatter(1, top, 0.0).sum(1, keepdim=True).log1p()
    logp = d - logsum
    p = logp.exp()
    at, has = ids.clamp_min(0)[:, None], ids >= 0
    logprob = logp.gather(1, at)[:, 0]
    entropy = -torch.where(p > 0, p * logp, 0.0).sum(1)
    delta = logprob.double() - st["old"].double()
    _, _, loss, slope, bonus, _ = _plain_policy_tokens(case, delta, logprob, st, entropy)
    g = torch.where(has, slope, 0.0)[:, None]
    grad = p * -g
    own_entry = -g * logp.gather(1, at).expm1()            # g (1 - p), also where p is near 1
    if case["entropy"]:
        h = torch.where(has, bonus, 0.0)[:, None]
        tilt = torch.where(p > 0, p * (logp + entropy[:, None]) * h, 0.0)
        grad -= tilt
        own_entry -= tilt.gather(1, at)
    grad.scatter_(1, at, own_entry)
    out = [torch.where(has, loss, 0.0), torch.where(has, logprob, 0.0),
           (grad * scale).to(st["logits"].dtype)]
    if case["entropy"]:
        out.append(torch.where(has, entropy, 0.0))
    return tuple(out)


_PLAIN = dict(lookup=_plain_lookup, embed_grad=_plain_embed_grad, policy=_plain_policy,
              preference=_plain_preference, policy_step=_plain_step)


# ----------------------------------------------------------------------------------- one pass

def run(state):
    st, op = state, state["op"]
    if not own:
        return _PLAIN[op](st)
    F, case = st["F"], st.get("case")
    if op == "lookup":
        F.embedding_lookup(st["table"], st["ids"], st["result"], scale=st["scale"])
        return st["result"]
    if op == "embed_grad":
        F.embedding_grad(st["ids"], st["dout"], st["dtable"], scale=st["scale"],
                         accumulate=st["accumulate"], workspace=st["workspace"])
        return st["dtable"]
    if op == "preference":
        F.preference_loss(st["logprob"], st["offsets"], st["loss"], rewards=st["rewards"],
                          ref_logprob=st.get("ref"), weight=st["weight"], dloss=st["dloss"],
                          dlogprob=st["dlogprob"], kind=case["kind"], beta=case["beta"],
                          margin=case["margin"], label_smoothing=case["smoothing"],
                          length_normalised=case["normalised"], workspace=st["workspace"])
        return st["loss"], st["rewards"], st["dlogprob"]
    terms = dict(old_logprob=st["old"], ref_logprob=st.get("ref"), clip_low=case["low"],
                 clip_high=case["high"], dual_clip=case["dual"], kl_coef=case["kl"],
                 entropy_coef=case["entropy"], entropy=st.get("entropy"),
                 workspace=st["workspace"])
    if op == "policy":
        F.policy_loss(st["logprob"], st["advantage"], st["weight"], st["dlogprob"],
                      loss=st["loss"], totals=st["totals"], counts=st["counts"],
                      dentropy=st.get("dentropy"), offsets=st.get("offsets"), **terms)
        out = [st["loss"], st["dlogprob"], st["totals"], st["counts"], st.get("dentropy")]
        return tuple(x for x in out if x is not None)
    F.policy_logits_loss_grad(st["logits"], st["ids"], st["advantage"], st["weight"], st["loss"],
                              st["dlogits"], logprob=st["logprob"], scale=st["scale"], **terms)
    out = [st["loss"], st["logprob"], st["dlogits"], st.get("entropy")]
    return tuple(x for x in out if x is not None)


# ------------------------------------------------------------------------------ in 64 bits

def _exact_embed(case, st):
    ids, scale = st["ids"], float(torch.tensor(case["scale"], dtype=torch.float32))
    has = ids >= 0
    if case["op"] == "lookup":
        out = torch.zeros(case["tokens"], case["dim"], dtype=torch.float64, device="cuda")
        out[has] = st["table"][ids[has]].double() * scale
        return out
    out = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device="cuda")
    order = torch.argsort(ids, stable=True)
    order = order[ids[order] >= 0]
    for part in order.split(8192):                 # bounded memory
        out.index_put_((ids[part],), st["dout"][part].double() * scale, accumulate=True)
    return st["dtable"].double() + out if case["accumulate"] else out


def _exact_terms(case, a, r, lp, ref, H):
    """Value and slopes of one token's loss, from its ratio."""
    lo, hi = 1 - case["low"], 1 + case["high"]
    value = torch.minimum(r * a, r.clamp(lo, hi) * a)
    flows = r * a <= r.clamp(lo, hi) * a
    if case["dual"]:
        floor = torch.where(a < 0, case["dual"] * a, -math.inf)
        flows = flows & (value >= floor)
        value = torch.maximum(value, floor)
    kl, klslope = torch.zeros_like(r), torch.zeros_like(r)
    if case["kl"]:
        kl, klslope = torch.expm1(ref - lp) - (ref - lp), -torch.expm1(ref - lp)
    total = -value + case["kl"] * kl - (case["entropy"] * H if case["entropy"] else 0)
    return value, kl, total, flows, klslope


def _wide(st, name):
    return st[name].double() if name in st else None


def _exact_policy(case, st):
    lp, old, a, w = (_wide(st, n) for n in ("logprob", "old", "advantage", "weight"))
    ref, H, n = _wide(st, "ref"), _wide(st, "entropy"), case["tokens"]
    keep = w != 0
    r = torch.exp(lp - old)
    if case["sequences"]:
        cuts = st["offsets"].tolist()
        seq = torch.full((n,), case["sequences"], dtype=torch.int64, device="cuda")
        lengths = torch.tensor([q - p for p, q in zip(cuts, cuts[1:])], device="cuda")
        seq[cuts[0]:cuts[-1]] = torch.repeat_interleave(
            torch.arange(case["sequences"], device="cuda"), lengths)
        keep = keep & (seq < case["sequences"])
        into = lambda x: torch.zeros(case["sequences"] + 1, dtype=torch.float64,
                                     device="cuda").index_add_(0, seq, x * keep)
        size = into(torch.ones_like(lp)).clamp_min(1)
        r = torch.exp(into(lp - old) / size)[seq]
    value, kl, total, flows, klslope = _exact_terms(case, a, r, lp, ref, H)
    if case["sequences"]:
        slope = -r / size[seq] * into(w * a * flows)[seq]
    else:
        slope = -w * r * a * flows
    slope = (slope + w * case["kl"] * klslope) * keep
    loss, w = w * total * keep, w * keep
    totals = torch.stack([loss.sum(), -(w * value).sum(), (w * kl).sum(),
                          (w * H).sum() if H is not None else loss.sum() * 0])
    counts = torch.stack([keep.sum(), (keep & ~flows).sum()])
    out = [loss, slope, totals, counts]
    return tuple(out + [-case["entropy"] * w] if case["entropy"] else out)


def _exact_preference(case, st):
    cuts, pairs = st["offsets"], case["pairs"]
    lengths = cuts[1:] - cuts[:-1]
    seq = torch.repeat_interleave(torch.arange(2 * pairs, device="cuda"), lengths)
    w = st["weight"].double()
    gap = st["logprob"].double() - (st["ref"].double() if "ref" in st else 0)
    into = lambda x: torch.zeros(2 * pairs, dtype=torch.float64,
                                 device="cuda").index_add_(0, seq, x)
    count, norm = into((w != 0).double()), torch.ones(2 * pairs, dtype=torch.float64,
                                                      device="cuda")
    if case["normalised"]:
        norm = into(w)
    score = torch.where(count > 0, into(w * gap) / norm, 0.0).requires_grad_()
    live = (count.view(pairs, 2) > 0).all(1)
    both = score.view(pairs, 2)
    lead = both[:, 0] - both[:, 1]
    h = case["beta"] * lead - case["margin"]
    if case["kind"] == "logistic":
        eps = case["smoothing"]
        sure = torch.nn.functional.logsigmoid
        loss = -(1 - eps) * sure(h) - eps * sure(-h)
    elif case["kind"] == "hinge":
        loss = torch.relu(1 - h)
    else:
        loss = (lead - case["margin"] - 1 / (2 * case["beta"])) ** 2
    loss = torch.where(live, loss, 0.0)
    slope, = torch.autograd.grad((loss * st["dloss"].double()).sum(), score)
    dlogprob = torch.where(w != 0, (slope / norm)[seq] * w, 0.0)
    rewards = case["beta"] * both * live[:, None]
    return loss.detach(), rewards.detach(), dlogprob


def _exact_step(case, st):
    out, step = [], max(1, (1 << 26) // case["vocab"])
    scale = float(torch.tensor(case["scale"], dtype=torch.float32))
    for lo in range(0, case["rows"], step):
        cut = {k: v[lo:lo + step] for k, v in st.items() if isinstance(v, torch.Tensor)}
        keep = cut["ids"] >= 0
        y, each = cut["ids"].clamp_min(0), torch.arange(keep.numel(), device="cuda")
        logp = torch.log_softmax(cut["logits"].double() * scale, 1)
        p = logp.exp()
        lp, H = logp[each, y], -torch.special.xlogy(p, p).sum(1)
        a, w, ref = _wide(cut, "advantage"), cut["weight"].double() * keep, _wide(cut, "ref")
        r = torch.exp(lp - cut["old"].double())
        _, _, total, flows, klslope = _exact_terms(case, a, r, lp, ref, H)
        g = w * (-r * a * flows + case["kl"] * klslope)
        grad = -g[:, None] * p
        grad[each, y] += g
        if case["entropy"]:
            grad += (case["entropy"] * w)[:, None] * (torch.special.xlogy(p, p) + p * H[:, None])
        part = [w * total, lp * keep, grad * scale]
        out.append(part + [H * keep] if case["entropy"] else part)
    return tuple(torch.cat(cols) for cols in zip(*out))


def exact(case, seed):
    st = prepare(case, seed)
    return {"lookup": _exact_embed, "embed_grad": _exact_embed, "policy": _exact_policy,
            "preference": _exact_preference, "policy_step": _exact_step}[case["op"]](case, st)
