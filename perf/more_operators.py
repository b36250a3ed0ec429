"""The workloads of the operators of a policy's update, in plain torch form and
through the library's entry points.

Four operators, in the order in which a trainer runs them on rollouts:

  logp        log-probabilities and entropies of the rollouts' tokens from
              logit rows, and their gradient in the logits (``token_logp``,
              ``token_logp_grad``);
  policy      the clipped policy loss with a divergence from a reference and
              an entropy bonus, and its gradient (``policy_loss``);
  preference  a loss of pairs of sequences, one preferred, and its gradient
              (``preference_loss``);
  clip        the norm of many gradients together, and their scaling to a
              largest norm (``clip_gradients``).
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # the log-probabilities of one interactive sequence's verified round: latency
        dict(name="logp_one_round", op="logp", n_seq=1, t_len=4, V=128256, dtype="bf16", T=1.0, entropy=False,
             grad=False, ragged=False),
        # the old policy's log-probabilities and entropies of a batch of rollouts, Qwen vocabulary
        dict(name="logp_rollouts_entropy", op="logp", n_seq=64, t_len=64, V=151936, dtype="bf16", T=1.0, entropy=True,
             grad=False, ragged=True),
        # a loss of the user's own: gradients from those of log-probabilities and entropies, odd vocabulary
        dict(name="logp_grad_f32_odd", op="logp", n_seq=16, t_len=32, V=50001, dtype="f32", T=0.8, entropy=True,
             grad=True, ragged=False),
        # a micro-batch of a policy that is updated while it decodes: latency
        dict(name="policy_micro_batch", op="policy", n_seq=2, t_len=8, V=128256, dtype="bf16", T=1.0, old=True,
             kl=0.0, entropy=0.0, dual=0.0, per_token=False, grad=True, ragged=False),
        # a training step's batch of rollouts of different lengths, with a divergence from the reference
        dict(name="policy_rollouts", op="policy", n_seq=64, t_len=64, V=151936, dtype="bf16", T=1.0, old=True,
             kl=0.04, entropy=0.0, dual=0.0, per_token=False, grad=True, ragged=True),
        # float32 rows of an odd vocabulary, advantages a token each, entropy bonus, both clips
        dict(name="policy_f32_entropy", op="policy", n_seq=16, t_len=32, V=100003, dtype="f32", T=0.8, old=True,
             kl=0.0, entropy=0.01, dual=3.0, per_token=True, grad=True, ragged=False),
        # one pair of short answers: latency
        dict(name="preference_one_pair", op="preference", n_pair=1, t_len=16, V=128256, dtype="bf16", T=1.0, beta=0.1,
             kind="sigmoid", smoothing=0.0, average=False, grad=True, ragged=False),
        # a batch of pairs of answers after their prompts, padded to one length
        dict(name="preference_batch", op="preference", n_pair=16, t_len=64, V=128256, dtype="bf16", T=1.0, beta=0.1,
             kind="sigmoid", smoothing=0.1, average=False, grad=True, ragged=True),
        # long answers in float32, log-probabilities averaged over each
        dict(name="preference_f32_long", op="preference", n_pair=2, t_len=500, V=50001, dtype="f32", T=1.0, beta=0.5,
             kind="ipo", smoothing=0.0, average=True, grad=True, ragged=True),
        # a drafter's few tensors, scaled into the optimizer's float32 buffers: latency
        dict(name="clip_drafter", op="clip", kind="drafter", layers=1, width=640, vocab=32000, dtype="bf16",
             share=0.25, out="f32"),
        # a policy's gradients, whose norm is within bounds: the norm alone has to be found
        dict(name="clip_policy_within", op="clip", kind="decoder", layers=16, width=2048, vocab=128256, dtype="bf16",
             share=4.0, out="place"),
        # matrices in bf16, norms and embeddings of odd sizes in float32, scaled copies
        dict(name="clip_mixed_odd", op="clip", kind="odd", layers=12, width=1531, vocab=50001, dtype="bf16", share=0.1,
             out="same"),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("logp", "policy", "preference", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "clip":
        kind = rng.choice(("drafter", "decoder", "odd"))
        return dict(op=op, kind=kind, layers=_spread(rng, 1, 16), width=_spread(rng, 64, 2048),
                    vocab=_spread(rng, 4000, 128256), dtype=dtype, share=rng.choice((0.1, 0.5, 4.0)),
                    out=rng.choice(("same", "f32")))
    V = _spread(rng, 4000, 160000)
    if rng.random() < 0.5:
        V -= V % 16
    most = int(3e8 * 2 / (2 if dtype == "bf16" else 4) / V)  # rows
    case = dict(op=op, V=V, dtype=dtype, T=rng.choice((0.6, 0.8, 1.0, 1.0, 1.3)), ragged=rng.random() < 0.5)
    if op == "preference":
        t_len = _spread(rng, 1, min(512, most // 2))
        kind = rng.choice(("sigmoid", "hinge", "ipo"))
        case.update(n_pair=_spread(rng, 1, max(1, most // (2 * t_len))), t_len=t_len, beta=rng.choice((0.05, 0.1, 0.5)),
                    kind=kind, smoothing=rng.choice((0.0, 0.1)) if kind == "sigmoid" else 0.0,
                    average=rng.random() < 0.3, grad=rng.random() < 0.8)
        return case
    t_len = _spread(rng, 1, 64)
    case.update(n_seq=_spread(rng, 1, max(1, most // t_len)), t_len=t_len)
    if op == "logp":
        case.update(entropy=rng.random() < 0.5, grad=rng.random() < 0.5)
    else:
        case.update(old=rng.random() < 0.8, kl=rng.choice((0.0, 0.04)), entropy=rng.choice((0.0, 0.0, 0.01)),
                    dual=rng.choice((0.0, 3.0)), per_token=rng.random() < 0.5, grad=rng.random() < 0.8)
    return case


CLIP_LOW, CLIP_HIGH = 0.2, 0.28

# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(shape, g, dtype, T):
    """Rows of a trained policy, half of them nearly sure of their token, and
    the tokens that it drew."""
    V = shape[-1]
    z = torch.empty(shape, dtype=dtype, device="cuda")
    tokens = torch.empty(shape[:-1], dtype=torch.int32, device="cuda")
    flat, said = z.view(-1, V), tokens.view(-1)
    for s in range(0, flat.shape[0], 512):
        n = min(512, flat.shape[0] - s)
        r = torch.randn(n, V, generator=g, device="cuda") * 2.0
        ids = torch.randint(0, V, (n, 20), generator=g, device="cuda")
        boost = torch.rand(n, 20, generator=g, device="cuda") * 10.0
        boost[:, 0] += (torch.rand(n, generator=g, device="cuda") < 0.5) * 14.0
        flat[s:s + n] = r.scatter_add_(1, ids, boost)
        noise = torch.rand(n, V, generator=g, device="cuda").clamp_(1e-20, 1.0)
        said[s:s + n] = (flat[s:s + n].float() / T - torch.log(-torch.log(noise).clamp_(min=1e-10))).argmax(1).to(torch.int32)
    return z, tokens


def _stats(z, tokens, T):
    """(logp, entropy, lse) of the rows in 64 bits."""
    V = z.shape[-1]
    flat, said = z.reshape(-1, V), tokens.reshape(-1).long().clamp(min=0)
    out = torch.empty(3, flat.shape[0], dtype=torch.float64, device=z.device)
    for a in range(0, flat.shape[0], 256):
        x = flat[a:a + 256].double() / T
        lse = torch.logsumexp(x, 1)
        lp = x - lse[:, None]
        out[0, a:a + 256] = lp.gather(1, said[a:a + 256, None])[:, 0]
        out[1, a:a + 256] = -torch.xlogy(lp.exp(), lp.exp()).sum(1)
        out[2, a:a + 256] = lse
    return out.view(3, *tokens.shape)


def _pad(tokens, ragged, prompt, g):
    """-1 where nothing is learnt: after each sequence's end, and on its prompt."""
    n, t = tokens.shape
    if ragged:
        at = torch.arange(t, device="cuda")
        end = torch.randint(1, t + 1, (n, 1), generator=g, device="cuda")
        tokens[at >= end] = -1
        if prompt:
            tokens[at < (end * torch.rand(n, 1, generator=g, device="cuda") * 0.4).long()] = -1
    return tokens


def _shapes(c):
    """The tensors of a model: (shape, float32 whatever the type)."""
    w, V, n = c["width"], c["vocab"], c["layers"]
    if c["kind"] == "drafter":  # one narrow layer and its head
        return [((w, w), False), ((4 * w, w), False), ((w, 4 * w), False), ((w,), False), ((V, w), False)]
    if c["kind"] == "decoder":
        one = [((w, w), False), ((w // 4, w), False), ((w // 4, w), False), ((w, w), False), ((4 * w, w), False),
               ((4 * w, w), False), ((w, 4 * w), False), ((w,), False), ((w,), False)]
        return [((V, w), False)] + one * n + [((w,), False)]
    one = [((w, w), False), ((w, 3 * w + 1), False), ((3 * w + 1, w), False), ((w,), True), ((1,), True)]
    return [((V, w), True)] + one * n


def _packed(c, wide, dtype):
    """One buffer for the tensors that are float32 anyway (`wide`) or not."""
    n = sum(math.prod(shape) for shape, w in _shapes(c) if w == wide)
    return torch.zeros(n, dtype=torch.float32 if wide else DTYPES[dtype], device="cuda")


def _views(c, flat):
    at, views = [0, 0], []
    for shape, wide in _shapes(c):
        n = math.prod(shape)
        views.append(flat[wide][at[wide]:at[wide] + n].view(shape))
        at[wide] += n
    return views


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c = case
    s = {"case": c}
    if c["op"] == "clip":
        s["flat"] = [_packed(c, wide, c["dtype"]) for wide in (False, True)]
        for flat in s["flat"]:  # the tensors lie end to end, as in a trainer's buckets
            for part in flat.split(1 << 26):
                part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * 1e-3)
        s["grads"] = _views(c, s["flat"])
        # a largest norm that is `share` of the gradients' own, to a few percent
        s["max_norm"] = c["share"] * 1e-3 * math.sqrt(sum(x.numel() for x in s["grads"]))
        s["out"], s["out_flat"] = None, s["flat"]
        if c["out"] != "place":
            s["out_flat"] = [_packed(c, wide, "f32" if c["out"] == "f32" else c["dtype"]) for wide in (False, True)]
            s["out"] = _views(c, s["out_flat"])
        return s
    n_seq = 2 * c["n_pair"] if c["op"] == "preference" else c["n_seq"]
    t_len, T = c["t_len"], c["T"]
    s["logits"], tokens = _rows((n_seq, t_len, c["V"]), g, DTYPES[c["dtype"]], T)
    s["tokens"] = _pad(tokens, c["ragged"], c["op"] == "preference", g)
    logp, entropy, lse = _stats(s["logits"], s["tokens"], T)
    noise = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    if c["op"] == "logp" and c["grad"]:
        s["logp"], s["lse"], s["entropy"] = logp.float(), lse.float(), entropy.float() if c["entropy"] else None
        s["d_logp"] = noise(n_seq, t_len)
        s["d_entropy"] = noise(n_seq, t_len) * 0.01 if c["entropy"] else None
    if c["op"] == "policy":
        s["advantages"] = noise(n_seq, t_len) if c["per_token"] else noise(n_seq)
        s["weights"] = torch.full((n_seq,), 1.0 / (n_seq * t_len), device="cuda")
        s["old"] = s["ref"] = None
        if c["old"]:
            old = (logp + noise(n_seq, t_len) * 0.15).float()
            ratio = torch.exp(logp - old.double())
            for edge in (1 - CLIP_LOW, 1 + CLIP_HIGH, c["dual"]):  # the gradient jumps there
                old = torch.where((ratio - edge).abs() < 1e-4, logp.float(), old)
            s["old"] = old
        if c["kl"]:
            s["ref"] = (logp + noise(n_seq, t_len) * 0.3).float()
    if c["op"] == "preference":
        have = s["tokens"] >= 0
        total = torch.where(have, logp, 0.0).sum(1)
        if c["average"]:
            total = total / have.sum(1).clamp(min=1)
        # the margin between a pair's sequences has moved from the reference's, one way or the other
        h = torch.sign(noise(c["n_pair"])) * (1 + 3 * torch.rand(c["n_pair"], generator=g, device="cuda"))
        h = h * (0.1 if c["average"] else 1.0)
        s["ref"] = (total + noise(n_seq)).float()
        s["ref"][0::2] = ((total[0::2] - total[1::2]) + s["ref"][1::2] - h).float()
        if c["kind"] == "hinge":  # the gradient jumps where beta h is 1
            h = (total[0::2] - total[1::2]) - (s["ref"][0::2].double() - s["ref"][1::2])
            s["ref"][0::2] += torch.where((h * c["beta"] - 1).abs() < 1e-3, 1.0, 0.0).float()
        s["weights"] = torch.full((c["n_pair"],), 1.0 / c["n_pair"], device="cuda")
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_71_gb300 as svp
        if c["op"] == "clip":
            norm = svp.clip_gradients(s["grads"], s["max_norm"], out=s["out"])
            return norm, s["out_flat"]
        if c["op"] == "logp":
            if c["grad"]:
                return svp.token_logp_grad(s["logits"], s["tokens"], s["logp"], s["lse"], s["d_logp"],
                                           entropy=s["entropy"], d_entropy=s["d_entropy"], temperature=c["T"])
            return svp.token_logp(s["logits"], s["tokens"], c["T"], entropy=c["entropy"])
        if c["op"] == "policy":
            return svp.policy_loss(s["logits"], s["tokens"], s["advantages"], s["weights"], old_logp=s["old"],
                                   ref_logp=s["ref"], temperature=c["T"], clip_low=CLIP_LOW, clip_high=CLIP_HIGH,
                                   dual_clip=c["dual"] or None, kl_coef=c["kl"], entropy_coef=c["entropy"],
                                   grad=c["grad"])
        return svp.preference_loss(s["logits"], s["tokens"], s["ref"], s["weights"], beta=c["beta"],
                                   temperature=c["T"], kind=c["kind"], smoothing=c["smoothing"],
                                   average=c["average"], grad=c["grad"])
    return {"clip": _clip, "logp": _logp, "policy": _policy, "preference": _preference}[c["op"]](s)


def _softmax(s):
    """Where a row has a token, the token's column, the rows' probabilities,
    their logarithms and the log-sum-exp, all in 32 bits, and the tokens'
    log-probabilities with the additions in 64."""
    have = s["tokens"] >= 0
    at = s["tokens"].long().clamp(min=0)[..., None]
    z = s["logits"].float() / s["case"]["T"]
    m = z.amax(-1, keepdim=True)
    lp = z - m
    log_sum = torch.log(torch.exp(lp).sum(-1, keepdim=True))
    lp = lp - log_sum
    logp = s["logits"].gather(-1, at).double() / s["case"]["T"] - m.double() - log_sum.double()
    return have, at, torch.exp(lp), lp, (m + log_sum)[..., 0], torch.where(have, logp[..., 0], 0.0)


def _gradient(s, have, at, p, g, lp=None, entropy=None, gh=None):
    """The gradient in the logits from those of the tokens' log-probabilities
    and of the entropies."""
    d = -p * g[..., None]
    d.scatter_add_(-1, at, g[..., None])
    if gh is not None:
        d = d - gh[..., None] * p * (lp + entropy[..., None])
    d = d / s["case"]["T"]
    return torch.where(have[..., None], d, 0.0).to(s["logits"].dtype)


def _logp(s):
    c = s["case"]
    have, at, p, lp, lse, logp = _softmax(s)
    if c["grad"]:
        return _gradient(s, have, at, p, s["d_logp"], lp, s["entropy"], s["d_entropy"])
    entropy = torch.where(have, -(p * lp).sum(-1), 0.0) if c["entropy"] else None
    return logp.float(), entropy, torch.where(have, lse, -math.inf)


def _policy(s):
    c = s["case"]
    have, at, p, lp, _, logp = _softmax(s)
    A = s["advantages"] if c["per_token"] else s["advantages"][:, None].expand_as(logp)
    r = torch.exp(logp - s["old"]) if c["old"] else torch.ones_like(logp)
    free, held = r * A, r.clamp(1 - CLIP_LOW, 1 + CLIP_HIGH) * A
    loss = -torch.minimum(free, held)
    slope = torch.where(free <= held, -free, 0.0)
    if c["dual"]:
        cut = (A < 0) & (loss > -c["dual"] * A)
        loss, slope = torch.where(cut, -c["dual"] * A, loss), torch.where(cut, 0.0, slope)
    if c["kl"]:
        d = s["ref"] - logp
        loss = loss + c["kl"] * (torch.expm1(d) - d)
        slope = slope - c["kl"] * torch.expm1(d)
    entropy = None
    if c["entropy"]:
        entropy = torch.where(have, -(p * lp).sum(-1), 0.0)
        loss = loss - c["entropy"] * entropy
    row_loss = torch.where(have, loss, 0.0).float()
    total = s["weights"] * row_loss.sum(1)
    grad = None
    if c["grad"]:
        w = s["weights"][:, None]
        grad = _gradient(s, have, at, p, (w * slope).float(), lp, entropy,
                         (-c["entropy"] * w).expand_as(logp) if c["entropy"] else None)
    return logp.float(), entropy, row_loss, total, grad


def _preference(s):
    c, w = s["case"], s["weights"]
    have, at, p, lp, _, logp = _softmax(s)
    total = logp.sum(1)  # in 64 bits: the margin is a difference of sums
    n = have.sum(1).clamp(min=1)
    if c["average"]:
        total = total / n
    h = (total[0::2] - total[1::2]) - (s["ref"][0::2].double() - s["ref"][1::2])
    margin = c["beta"] * h
    if c["kind"] == "sigmoid":
        e = c["smoothing"]
        soft = lambda x: torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))
        loss = (1 - e) * soft(-margin) + e * soft(margin)
        slope = c["beta"] * (e / (1 + torch.exp(-margin)) - (1 - e) / (1 + torch.exp(margin)))
    elif c["kind"] == "hinge":
        loss = torch.clamp(1 - margin, min=0)
        slope = torch.where(margin < 1, -c["beta"], 0.0).double()
    else:
        off = h - 1 / (2 * c["beta"])
        loss, slope = off * off, 2 * off
    grad = None
    if c["grad"]:
        g = torch.stack([w * slope, -w * slope], 1).view(-1)
        if c["average"]:
            g = g / n
        grad = _gradient(s, have, at, p, g.float()[:, None].expand_as(logp))
    return logp.float(), margin.float(), (w * loss).float(), grad


def _clip(s):
    total = torch.stack([x.float().square().sum() for x in s["grads"]]).double().sum()
    norm = torch.sqrt(total).float()
    scale = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    if s["out"] is None:
        for x in s["grads"]:
            x.copy_(x.float() * scale)
        return norm, s["flat"]
    for x, o in zip(s["grads"], s["out"]):
        o.copy_(x.float() * scale)
    return norm, s["out_flat"]


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    elt = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "clip":
        read = sum(math.prod(shape) * (4 if wide else elt) for shape, wide in _shapes(c))
        n = sum(math.prod(shape) for shape, _ in _shapes(c))
        if c["out"] == "place" and c["share"] > 1:  # nothing to scale
            return {"bytes": read, "flops": 2 * n}
        return {"bytes": read + (4 * n if c["out"] == "f32" else read), "flops": 3 * n}
    n_seq = 2 * c["n_pair"] if c["op"] == "preference" else c["n_seq"]
    every = n_seq * c["t_len"]
    rows = n_seq * (c["t_len"] + 1) / 2 if c["ragged"] else every
    if c["op"] == "preference" and c["ragged"]:
        rows *= 0.8  # prompts
    wide = bool(c.get("entropy"))
    # a scale, an exponential and a sum for each logit; a product more for the entropy, three for a gradient
    flops = rows * c["V"] * (3 + 2 * wide + (3 + wide if c["grad"] else 0))
    return {"bytes": rows * c["V"] * elt + (every * c["V"] * elt if c["grad"] else 0) + every * 24, "flops": flops}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a sequence at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "clip":
        norm = math.sqrt(math.fsum(float(v.double().square().sum()) for x in s["flat"] for v in x.split(1 << 24)))
        scale = min(1.0, s["max_norm"] / (norm + 1e-6))
        return torch.tensor(norm, dtype=torch.float64), [x.double() * scale for x in s["flat"]]
    logits, tokens, T = s["logits"], s["tokens"], c["T"]
    n_seq, t_len, V = logits.shape
    dev = logits.device
    logp, entropy = torch.zeros(n_seq, t_len, dtype=torch.float64, device=dev), torch.zeros(n_seq, t_len, dtype=torch.float64, device=dev)
    lse = torch.full((n_seq, t_len), -math.inf, dtype=torch.float64, device=dev)
    for b in range(n_seq):
        live = (tokens[b] >= 0).nonzero()[:, 0]
        for at in live.split(128):
            x = logits[b, at].double() / T
            lp = torch.log_softmax(x, 1)
            logp[b, at] = lp[torch.arange(len(at), device=dev), tokens[b, at].long()]
            entropy[b, at] = -(lp.exp() * lp).sum(1)
            lse[b, at] = torch.logsumexp(x, 1)
    gh = torch.zeros(n_seq, t_len, dtype=torch.float64, device=dev)
    if c["op"] == "logp":
        if not c["grad"]:
            return logp, entropy if c["entropy"] else None, lse
        result, g = (), s["d_logp"].double()
        if c["entropy"]:
            gh = s["d_entropy"].double()
    elif c["op"] == "policy":
        w = s["weights"].double()[:, None]
        A = s["advantages"].double()
        A = A if c["per_token"] else A[:, None].expand(n_seq, t_len)
        x = logp.clone().requires_grad_()
        r = torch.exp(x - s["old"].double()) if c["old"] else torch.exp(x - logp)
        a, b = r * A, torch.where(r < 1 - CLIP_LOW, 1 - CLIP_LOW, torch.where(r > 1 + CLIP_HIGH, 1 + CLIP_HIGH, r)) * A
        gain = torch.where(a <= b, a, b)
        if c["dual"]:
            gain = torch.where((A < 0) & (gain < c["dual"] * A), c["dual"] * A, gain)
        row = -gain
        if c["kl"]:
            d = s["ref"].double() - x
            row = row + c["kl"] * (torch.exp(d) - d - 1)
        row.sum().backward()
        g = w * x.grad
        row = row.detach() - c["entropy"] * entropy
        row = torch.where(tokens >= 0, row, 0.0)
        gh = (-c["entropy"] * w).expand(n_seq, t_len)
        result = (logp, entropy if c["entropy"] else None, row, s["weights"].double() * row.sum(1))
    else:
        n = (tokens >= 0).sum(1).clamp(min=1).double()
        total = (logp.sum(1) / (n if c["average"] else 1)).requires_grad_()
        ref = s["ref"].double()
        h = (total[0::2] - total[1::2]) - (ref[0::2] - ref[1::2])
        m = c["beta"] * h
        if c["kind"] == "sigmoid":
            loss = (1 - c["smoothing"]) * torch.logaddexp(-m, torch.zeros_like(m)) + c["smoothing"] * torch.logaddexp(m, torch.zeros_like(m))
        elif c["kind"] == "hinge":
            loss = torch.relu(1 - m)
        else:
            loss = (h - 0.5 / c["beta"]) ** 2
        loss = s["weights"].double() * loss
        loss.sum().backward()
        g = (total.grad / (n if c["average"] else 1))[:, None].expand(n_seq, t_len)
        result = (logp, m.detach(), loss.detach())
    grad = None
    if c["grad"]:
        grad = torch.zeros(n_seq, t_len, V, dtype=torch.float64, device=dev)
        for b in range(n_seq):
            for at in (tokens[b] >= 0).nonzero()[:, 0].split(128):
                lp = torch.log_softmax(logits[b, at].double() / T, 1)
                p = lp.exp()
                d = -p * g[b, at, None] - gh[b, at, None] * p * (lp + entropy[b, at, None])
                d[torch.arange(len(at), device=dev), tokens[b, at].long()] += g[b, at]
                grad[b, at] = d / T
    return grad if c["op"] == "logp" else (*result, grad)
