"""The workloads of the logit operators around verification, in plain torch
form and through the library's entry points.

Three operators, in the order in which a rollout system runs them:

  process   penalties for repeated tokens, biases and grammar masks on target
            or draft logits, row i of a sequence seeing its first i drafts
            (``process_logits``);
  top       a teacher row's K largest logits as log-probabilities, with their
            ids and the row's log-sum-exp (``kd_top``);
  loss      distillation of the drafter from such lists, with the gradient in
            the draft logits (``kd_top_loss``).
"""
import math

import torch

own = False

#: the tail's mass below which a list counts as complete: float32
#: log-probabilities cannot tell less
COMPLETE = 2.0 ** -20

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one interactive sequence, plain decoding: latency
        dict(name="process_decode_one", op="process", B=1, k=0, V=128256, dtype="bf16", H=1000, bias=16, mask=False,
             tight=0.0, inplace=False),
        # a rollout round with ragged drafts and the usual penalties, Llama-3 vocabulary
        dict(name="process_ragged_round", op="process", B=256, k=3, V=128256, dtype="bf16", H=4096, bias=0, mask=False,
             tight=0.0, inplace=False),
        # constrained decoding: a grammar's masks on the round's rows where they lie, Qwen vocabulary
        dict(name="process_grammar_in_place", op="process", B=32, k=3, V=151936, dtype="bf16", H=0, bias=0, mask=True,
             tight=0.5, inplace=True),
        # everything at once on float32 rows of an odd vocabulary, long drafts, long histories
        dict(name="process_all_f32_odd", op="process", B=48, k=7, V=100003, dtype="f32", H=16384, bias=300, mask=True,
             tight=0.3, inplace=False),
        # the teacher's list for one row: latency
        dict(name="top_one_row", op="top", n_seq=1, t_len=1, V=151936, dtype="bf16", K=20, T=1.0, ragged=False),
        # the lists of a verified round: the emitted rows of a ragged batch
        dict(name="top_ragged_round", op="top", n_seq=256, t_len=4, V=128256, dtype="bf16", K=64, T=1.0, ragged=True),
        # float32 teacher rows of an odd vocabulary, long lists, a low temperature
        dict(name="top_f32_long_lists", op="top", n_seq=24, t_len=16, V=50001, dtype="f32", K=256, T=0.6, ragged=False),
        # a micro-batch of a drafter kept up to date while decoding: latency
        dict(name="loss_micro_batch", op="loss", n_seq=2, t_len=8, V=128256, dtype="bf16", K=20, T=1.0, tail=True,
             grad=True, ragged=False),
        # a training step's batch of rollouts of different lengths, Qwen vocabulary
        dict(name="loss_rollouts", op="loss", n_seq=64, t_len=64, V=151936, dtype="bf16", K=64, T=1.0, tail=True,
             grad=True, ragged=True),
        # float32 rows of an odd vocabulary, lists scaled to sum to one
        dict(name="loss_f32_renormalised", op="loss", n_seq=16, t_len=32, V=50001, dtype="f32", K=128, T=0.8,
             tail=False, grad=True, ragged=False),
        # the loss of held-out rollouts, without a gradient
        dict(name="loss_only", op="loss", n_seq=32, t_len=32, V=128256, dtype="bf16", K=64, T=1.0, tail=True,
             grad=False, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("process", "top", "loss"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    V = _spread(rng, 4000, 160000)
    if rng.random() < 0.5:
        V -= V % 16
    most = int((3e8 if op == "loss" else 1.2e8) * 2 / (2 if dtype == "bf16" else 4) / V)  # rows
    if op == "process":
        k = rng.randint(0, 7)
        mask = rng.random() < 0.6
        return dict(op=op, B=_spread(rng, 1, max(1, min(512, most // (k + 1)))), k=k, V=V, dtype=dtype,
                    H=rng.choice((0, 1)) * _spread(rng, 16, 16384), bias=rng.choice((0, 1, 17, 300)), mask=mask,
                    tight=round(rng.uniform(0, 1), 2) if mask else 0.0, inplace=False)
    t_len = _spread(rng, 1, 32)
    case = dict(op=op, n_seq=_spread(rng, 1, max(1, most // t_len)), t_len=t_len, V=V, dtype=dtype,
                K=_spread(rng, 1, 256), T=rng.choice((0.6, 0.8, 1.0, 1.0, 1.3)), ragged=rng.random() < 0.5)
    if op == "loss":
        case.update(tail=rng.random() < 0.6, grad=rng.random() < 0.8)
    return case


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _logits(shape, g, dtype):
    """Rows with a few likely tokens on a broad floor, as language models' are."""
    V = shape[-1]
    z = torch.empty(shape, dtype=dtype, device="cuda")
    flat = z.view(-1, V)
    for s in range(0, flat.shape[0], 512):
        n = min(512, flat.shape[0] - s)
        r = torch.randn(n, V, generator=g, device="cuda") * 3.0
        ids = torch.randint(0, V, (n, 20), generator=g, device="cuda")
        r.scatter_add_(1, ids, torch.rand(n, 20, generator=g, device="cuda") * 8.0)
        flat[s:s + n] = r
    return z


def _tokens(shape, V, g):
    """Token ids of which the low ones come often, so that tokens repeat."""
    return (torch.rand(shape, generator=g, device="cuda") ** 4 * V).to(torch.int32).clamp_(max=V - 1)


def _lengths(n, most, g):
    return torch.randint(1, most + 1, (n,), generator=g, device="cuda").to(torch.int32)


def _mask(rows, V, tight, g):
    """Grammar masks [rows, ceil(V / 32)]: a share `tight` of the rows allows
    twenty tokens (a keyword, a bracket), the others all but one in a hundred
    (inside a string)."""
    W = (V + 31) // 32
    m = torch.empty(rows, W, dtype=torch.int32, device="cuda")
    bit = torch.arange(32, device="cuda")
    narrow = torch.rand(rows, generator=g, device="cuda") < tight
    for s in range(0, rows, 256):
        n = min(256, rows - s)
        allowed = torch.rand(n, W * 32, generator=g, device="cuda") >= 0.01
        few = torch.zeros(n, W * 32, dtype=torch.bool, device="cuda")
        few.scatter_(1, torch.randint(0, V, (n, 20), generator=g, device="cuda"), True)
        allowed = torch.where(narrow[s:s + n, None], few, allowed)
        words = (allowed.view(n, W, 32).to(torch.int64) << bit).sum(-1)
        m[s:s + n] = torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)
    return m


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    c, V, dtype = case, case["V"], DTYPES[case["dtype"]]
    s = {"case": c}
    if c["op"] == "process":
        B, k, H = c["B"], c["k"], c["H"]
        R = k + 1
        s["logits"] = _logits((B, R, V), g, dtype)
        s["out"] = s["logits"] if c["inplace"] else torch.zeros_like(s["logits"])
        s["draft_len"] = torch.randint(0, k + 1, (B,), generator=g, device="cuda").to(torch.int32)
        s["tokens"] = _tokens((B, k), V, g) if k else None
        for name in ("history", "prompt_len", "history_len", "repetition", "presence", "frequency", "bias_ids",
                     "bias_values", "mask"):
            s[name] = None
        if H:
            s["history"] = _tokens((B, H), V, g)
            s["history_len"] = _lengths(B, H, g)
            s["prompt_len"] = (s["history_len"] * torch.rand(B, generator=g, device="cuda") * 0.5).to(torch.int32)
        if H or (k and not c["inplace"]):
            s["repetition"] = 1.0 + torch.rand(B, generator=g, device="cuda") * 0.3
            s["presence"] = torch.rand(B, generator=g, device="cuda")
            s["frequency"] = torch.rand(B, generator=g, device="cuda") * 0.5
        if c["bias"]:
            s["bias_ids"] = _tokens((B, c["bias"]), V, g)
            s["bias_values"] = torch.randn(B, c["bias"], generator=g, device="cuda") * 4.0
        if c["mask"]:
            s["mask"] = _mask(B * R, V, c["tight"], g).view(B, R, -1)
        return s
    n_seq, t_len, K = c["n_seq"], c["t_len"], c["K"]
    rows = _lengths(n_seq, t_len, g) if c["ragged"] else None
    if c["op"] == "top":
        s["target"] = _logits((n_seq, t_len, V), g, dtype)
        s["n_rows"] = rows
        return s
    # the teacher's lists, as a rollout kept them, and the drafter's logits, not far from the teacher's
    teacher = _logits((n_seq, t_len, V), g, dtype)
    n = n_seq * t_len
    s["draft"] = torch.empty_like(teacher)
    s["ids"] = torch.empty(n, K, dtype=torch.int32, device="cuda")
    s["logp"] = torch.empty(n, K, dtype=torch.float32, device="cuda")
    flat, draft = teacher.view(n, V), s["draft"].view(n, V)
    for a in range(0, n, 512):
        z = flat[a:a + 512].float()
        draft[a:a + 512] = z + torch.randn(z.shape, generator=g, device="cuda") * 0.7
        z = z / c["T"]
        top = z.topk(min(K, V), dim=1)
        s["ids"][a:a + 512] = top.indices
        s["logp"][a:a + 512] = top.values - torch.logsumexp(z, 1, keepdim=True)
    s["ids"], s["logp"] = s["ids"].view(n_seq, t_len, K), s["logp"].view(n_seq, t_len, K)
    if rows is not None:  # positions after a rollout's end have no list
        gone = torch.arange(t_len, device="cuda") >= rows[:, None]
        s["ids"][gone] = -1
        s["logp"][gone] = -math.inf
    s["weights"] = torch.rand(n_seq, generator=g, device="cuda") * 2.0
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        import speculative_decoding_verification_71_gb300 as svp
        if c["op"] == "process":
            return svp.process_logits(s["logits"], history=s["history"], prompt_len=s["prompt_len"],
                                      history_len=s["history_len"], tokens=s["tokens"], draft_len=s["draft_len"],
                                      repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                                      bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"],
                                      out=s["out"])
        if c["op"] == "top":
            return svp.kd_top(s["target"], c["K"], c["T"], n_rows=s["n_rows"])
        return svp.kd_top_loss(s["ids"], s["logp"], s["draft"], s["weights"], c["T"], tail=c["tail"], grad=c["grad"])
    if c["op"] == "process":
        return _process(s)
    if c["op"] == "top":
        return _top(s)
    return _loss(s)


def _process(s):
    logits, out = s["logits"], s["out"]
    B, R, V = logits.shape
    dev = logits.device
    z = logits.float()
    row = torch.arange(R, device=dev)
    n = torch.zeros(B, R, V + 1, device=dev)  # one place more, for what does not count
    prompt = torch.zeros(B, V + 1, device=dev)
    if s["history"] is not None:
        at = torch.arange(s["history"].shape[1], device=dev)
        ids = s["history"].long()
        generated = (at >= s["prompt_len"][:, None]) & (at < s["history_len"][:, None])
        first = torch.zeros(B, V + 1, device=dev).scatter_add_(1, torch.where(generated, ids, V), torch.ones_like(ids, dtype=torch.float32))
        n += first[:, None]
        prompt.scatter_(1, torch.where(at < s["prompt_len"][:, None], ids, V), 1.0)
    if s["tokens"] is not None:
        k = s["tokens"].shape[1]
        earlier = torch.arange(k, device=dev) < row[:, None]
        ids = torch.where(earlier[None], s["tokens"].long()[:, None], V)
        n.scatter_add_(2, ids, torch.ones_like(ids, dtype=torch.float32))
    n = n[:, :, :V]
    if s["repetition"] is not None:
        r = s["repetition"][:, None, None]
        seen = (n > 0) | (prompt[:, None, :V] > 0)
        z = torch.where(seen, torch.where(z > 0, z / r, z * r), z)
        z = z - s["frequency"][:, None, None] * n - s["presence"][:, None, None] * (n > 0)
    if s["bias_ids"] is not None:  # the last entry of a token counts
        ids = s["bias_ids"].long()
        M = ids.shape[1]
        at = torch.arange(1, M + 1, device=dev).expand(B, M)
        last = torch.zeros(B, V, dtype=torch.int64, device=dev).scatter_reduce_(1, ids, at, "amax")
        value = torch.cat([torch.zeros(B, 1, device=dev), s["bias_values"]], 1).gather(1, last)
        z = z + value[:, None]
    if s["mask"] is not None:
        v = torch.arange(V, device=dev)
        z = torch.where((s["mask"][:, :, v >> 5] >> (v & 31).to(torch.int32)) & 1 == 1, z, -math.inf)
    live = (row < s["draft_len"][:, None] + 1)[:, :, None]
    out.copy_(torch.where(live, z.to(logits.dtype), out))
    return out


def _top(s):
    c, K = s["case"], s["case"]["K"]
    t = s["target"]
    n_seq, t_len, V = t.shape
    z = t.float() + 0.0  # -0 and 0 are one value
    bits = z.view(torch.int32)
    key = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long() * 2 ** 32 + (2 ** 32 - 1 - torch.arange(V, device=t.device))
    ids = key.topk(min(K, V), dim=2).indices
    z = z / c["T"]
    m = z.amax(2, keepdim=True)
    log_sum = torch.log(torch.exp(z - m).sum(2, keepdim=True))
    logp = z.gather(2, ids) - m - log_sum
    ids = torch.where(logp == -math.inf, -1, ids).to(torch.int32)
    lse = (m + log_sum)[:, :, 0]
    if s["n_rows"] is not None:
        gone = torch.arange(t_len, device=t.device) >= s["n_rows"][:, None]
        ids = torch.where(gone[:, :, None], -1, ids).to(torch.int32)
        logp = torch.where(gone[:, :, None], -math.inf, logp)
        lse = torch.where(gone, -math.inf, lse)
    return ids, logp, lse


def _loss(s):
    c = s["case"]
    draft, logp = s["draft"], s["logp"]
    used = s["ids"] >= 0
    ids = torch.where(used, s["ids"], 0).long()
    z = draft.float() / c["T"]
    z = z - z.amax(2, keepdim=True)
    e = torch.exp(z)
    total = e.sum(2, keepdim=True)
    logq = z.gather(2, ids) - torch.log(total)
    p = torch.where(used, torch.exp(logp), 0.0)
    P = p.sum(2, keepdim=True)
    listed_ = torch.zeros_like(z).scatter_add_(2, ids, used.float()) > 0
    rest = torch.where(listed_, 0.0, e).sum(2, keepdim=True) / total  # 1 - Q
    any_ = used.any(2, keepdim=True)
    if c["tail"]:
        r = torch.where(1 - P < COMPLETE, 0.0, 1 - P)
        kl = torch.where(p > 0, p * (logp - logq), 0.0).sum(2)
        kl = kl + torch.where(r > 0, r * (torch.log(r) - torch.log(rest)), 0.0)[:, :, 0]
        away = 1 - torch.where(rest > 0, r / rest, 0.0)
    else:
        p = torch.where(any_, p / P, 0.0)
        kl = torch.where(p > 0, p * (torch.log(p) - logq), 0.0).sum(2)
        away = torch.ones_like(P)
    kl = torch.where(any_[:, :, 0], kl, 0.0)
    loss = s["weights"] * kl.sum(1)
    if not c["grad"]:
        return kl, loss, None
    grad = (e / total) * torch.where(listed_, 1.0, away)
    grad = grad.scatter_add_(2, ids, torch.where(used, -p, 0.0))
    grad = torch.where(any_, grad * (s["weights"][:, None, None] / c["T"]), 0.0)
    return kl, loss, grad.to(draft.dtype)


# ---------------------------------------------------------------------------
# What a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c, V = case, case["V"]
    elt = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "process":
        rows = c["B"] * (c["k"] / 2 + 1)  # draft lengths are spread evenly over 0..k
        allowed = 1.0 if not c["mask"] else (1 - c["tight"]) * 0.99
        small = 4 * c["B"] * (c["H"] / 2 + c["k"] + 2 * c["bias"] + 6) + rows * (V / 8 if c["mask"] else 0)
        if c["inplace"]:  # what is masked is written, the rest stays
            return {"bytes": rows * V * elt * (1 - allowed) + small, "flops": rows * V}
        return {"bytes": rows * V * elt * (1 + allowed) + small, "flops": rows * V * (4 if c["H"] else 1)}
    all_rows = c["n_seq"] * c["t_len"]
    rows = c["n_seq"] * (c["t_len"] + 1) / 2 if c["ragged"] else all_rows
    small = all_rows * (8 * c["K"] + 8)
    if c["op"] == "top":  # a scale, an exponential, a sum and a comparison for each logit
        return {"bytes": rows * V * elt + small, "flops": rows * V * 4}
    return {"bytes": rows * V * elt + (all_rows * V * elt if c["grad"] else 0) + small,
            "flops": rows * V * (6 if c["grad"] else 3)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits, a sequence at a time
# ---------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"process": _exact_process, "top": _exact_top, "loss": _exact_loss}[case["op"]](s)


def _exact_process(s):
    logits = s["logits"]
    B, R, V = logits.shape
    out = s["out"].double()
    for b in range(B):
        generated = prompt = torch.zeros(0, dtype=torch.int64, device=logits.device)
        if s["history"] is not None:
            p, h = int(s["prompt_len"][b]), int(s["history_len"][b])
            prompt, generated = s["history"][b, :p].long(), s["history"][b, p:h].long()
        for i in range(int(s["draft_len"][b]) + 1):
            z = logits[b, i].double()
            said = generated if s["tokens"] is None else torch.cat([generated, s["tokens"][b, :i].long()])
            if s["repetition"] is not None:
                count = torch.bincount(said, minlength=V).double()
                again = torch.unique(torch.cat([prompt, said]))
                r = float(s["repetition"][b])
                z[again] = torch.where(z[again] > 0, z[again] / r, z[again] * r)
                z -= count * float(s["frequency"][b])
                z[torch.unique(said)] -= float(s["presence"][b])
            if s["bias_ids"] is not None:
                entries = dict(zip(s["bias_ids"][b].tolist(), s["bias_values"][b].double().tolist()))
                z[torch.tensor(list(entries), device=z.device)] += torch.tensor(list(entries.values()), dtype=torch.float64, device=z.device)
            if s["mask"] is not None:
                bits = (s["mask"][b, i].long()[:, None] >> torch.arange(32, device=z.device)) & 1
                z[bits.reshape(-1)[:V] == 0] = -math.inf
            out[b, i] = z
    return out


def _exact_top(s):
    c, t = s["case"], s["target"]
    n_seq, t_len, V = t.shape
    K = c["K"]
    ids = torch.full((n_seq, t_len, K), -1, dtype=torch.int32, device=t.device)
    logp = torch.full((n_seq, t_len, K), -math.inf, dtype=torch.float64, device=t.device)
    lse = torch.full((n_seq, t_len), -math.inf, dtype=torch.float64, device=t.device)
    for b in range(n_seq):
        n = t_len if s["n_rows"] is None else int(s["n_rows"][b])
        z = t[b, :n].double()
        order = torch.sort(z, dim=1, descending=True, stable=True)
        full = torch.log_softmax(z / c["T"], dim=1)
        kept = order.indices[:, :K]
        ids[b, :n], logp[b, :n] = kept.to(torch.int32), full.gather(1, kept)
        lse[b, :n] = torch.logsumexp(z / c["T"], dim=1)
    return ids, logp, lse


def _exact_loss(s):
    c = s["case"]
    draft, K = s["draft"], c["K"]
    n_seq, t_len, V = draft.shape
    kl = torch.zeros(n_seq, t_len, dtype=torch.float64, device=draft.device)
    grad = torch.zeros(draft.shape, dtype=torch.float64, device=draft.device) if c["grad"] else None
    for b in range(n_seq):
        have = s["ids"][b, :, 0] >= 0  # a list is whole or not there
        if not bool(have.any()):
            continue
        ids = s["ids"][b][have].long()
        logp = s["logp"][b][have].double()
        logq = torch.log_softmax(draft[b][have].double() / c["T"], dim=1)
        q = logq.exp()
        p = logp.exp()
        if c["tail"]:  # a distribution over the K listed tokens and one event for all others
            others = torch.ones_like(q).scatter_(1, ids, 0.0)
            rest = (q * others).sum(1)
            r = 1 - p.sum(1)
            r = torch.where(r < COMPLETE, torch.zeros_like(r), r)
            kl[b, have] = (p * (logp - logq.gather(1, ids))).sum(1) + torch.xlogy(r, r) - torch.xlogy(r, rest)
            target = q * others * (r / rest)[:, None]
            target.scatter_(1, ids, p)
        else:
            p = p / p.sum(1, keepdim=True)
            kl[b, have] = (p * (p.log() - logq.gather(1, ids))).sum(1)
            target = torch.zeros_like(q).scatter_(1, ids, p)
        if grad is not None:
            grad[b, have] = (q - target) * (float(s["weights"][b]) / c["T"])
    return kl, s["weights"].double() * kl.sum(1), grad
