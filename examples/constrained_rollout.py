"""A rollout with sampling rules, verified without loss, whose drafter learns
from the target's top log-probabilities.

One round for a batch of sequences:

  1. the drafter proposes k tokens, its rows processed like the target's
     (``process_logits``: penalties, a bias, a grammar's mask);
  2. the target scores them, and its rows are processed with each row's own
     history;
  3. ``SpecVerifier.verify`` accepts or redraws, so the rollout follows the
     processed target exactly;
  4. ``kd_top`` keeps the target's likeliest tokens at the emitted positions;
  5. every few rounds ``kd_top_loss`` gives the drafter's gradient from the
     kept lists.

The models are synthetic: the target's next-token logits depend on the last
token through a fixed table, the drafter has a table of lower rank that starts
at random.  The grammar alternates two classes of tokens.

    python examples/constrained_rollout.py --rounds 60
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_71_gb300 as svp  # noqa: E402


def grammar_words(V, device):
    """Two masks [2, ceil(V / 32)]: after a token of one class (even, odd) only
    the other class is allowed."""
    token = torch.arange((V + 31) // 32 * 32, device=device).view(-1, 32)
    bit = 1 << torch.arange(32, device=device)
    words = torch.stack([((token % 2 == c) * bit).sum(1) for c in (1, 0)])
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


class Drafter:
    """Logits A[last token] W, trained by Adam on gradients in the logits."""

    def __init__(self, V, rank, g, lr=0.03):
        dev = g.device
        self.p = [torch.randn(V, rank, generator=g, device=dev) * 0.5, torch.randn(rank, V, generator=g, device=dev) * 0.1]
        self.m = [torch.zeros_like(x) for x in self.p]
        self.v = [torch.zeros_like(x) for x in self.p]
        self.lr, self.t = lr, 0

    def logits(self, last):
        return self.p[0][last] @ self.p[1]

    def step(self, last, grad):
        rows, W = self.p[0][last], self.p[1]
        grads = [torch.zeros_like(self.p[0]).index_put_((last,), grad @ W.t(), accumulate=True), rows.t() @ grad]
        self.t += 1
        for x, d, m, v in zip(self.p, grads, self.m, self.v):
            m.mul_(0.9).add_(d, alpha=0.1)
            v.mul_(0.99).addcmul_(d, d, value=0.01)
            x.sub_(self.lr * (m / (1 - 0.9 ** self.t)) / ((v / (1 - 0.99 ** self.t)).sqrt() + 1e-8))


def run(B=64, V=2000, k=3, rounds=60, train_every=2, K=32, rank=64, T=1.0, seed=0, device="cuda", log=print):
    """Returns the mean number of tokens emitted a round, per round, and the
    sequences (token history, prompt length, length)."""
    g = torch.Generator(device=device).manual_seed(seed)
    table = torch.randn(V, 32, generator=g, device=device) @ torch.randn(32, V, generator=g, device=device) * 0.6
    drafter = Drafter(V, rank, g)
    verifier = svp.SpecVerifier(B, k, V, torch.float32)
    words = grammar_words(V, device)
    prompt = 4
    H = prompt + rounds * (k + 1) + k
    history = torch.zeros(B, H, dtype=torch.int32, device=device)
    history[:, :prompt] = torch.randint(0, V // 2, (B, prompt), generator=g, device=device).to(torch.int32) * 2
    history[:, 1::2] += 1                     # the prompt keeps to the grammar: even, odd, even, odd
    length = torch.full((B,), prompt, dtype=torch.int32, device=device)
    prompt_len = length.clone()
    rules = dict(repetition=torch.full((B,), 1.1, device=device), presence=torch.full((B,), 0.2, device=device),
                 frequency=torch.full((B,), 0.1, device=device),
                 bias_ids=torch.zeros(B, 1, dtype=torch.int32, device=device),
                 bias_values=torch.full((B, 1), -4.0, device=device))   # token 0 is unwelcome
    seq = torch.arange(B, device=device)
    draft_len = torch.full((B,), k, dtype=torch.int32, device=device)
    kept, emitted = [], []
    for step in range(rounds):
        last = history[seq, length.long() - 1].long()
        tokens = torch.empty(B, k, dtype=torch.int32, device=device)
        draft = torch.empty(B, k, V, device=device)
        follows = torch.empty(B, k + 1, dtype=torch.long, device=device)   # the token before each position
        follows[:, 0] = last
        for j in range(k):
            row = drafter.logits(follows[:, j]).view(B, 1, V)
            # drafted tokens are appended, so the history of row j ends with them
            svp.process_logits(row, history=history, prompt_len=prompt_len, history_len=length + j,
                               mask=words[follows[:, j] % 2].view(B, 1, -1), out=row, **rules)
            draft[:, j] = row[:, 0]
            tokens[:, j] = torch.multinomial(torch.softmax(row[:, 0] / T, 1), 1, generator=g)[:, 0].to(torch.int32)
            follows[:, j + 1] = tokens[:, j].long()
            history[seq, length.long() + j] = tokens[:, j]
        target = table[follows]
        processed = svp.process_logits(target, history=history, prompt_len=prompt_len, history_len=length, tokens=tokens,
                                       draft_len=draft_len, mask=words[follows % 2], **rules)
        uniforms = torch.rand(B, k + 1, generator=g, device=device)
        out, out_len = verifier.verify(processed, draft, tokens, draft_len, uniforms, T)
        # what was emitted replaces what was drafted
        place = length.long()[:, None] + torch.arange(k + 1, device=device)
        history.scatter_(1, place, torch.where(torch.arange(k + 1, device=device) < out_len[:, None], out, 0))
        length = length + out_len
        ids, logp, _ = svp.kd_top(target, K, T, n_rows=out_len)
        kept.append((ids, logp, follows.clone()))
        emitted.append(out_len.float().mean().item())
        if (step + 1) % train_every == 0:
            ids, logp = (torch.cat([x[i] for x in kept[-4:]], 1).contiguous() for i in (0, 1))
            before = torch.cat([x[2] for x in kept[-4:]], 1)
            rows = drafter.logits(before.reshape(-1)).view(B, -1, V)
            weights = torch.full((B,), 1.0 / before.numel(), device=device)
            _, loss, grad = svp.kd_top_loss(ids, logp, rows, weights, T)
            drafter.step(before.reshape(-1), grad.view(-1, V))
            if log and (step + 1) % (train_every * 5) == 0:
                log(f"round {step + 1:4d}: {sum(emitted[-10:]) / len(emitted[-10:]):.2f} tokens emitted a round, "
                    f"loss {loss.sum().item():.3f}")
    status, _ = verifier.stats()
    if status != svp.SV_OK:
        raise RuntimeError(f"verification reported {status}")
    verifier.close()
    return emitted, (history, prompt_len, length)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("--batch", 64), ("--vocab", 2000), ("--drafts", 3), ("--rounds", 60), ("--keep", 32), ("--seed", 0)):
        ap.add_argument(name, type=int, default=value)
    a = ap.parse_args()
    run(B=a.batch, V=a.vocab, k=a.drafts, rounds=a.rounds, K=a.keep, seed=a.seed)
