"""A policy updated on verified rollouts.

  1. ``constrained_rollout.run`` gives rollouts whose tokens follow the target
     exactly (drafted, verified, redrawn);
  2. ``token_logp`` keeps the tokens' log-probabilities under the policy as it
     is: the old policy's for the ratios, and the reference's;
  3. a few steps of ``policy_loss`` on advantages within the batch, and one of
     ``preference_loss`` on pairs of a better and a worse rollout.  Both write the
     gradient over the logits;
  4. ``clip_gradients`` scales the parameters' gradients together before each
     step.

The policy is synthetic: logits A[last token] W.  A rollout's reward is the
share of its tokens that lie in the lower half of the vocabulary.

    python examples/policy_update.py --steps 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import speculative_decoding_verification_71_gb300 as svp  # noqa: E402
import constrained_rollout  # noqa: E402


class Policy:
    """Logits A[last token] W, and the gradients of A and W from those of the
    logits."""

    def __init__(self, V, rank, g):
        dev = g.device
        self.p = [torch.randn(V, rank, generator=g, device=dev) * 0.5, torch.randn(rank, V, generator=g, device=dev) * 0.3]

    def logits(self, before):
        return self.p[0][before] @ self.p[1]

    def gradients(self, before, d):
        rows = self.p[0][before].flatten(0, 1)
        d = d.flatten(0, 1)
        dA = torch.zeros_like(self.p[0]).index_put_((before.flatten(),), d @ self.p[1].t(), accumulate=True)
        return [dA, rows.t() @ d]


def batch(history, prompt_len, length, most):
    """(tokens, the tokens before them) of the rollouts, -1 where nothing is
    learnt: on prompts and after a rollout's end."""
    history = history[:, :most + 1]
    at = torch.arange(1, history.shape[1], device=history.device)
    learnt = (at >= prompt_len[:, None]) & (at < length[:, None])
    return torch.where(learnt, history[:, 1:], -1).contiguous(), history[:, :-1].long()


def rewards(tokens, V):
    have = tokens >= 0
    return (have & (tokens < V // 2)).sum(1) / have.sum(1).clamp(min=1)


def policy_step(policy, tokens, before, advantages, weights, old, ref, max_norm, lr):
    """One step of the policy loss; the losses, the gradients before they are
    scaled to ``max_norm``, and their norm."""
    z = policy.logits(before)
    _, _, _, loss, d = svp.policy_loss(z, tokens, advantages, weights, old_logp=old, ref_logp=ref, clip_high=0.28,
                                       kl_coef=0.02, entropy_coef=0.001, out=z)
    return (loss, *update(policy, before, d, max_norm, lr))


def preference_step(policy, tokens, before, ref, weights, max_norm, lr):
    z = policy.logits(before)
    _, _, loss, d = svp.preference_loss(z, tokens, ref, weights, beta=0.2, out=z)
    return (loss, *update(policy, before, d, max_norm, lr))


def update(policy, before, d, max_norm, lr):
    grads = policy.gradients(before, d)
    scaled = [torch.empty_like(x) for x in grads]
    norm = svp.clip_gradients(grads, max_norm, out=scaled)
    for p, x in zip(policy.p, scaled):
        p.sub_(lr * x)
    return grads, norm


def run(B=32, V=2000, rounds=20, steps=8, rank=32, max_norm=0.5, lr=0.5, seed=0, device="cuda", log=print):
    """Returns (losses, norms) of the steps and the policy."""
    _, rollouts = constrained_rollout.run(B=B, V=V, rounds=rounds, seed=seed, device=device, log=None)
    tokens, before = batch(*rollouts, most=int(rollouts[2].max()))
    policy = Policy(V, rank, torch.Generator(device=device).manual_seed(seed + 1))
    r = rewards(tokens, V)
    advantages = (r - r.mean()) / (r.std() + 1e-6)
    weights = 1.0 / (B * (tokens >= 0).sum(1).clamp(min=1)).float()
    old = ref = svp.token_logp(policy.logits(before), tokens)[0]
    losses, norms = [], []
    for step in range(steps):
        loss, _, norm = policy_step(policy, tokens, before, advantages, weights, old, ref, max_norm, lr)
        losses.append(loss.sum()), norms.append(norm)
    order = r.argsort(descending=True)
    pairs = torch.stack([order[:B // 2], order.flip(0)[:B // 2]], 1).flatten()   # the best with the worst, ...
    loss, _, norm = preference_step(policy, tokens[pairs].contiguous(), before[pairs], ref[pairs].sum(1),
                                    torch.full((B // 2,), 2.0 / B, device=device), max_norm, lr)
    losses.append(loss.sum()), norms.append(norm)
    if log:
        for i, (a, b) in enumerate(zip(losses, norms)):
            log(f"step {i + 1:3d}: loss {a.item():8.4f}, norm of the gradients {b.item():.4f}")
    return torch.stack(losses), torch.stack(norms), policy


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("--batch", 32), ("--vocab", 2000), ("--rounds", 20), ("--steps", 8), ("--seed", 0)):
        ap.add_argument(name, type=int, default=value)
    a = ap.parse_args()
    run(B=a.batch, V=a.vocab, rounds=a.rounds, steps=a.steps, seed=a.seed)
