"""The operators of a policy's update together, as the example uses them: its
parameters' gradients against automatic differentiation in 64 bits."""
import os
import sys

import pytest
import torch

from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _setup(B, V, T):
    svbuild.build()
    import policy_update
    g = torch.Generator(device="cuda").manual_seed(5)
    policy = policy_update.Policy(V, 16, g)
    history = torch.randint(0, V, (B, T + 1), generator=g, device="cuda").to(torch.int32)
    length = torch.randint(4, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    prompt = torch.full((B,), 3, dtype=torch.int32, device="cuda")
    return policy_update, policy, *policy_update.batch(history, prompt, length, T), g


def _logp64(p, tokens, before):
    lp = torch.log_softmax(p[0][before] @ p[1], -1)
    x = lp.gather(-1, tokens.long().clamp(min=0)[..., None])[..., 0]
    return torch.where(tokens >= 0, x, 0.0), -(lp.exp() * lp).sum(-1)


def _same(grads, p, norm):
    """float32 products of float32 gradients: a matrix product of up to a few
    hundred terms each way is off by 1e-5 of the terms' sizes, the gradients in
    the logits by 4e-5 of theirs."""
    total = sum(float(x.grad.square().sum()) for x in p) ** 0.5
    for d, x in zip(grads, p):
        assert (d.double() - x.grad).norm() <= 1e-4 * x.grad.norm()
    assert abs(norm.item() - total) <= 1e-4 * total


def test_the_policy_losses_gradients():
    example, policy, tokens, before, g = _setup(6, 501, 20)
    p = [x.double().clone().requires_grad_() for x in policy.p]
    logp, H = _logp64(p, tokens, before)
    # ratios away from the clipping's edges
    ratio = torch.tensor([0.6, 0.9, 1.0, 1.1, 1.6], device="cuda")[torch.randint(0, 5, tokens.shape, generator=g, device="cuda")]
    old = (logp.detach() - torch.log(ratio)).float()
    ref = (logp.detach() + 0.3 * torch.randn(tokens.shape, generator=g, device="cuda")).float()
    A = torch.randn(6, generator=g, device="cuda")
    w = torch.rand(6, generator=g, device="cuda")
    r = torch.exp(logp - old.double())
    a = A.double()[:, None]
    d = ref.double() - logp
    row = -torch.minimum(r * a, r.clamp(0.8, 1.28) * a) + 0.02 * (torch.exp(d) - d - 1) - 0.001 * H
    loss = w.double() * torch.where(tokens >= 0, row, 0.0).sum(1)
    loss.sum().backward()
    got, grads, norm = example.policy_step(policy, tokens, before, A, w, old, ref, 0.1, 0.1)
    assert (got.double() - loss.detach()).abs().max() <= 1e-4 * loss.detach().abs().max()
    _same(grads, p, norm)
    scale = min(1.0, 0.1 / (norm.item() + 1e-6))
    for x, q in zip(policy.p, p):                     # the step went along the scaled gradient
        assert (x.double() - (q.detach() - 0.1 * scale * q.grad)).abs().max() <= 1e-5


def test_the_preference_losses_gradients():
    example, policy, tokens, before, g = _setup(8, 501, 20)
    p = [x.double().clone().requires_grad_() for x in policy.p]
    s = _logp64(p, tokens, before)[0].sum(1)
    ref = (s.detach() + torch.randn(8, generator=g, device="cuda")).float()
    w = torch.rand(4, generator=g, device="cuda")
    h = (s[0::2] - s[1::2]) - (ref[0::2].double() - ref[1::2].double())
    loss = -w.double() * torch.nn.functional.logsigmoid(0.2 * h)
    loss.sum().backward()
    got, grads, norm = example.preference_step(policy, tokens, before, ref, w, 0.1, 0.1)
    assert (got.double() - loss.detach()).abs().max() <= 1e-4 * loss.detach().abs().max()
    _same(grads, p, norm)


def test_the_example_runs_and_repeats():
    svbuild.build()
    import policy_update
    a = policy_update.run(B=8, V=1003, rounds=6, steps=3, log=None)
    assert a[0].shape == (4,) and a[0].isfinite().all() and (a[1] > 0).all()
    torch.use_deterministic_algorithms(True, warn_only=True)    # index_put_ adds in one order
    try:
        runs = [policy_update.run(B=8, V=1003, rounds=6, steps=3, log=None) for _ in range(2)]
    finally:
        torch.use_deterministic_algorithms(False)
    assert torch.equal(runs[0][0], runs[1][0]) and torch.equal(runs[0][1], runs[1][1])
