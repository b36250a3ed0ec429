"""The operators together, as the example uses them: rules on both models'
rows, verification, the target's lists and the drafter's update."""
import os
import sys

import pytest
import torch

from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_the_drafter_learns_and_the_grammar_holds():
    svbuild.build()
    import constrained_rollout
    emitted, (history, prompt_len, length) = constrained_rollout.run(rounds=60, log=None)
    first, last = sum(emitted[:8]) / 8, sum(emitted[-8:]) / 8
    assert last > first + 0.3, (first, last)         # more drafts are accepted
    for b in range(history.shape[0]):
        seq = history[b, :int(length[b])].cpu()
        assert ((seq[1:] + seq[:-1]) % 2 == 1).all()  # even and odd alternate throughout
    assert int(length.min()) >= int(prompt_len[0]) + 60


def test_the_same_seed_gives_the_same_rollout():
    svbuild.build()
    import constrained_rollout
    a = constrained_rollout.run(B=8, V=1003, rounds=6, log=None)
    b = constrained_rollout.run(B=8, V=1003, rounds=6, log=None)
    assert a[0] == b[0] and torch.equal(a[1][0], b[1][0])
