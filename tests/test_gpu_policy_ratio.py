"""policy_loss where the ratio to the old policy passes float32's range and its
product with the advantage does not."""
import math

import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


@pytest.mark.parametrize("V", [100, 3000, 40008])
@pytest.mark.parametrize("per_token", [False, True])
def test_ratios_past_the_range(V, per_token):
    """An advantage of 0 (a group of equal rewards) has loss and gradient 0 at any
    ratio; a small one what the product comes to.  log p - old is rounded twice, at
    100: 2 x 2^-24 x 100 of the product, the exponentials and products a few steps
    more."""
    z = torch.zeros(6, 1, V, device=DEV)
    z[:, :, 1:] = -math.inf
    z[:, :, 1] = 1.0
    x = torch.zeros(6, 1, dtype=torch.int32, device=DEV)
    logp = -math.log1p(math.exp(1.0))
    old = torch.tensor([[-95.0], [-300.0], [-5000.0], [-95.0], [-95.0], [-95.0]], device=DEV)
    A = torch.tensor([0.0, -0.0, 0.0, -1e-12, 1e-12, -1e-12], device=DEV)
    w = torch.tensor([1.0, 1.0, 0.5, 1.0, 1.0, 0.25], device=DEV)
    _, _, row, loss, grad = svp.policy_loss(z, x, A[:, None] if per_token else A, w, old_logp=old)
    row, loss, grad = row[:, 0].double().cpu(), loss.double().cpu(), grad[:, 0, :2].double().cpu()
    assert (row[:3] == 0).all() and (loss[:3] == 0).all() and (grad[:3] == 0).all()
    assert row[4].item() == pytest.approx(-1.2e-12, rel=1e-6) and (grad[4] == 0).all()
    big = 1e-12 * math.exp(logp + 95.0)
    rest = 1 - math.exp(logp)
    for i, weight in ((3, 1.0), (5, 0.25)):
        assert row[i].item() == pytest.approx(big, rel=2e-5) and loss[i].item() == pytest.approx(weight * big, rel=2e-5)
        assert grad[i, 0].item() == pytest.approx(weight * big * rest, rel=2e-5)
        assert grad[i, 1].item() == pytest.approx(-weight * big * rest, rel=2e-5)
    # with the other clip such a row is held
    _, _, row, _, grad = svp.policy_loss(z, x, A, w, old_logp=old, dual_clip=3.0)
    assert row[3, 0].item() == pytest.approx(3e-12, rel=1e-6) and (grad == 0).all()


@pytest.mark.parametrize("V", [100, 40008])
def test_divergences_past_the_range(V):
    """e^d with d = ref - log p above 88: where kl_coef times it is in range, so are
    the loss and the gradient.  d is rounded twice (2 x 2^-24 x 95 of the product)."""
    z = torch.full((3, 1, V), -math.inf, device=DEV)
    z[:, :, 0] = 0.0
    z[:, :, 1] = torch.tensor([-90.0, -95.0, -300.0], device=DEV)[:, None]
    x = torch.ones(3, 1, dtype=torch.int32, device=DEV)
    ref = torch.zeros(3, 1, device=DEV)
    w = torch.ones(3, device=DEV)
    _, _, row, loss, grad = svp.policy_loss(z, x, 0 * w, w, ref_logp=ref, kl_coef=1e-3)
    for i, d in enumerate((90.0, 95.0)):
        big = 1e-3 * math.exp(d)
        assert row[i, 0].item() == pytest.approx(big, rel=2e-5) and loss[i].item() == pytest.approx(big, rel=2e-5)
        assert grad[i, 0, 1].item() == pytest.approx(-big, rel=2e-5) and grad[i, 0, 0].item() == pytest.approx(big, rel=2e-5)
    assert row[2, 0].item() == math.inf and grad[2].isnan().all()       # past the range: as documented
