"""The policy operators' numbers to a few float32 steps, on rows whose sums are
exact: what is left are the roundings of the rows' own numbers."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
F32, BF16 = torch.float32, torch.bfloat16
HALF = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


def level(T):
    return float(np.float32(T))          # what the entry points take


def pair_of_alike_rows(V, k, low, dtype, n):
    """A pair whose preferred sequence has n rows of k tokens at 0 and its own at
    `low`; the other's rows have but their own token, log p = 0."""
    z = torch.full((2, n, V), -INF, dtype=dtype, device=DEV)
    z[0, :, V - k:] = 0.0
    at = V - k - 1 if low < 0 else V - 1
    z[0, :, at] = low
    z[1, :, 0] = 0.0
    x = torch.zeros(2, n, dtype=torch.int32, device=DEV)
    x[0] = at
    return z, x


@pytest.mark.parametrize("T", [1.0, 0.6, 1.3])
@pytest.mark.parametrize("low", [0.0, -3.0, -40.0])
@pytest.mark.parametrize("V,dtype", [(2900, F32), (6000, BF16), (40008, BF16), (21001, F32)])
def test_a_margin_does_not_gather_roundings(V, dtype, low, T):
    """500 equal rows: an error that a row's log p keeps is in the margin 500 times.
    log p = low / T - log(k + e^(low / T)) is exact but for a logarithm of at most
    0.41, one step of which is 2^-25; what it is rounded to is carried along."""
    n, T = 500, level(T)
    for k in (V - 2, V // 2 + 3, 1777, 1500, 711, 97, 5):
        z, x = pair_of_alike_rows(V, k, low, dtype, n)
        others = k - 1 if low == 0 else k
        one = low / T - math.log(others + math.exp(low / T))
        ref = np.float32(n * one)
        logp, margin, _, _ = svp.preference_loss(z, x, torch.tensor([float(ref), 0.0], device=DEV),
                                                 torch.ones(1, device=DEV), beta=1.0, temperature=T, grad=False)
        assert (logp[1] == 0).all()
        assert (logp[0].double() - one).abs().max().item() <= HALF * abs(one) + 2.0 ** -25
        want = n * one - float(ref)
        assert abs(margin.item() - want) <= n * 2.0 ** -25 * 1.01 + HALF * abs(want), (k, margin.item(), want)


@pytest.mark.parametrize("T", [1.0, 0.6, 1.3])
@pytest.mark.parametrize("base,low", [(0.0, -20.0), (0.0, -29.0), (3.3, -14.0), (50.0, 15.0), (-7.0, -60.0)])
@pytest.mark.parametrize("V", [64, 9001])
def test_gradients_from_kept_numbers(V, base, low, T):
    """Rows of one likely token and their own, unlikely one: the likely token's
    probability is e^((z - z(x)) / T + log p), or e^(z / T - lse) for log p <= -32,
    with log p and lse as they were given.  That exponent is near 0, so it has no
    rounding of its own: 2^-22 of ex2.approx and four steps of products remain."""
    n, T = 400, level(T)
    g = torch.Generator().manual_seed(int(V + 10 * base + low))
    z = torch.full((n, 1, V), -INF)
    z[:, 0, 5] = base + torch.rand(n, generator=g)
    z[:, 0, 40] = low + torch.rand(n, generator=g)
    x = torch.full((n, 1), 40, dtype=torch.int32)
    z64 = z.double().numpy()[:, 0, [5, 40]] / T
    lse = np.logaddexp(z64[:, 0], z64[:, 1])
    logp32, lse32 = (z64[:, 1] - lse).astype(np.float32), lse.astype(np.float32)
    to = lambda a: torch.from_numpy(a)[:, None].to(DEV)
    d = torch.full((n, 1), -1.0, device=DEV)
    got = svp.token_logp_grad(z.to(DEV), x.to(DEV), to(logp32), to(lse32), d, temperature=T)[:, 0, 5].double().cpu().numpy()
    near = logp32 > -32
    want = np.exp(np.where(near, z64[:, 0] - z64[:, 1] + logp32.astype(np.float64), z64[:, 0] - lse32.astype(np.float64))) / T
    off = np.abs(got / want - 1)
    assert off.max() <= 2.0 ** -22 + 4 * HALF, (off.max(), np.median(off))


@pytest.mark.parametrize("T", [1.0, 0.6])
def test_gradients_of_entropies_from_kept_numbers(T):
    """The same rows with a derivative in the entropy: p (log p + H) at the likely
    token, whose log p is known to an absolute 2^-24 of the numbers it comes of."""
    n, T, V = 200, level(T), 64
    g = torch.Generator().manual_seed(3)
    z = torch.full((n, 1, V), -INF)
    z[:, 0, 5] = torch.rand(n, generator=g)
    z[:, 0, 9] = torch.rand(n, generator=g) - 1
    z[:, 0, 40] = torch.rand(n, generator=g) - 12
    x = torch.full((n, 1), 40, dtype=torch.int32)
    lp = torch.log_softmax(z[:, 0, [5, 9, 40]].double() / T, 1)
    lse = torch.logsumexp(z[:, 0].double() / T, 1)
    H = -(lp.exp() * lp).sum(1)
    f = lambda t: t.float()[:, None].to(DEV)
    one = torch.ones(n, 1, device=DEV)
    got = svp.token_logp_grad(z.to(DEV), x.to(DEV), f(lp[:, 2]), f(lse), 0 * one, entropy=f(H), d_entropy=one,
                              temperature=T)[:, 0, [5, 9, 40]].double().cpu()
    want = -lp.exp() * (lp + H[:, None]) / T
    # log p(x) of up to 32 comes rounded (2^-20), and is part of every exponent; t of up to 2 is
    # rounded three times, ex2.approx 2^-22
    size = lp.exp() * ((lp + H[:, None]).abs() + 1) / T
    assert ((got - want).abs() <= size * (2.0 ** -20 + 2.0 ** -21 + 2.0 ** -22)).all()


@pytest.mark.parametrize("V,dtype", [(17000, BF16), (9001, F32), (3000, F32)])
def test_sums_of_long_padded_rollouts(V, dtype):
    """The log-sum-exps of rows without a token are -inf, all others numbers; a
    rollout's loss is the 64-bit sum of its rows' float32 losses, rounded once."""
    n_seq, t_len = 3, 6700
    g = torch.Generator(device=DEV).manual_seed(4)
    z = torch.empty(n_seq, t_len, V, dtype=dtype, device=DEV)
    for part in z.view(-1, V).split(1000):
        part.copy_(torch.randn(part.shape, device=DEV, generator=g) * 2)
    x = torch.randint(0, V, (n_seq, t_len), device=DEV, generator=g).to(torch.int32)
    x[0, 1500:] = -1
    x[1, :4000] = -1
    x[2][torch.rand(t_len, device=DEV, generator=g) < 0.5] = -1
    A, w = torch.randn(n_seq, t_len, device=DEV, generator=g), torch.rand(n_seq, device=DEV, generator=g)
    logp, _, row, loss, _ = svp.policy_loss(z, x, A, w, grad=False)
    again, _, lse = svp.token_logp(z, x)
    live = x >= 0
    for t in (logp, again, row, lse):
        assert t[live].isfinite().all()
    assert (lse[~live] == -INF).all()
    assert torch.equal(logp, again)
    for b in range(n_seq):
        for at in live[b].nonzero()[:, 0].split(500):
            want = torch.logsumexp(z[b, at].double(), 1)
            assert (lse[b, at].double() - want).abs().max() < 4e-5      # 2 REL, as the other tests have it
    total = w.double() * row.double().sum(1)
    size = w.double() * row.double().abs().sum(1)
    assert ((loss.double() - total).abs() <= HALF * total.abs() + 1e-12 * size).all()
