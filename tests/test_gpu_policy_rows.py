"""The policy operators on rows of up to 32 KB in batches that are padded: more
rows than the warps that hold them, with rows without a token in between."""
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild
from tests.policy_reference import REL

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


def padded(n, V, dtype, seed):
    """Rows and tokens: a row is dealt to the same warps as those 608 and 1216
    rows later, so runs of one, two and three rows without a token are laid
    along those, beside rows that lack one at random."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    z = torch.empty(n, 1, V, dtype=dtype, device=DEV)
    for part in z.split(500):
        part.copy_(torch.randn(part.shape, device=DEV, generator=g) * 2)
    x = torch.randint(0, V, (n, 1), device=DEV, generator=g).to(torch.int32)
    r = torch.arange(n, device=DEV)
    for stride in (608, 1216):
        turn, run = r // stride, 1 + r % 3              # one live row, then `run` without a token
        x[(turn % (run + 1) > 0) & (r % 2 == (stride == 608))] = -1
    x[torch.rand(n, 1, device=DEV, generator=g) < 0.1] = -1
    return z, x, g


# two or four warps to a row: rows of 8 to 16 KB and of 16 to 32 KB
PADDED = [(8000, BF16), (16000, BF16), (3000, F32), (8000, F32), (7001, BF16), (2051, F32)]


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("V,dtype", PADDED, ids=[f"{v}-{str(d)[6:]}" for v, d in PADDED])
def test_rows_without_a_token_between_others(V, dtype, grad):
    n = 8000
    z, x, g = padded(n, V, dtype, V)
    A, w = torch.randn(n, device=DEV, generator=g), torch.ones(n, device=DEV)
    logp, H, row, _, d = svp.policy_loss(z, x, A, w, entropy_coef=0.1, grad=grad)
    again, _, lse = svp.token_logp(z, x)
    live = x[:, 0] >= 0
    assert 2000 < int(live.sum()) < 6000
    for t in (logp, H, row, again):
        assert (t[~live] == 0).all()
    assert (lse[~live] == -INF).all()
    assert not grad or (d[~live] == 0).all()
    for at in live.nonzero()[:, 0].split(500):
        lp = torch.log_softmax(z[at, 0].double(), 1)
        p, tok = lp.exp(), x[at].long()
        lpx, ent = lp.gather(1, tok), -(p * lp).sum(1, keepdim=True)
        assert (logp[at] - lpx).abs().max() < 2 * REL and (again[at] - lpx).abs().max() < 2 * REL
        assert (lse[at] - torch.logsumexp(z[at, 0].double(), 1, keepdim=True)).abs().max() < 2 * REL
        assert (H[at] - ent).abs().max() < 10 * REL * (1 + ent.max())
        if not grad:
            continue
        a = -A[at].double()[:, None]
        want = -p * a + 0.1 * p * (lp + ent)
        want.scatter_add_(1, tok, a)
        # float32: 4 REL of the two parts' sizes, and half a step of the type
        size = p * a.abs() + 0.1 * p * (lp.abs() + ent + 1)
        size.scatter_add_(1, tok, a.abs() * (1 - p.gather(1, tok)))
        half = 2.0 ** -8 if dtype == BF16 else 2.0 ** -24
        assert ((d[at, 0].double() - want).abs() <= 4 * REL * size + half * want.abs() * 1.001 + 1e-37).all()


# rows of whole vectors: they begin on a 16-byte boundary wherever they lie (the order in
# which a row is summed follows its address modulo 16, so others change with their place)
ALIKE = [(v, d) for v, d in PADDED if v * (2 if d == BF16 else 4) % 16 == 0]


@pytest.mark.parametrize("V,dtype", ALIKE, ids=[f"{v}-{str(d)[6:]}" for v, d in ALIKE])
def test_the_same_bits_without_the_rows_in_between(V, dtype):
    n = 8000
    z, x, g = padded(n, V, dtype, V + 1)
    A, w = torch.randn(n, device=DEV, generator=g), torch.ones(n, device=DEV)
    live = (x[:, 0] >= 0).nonzero()[:, 0]
    whole = svp.policy_loss(z, x, A, w, entropy_coef=0.1)
    part = svp.policy_loss(z[live].contiguous(), x[live], A[live], w[live], entropy_coef=0.1)
    for a, b in zip(whole, part):
        assert torch.equal(a[live], b)
    n -= n % 2                                          # pairs: the rows' numbers, and the gradient from them
    pairs = svp.preference_loss(z[:n], x[:n], torch.zeros(n, device=DEV), w[:n // 2], beta=0.3)
    keep = ((x[:n:2, 0] >= 0) & (x[1:n:2, 0] >= 0)).nonzero()[:, 0]
    rows = torch.stack([2 * keep, 2 * keep + 1], 1).flatten()
    part = svp.preference_loss(z[rows].contiguous(), x[rows], torch.zeros(len(rows), device=DEV), w[:len(keep)], beta=0.3)
    for a, b, at in zip(pairs, part, (rows, keep, keep, rows)):
        assert torch.equal(a[at], b)


def test_the_workspace_is_what_the_library_asks_for(monkeypatch):
    """No formula of its own in the binding."""
    lib, asked = svp.load_library(), []
    real = lib.sv_preference_work
    monkeypatch.setattr(lib, "sv_preference_work", lambda n, t: asked.append((n, t)) or real(n, t))
    z = torch.zeros(6, 5, 40, device=DEV)
    x, w = torch.zeros(6, 5, dtype=torch.int32, device=DEV), torch.zeros(6, device=DEV)
    svp.preference_loss(z, x, w, w[:3])
    assert asked == [(3, 5)]
