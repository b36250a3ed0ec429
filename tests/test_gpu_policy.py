"""token_logp, token_logp_grad, policy_loss and preference_loss against their
definitions in 64 bits; tolerances as policy_reference.py derives them."""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild
from tests.policy_reference import REL, Rows, assert_close, policy, preference

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF, NAN = float("inf"), float("nan")
F32, BF16 = torch.float32, torch.bfloat16
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def make_rows(n_seq, t_len, V, dtype, seed=0, absent=0.2):
    """Rows of which half are nearly sure of one token, often the row's own."""
    g = gen(seed)
    z = torch.randn(n_seq, t_len, V, generator=g) * 2
    x = torch.randint(0, V, (n_seq, t_len), generator=g)
    boost = torch.rand(n_seq, t_len, generator=g) * 18
    z.scatter_add_(2, x[..., None], boost[..., None])
    other = torch.rand(n_seq, t_len, generator=g) < 0.25
    x = torch.where(other, torch.randint(0, V, (n_seq, t_len), generator=g), x)
    x[torch.rand(n_seq, t_len, generator=g) < absent] = -1
    return z.to(dtype), x.to(torch.int32)


def shifted(t, by):
    """The tensor at an address `by` elements past a 16-byte boundary."""
    flat = torch.empty(t.numel() + by, dtype=t.dtype, device=DEV)[by:]
    return flat.view(t.shape).copy_(t)


SHAPES = [  # n_seq, t_len, V, dtype, T
    (1, 1, 1, F32, 1.0), (1, 2, 1, BF16, 0.5), (2, 3, 5, BF16, 1.0), (3, 1, 100, F32, 0.7), (2, 3, 1000, BF16, 1.3),
    (2, 2, 4099, F32, 0.6), (2, 2, 4099, BF16, 1.0), (1, 3, 8191, F32, 1.0), (2, 2, 16379, BF16, 1.0),
    (1, 2, 16400, BF16, 1.0), (1, 2, 20000, BF16, 0.8), (1, 3, 50001, F32, 1.0), (1, 2, 100003, BF16, 1.0),
    (2, 2, 128256, BF16, 1.0), (1, 2, 151936, F32, 1.0), (1, 1, 262144, F32, 1.0), (1, 1, 524288, BF16, 1.0),
    (40, 9, 3000, BF16, 1.0), (400, 2, 777, F32, 1.0), (7, 50, 33001, BF16, 1.0),
]
IDS = [f"{a}x{b}x{c}-{str(d)[6:]}-T{e}" for a, b, c, d, e in SHAPES]


def check_logp(z, x, T, entropy, dev=None):
    R = Rows(z, x, T)
    logp, H, lse = svp.token_logp(z.to(DEV) if dev is None else dev, x.to(DEV), T, entropy=entropy)
    torch.cuda.synchronize()
    assert logp.shape == lse.shape == x.shape and (H is None) == (not entropy)
    assert_close(logp, R.logp, R.tol_logp, what="logp")
    assert_close(lse, R.lse, R.tol_lse, what="lse")
    if entropy:
        assert_close(H, R.H, R.tol_H, what="entropy")
    return R


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("n_seq,t_len,V,dtype,T", SHAPES, ids=IDS)
def test_logp_matches_the_definition(n_seq, t_len, V, dtype, T, entropy):
    check_logp(*make_rows(n_seq, t_len, V, dtype, seed=V), T, entropy)


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("n_seq,t_len,V,dtype,T", SHAPES, ids=IDS)
def test_logp_gradient_matches_the_formula(n_seq, t_len, V, dtype, T, entropy):
    z, x = make_rows(n_seq, t_len, V, dtype, seed=V + 1)
    R = Rows(z, x, T)
    g = torch.randn(n_seq, t_len, generator=gen(3))
    h = torch.randn(n_seq, t_len, generator=gen(4)) * 0.1
    # what token_logp gives, to float32
    f = lambda a: torch.from_numpy(a.reshape(x.shape)).float().to(DEV)
    got = svp.token_logp_grad(z.to(DEV), x.to(DEV), f(R.logp), f(R.lse), g.to(DEV), temperature=T,
                              entropy=f(R.H) if entropy else None, d_entropy=h.to(DEV) if entropy else None)
    g64, h64 = g.double().numpy().reshape(-1), h.double().numpy().reshape(-1) if entropy else np.zeros(R.n)
    ref, tol = R.gradient(g64, h64, 0 * g64)
    # logp and lse come rounded: every probability shares that
    tol = tol + np.abs(ref) * (2.0 ** -23 * (1 + np.abs(np.where(R.ok, R.lse, 0.0))))[:, None]
    assert got.dtype == dtype and got.shape == z.shape
    assert_close(got, ref, tol, dtype, "gradient")


def run_policy(z, x, T=1.0, seed=5, per_token=False, old=True, kl=0.0, ent=0.0, dual=None, entropy=False, grad=True,
               out=None, dev=None):
    n_seq, t_len, _ = z.shape
    g = gen(seed)
    R = Rows(z, x, T)
    A = torch.randn((n_seq, t_len) if per_token else (n_seq,), generator=g)
    w = torch.rand(n_seq, generator=g) + 0.1
    base = torch.from_numpy(np.where(np.isfinite(R.logp), R.logp, 0.0).reshape(x.shape))
    old_t = None
    if old:
        ratio = torch.exp(torch.randn(n_seq, t_len, generator=g) * 0.3).clamp(0.3, 8.0)
        ratio[torch.rand(n_seq, t_len, generator=g) < 0.1] = 5.0
        for edge in (0.8, 1.28, dual or 0.8):   # away from the ratios at which the gradient jumps
            ratio = torch.where((ratio - edge).abs() < 1e-3, torch.ones(()), ratio)
        old_t = (base - torch.log(ratio)).float()
    ref_t = (base + torch.randn(n_seq, t_len, generator=g) * 0.3).float() if kl else None
    to = lambda t: None if t is None else t.to(DEV)
    res = svp.policy_loss(z.to(DEV) if dev is None else dev, to(x), to(A), to(w), old_logp=to(old_t), ref_logp=to(ref_t),
                          temperature=T, clip_low=0.2, clip_high=0.28, dual_clip=dual, kl_coef=kl, entropy_coef=ent,
                          entropy=entropy, grad=grad, out=out)
    torch.cuda.synchronize()
    each = lambda t: None if t is None else (t if t.dim() == 2 else t[:, None].expand(n_seq, t_len)).double().numpy().reshape(-1)
    row, tol_row, slope, tol_slope, h = policy(R, each(A), each(w), each(old_t), each(ref_t), 0.2, 0.28, dual, kl, ent)
    logp, H, row_loss, loss, got = res
    assert_close(logp, R.logp, R.tol_logp, what="logp")
    assert (H is not None) == bool(entropy or ent)
    if H is not None:
        assert_close(H, R.H, R.tol_H, what="entropy")
    assert_close(row_loss, row, tol_row, what="row loss")
    total = w.double().numpy() * row.reshape(n_seq, t_len).sum(1)
    # the sum is of row losses rounded to float32, in 64 bits
    tol = w.double().numpy() * (tol_row + 2.0 ** -24 * np.abs(row)).reshape(n_seq, t_len).sum(1)
    assert_close(loss, total, np.where(np.isfinite(total), tol, 0.0), what="loss")
    if grad:
        ref, tol = R.gradient(slope, h, tol_slope)
        assert got.dtype == z.dtype and got.shape == z.shape
        assert_close(got, ref, tol, z.dtype, "gradient")
    else:
        assert got is None
    return res


@pytest.mark.parametrize("n_seq,t_len,V,dtype,T", SHAPES, ids=IDS)
def test_policy_loss_matches_the_definition(n_seq, t_len, V, dtype, T):
    z, x = make_rows(n_seq, t_len, V, dtype, seed=V + 2)
    run_policy(z, x, T)
    run_policy(z, x, T, per_token=True, kl=0.05, ent=0.01, dual=3.0, entropy=True)


@pytest.mark.parametrize("over", [dict(old=False), dict(old=False, kl=0.1), dict(kl=-0.02, per_token=True), dict(ent=-0.5),
                                  dict(dual=2.0), dict(entropy=True), dict(grad=False), dict(grad=False, ent=0.1, kl=0.1)],
                         ids=lambda o: ",".join(f"{k}={v}" for k, v in o.items()))
@pytest.mark.parametrize("V,dtype", [(5003, F32), (40008, BF16)])
def test_policy_loss_variants(V, dtype, over):
    z, x = make_rows(5, 7, V, dtype, seed=V + 3)
    run_policy(z, x, 0.9, **over)


def run_preference(z, x, T=1.0, beta=0.1, kind="sigmoid", smoothing=0.0, average=False, grad=True, out=None, seed=7,
                   dev=None, move=2.0):
    n_seq, t_len, _ = z.shape
    g = gen(seed)
    R = Rows(z, x, T)
    have = (x >= 0).sum(1).numpy()
    per = 1.0 / np.maximum(have, 1) if average else np.ones(n_seq)
    s = R.logp.reshape(n_seq, t_len).sum(1) * per
    ref = (torch.from_numpy(np.where(np.isfinite(s), s, 0.0)) + torch.randn(n_seq, generator=g) * move).float()
    w = torch.rand(n_seq // 2, generator=g) + 0.1
    logp, margin, loss, got = svp.preference_loss(z.to(DEV) if dev is None else dev, x.to(DEV), ref.to(DEV), w.to(DEV),
                                                  beta=beta, temperature=T, kind=kind, smoothing=smoothing,
                                                  average=average, grad=grad, out=out)
    torch.cuda.synchronize()
    assert_close(logp, R.logp, R.tol_logp, what="logp")
    fin = np.where(np.isfinite(R.logp), np.abs(R.logp), 0.0)
    off = np.where(np.isfinite(R.tol_logp), R.tol_logp, 0.0) + 2.0 ** -24 * fin
    tol_s = np.where(R.ok, off, 0.0).reshape(n_seq, t_len).sum(1) * per + 1e-12
    slopes, tol_g = np.zeros(n_seq), np.zeros(n_seq)
    for i in range(n_seq // 2):
        a, b = 2 * i, 2 * i + 1
        at = [preference((s[a] + d, s[b]), ref[a:b + 1], float(w[i]), beta, kind, smoothing)
              for d in (0.0, tol_s[a] + tol_s[b], -tol_s[a] - tol_s[b])]
        (m, l, k), spread = at[0], [max(abs(at[j][q] - at[0][q]) for j in (1, 2)) for q in range(3)]
        assert_close(margin[i], np.array(m), np.array(spread[0]), what="margin")
        # from m, rounded to float32 (2^-24 |m|, of which softplus passes on at most
        # w |slope| / beta and the sigmoid's logarithm all), the loss and its slope
        # come by up to eight float32 steps: expf and log1pf or a division (one ulp
        # each, 2^-23), a sum, 1 - e, the products with it, w, beta and 1 / n (2^-24)
        near = 2.0 ** -24 * (10 + abs(m)) if math.isfinite(m) else 0.0
        assert_close(loss[i], np.array(l), np.array(spread[1]) + near * (abs(l) + abs(k) / beta) + 1e-30, what="loss")
        slopes[a], slopes[b] = k * per[a], -k * per[b]
        tol_g[a], tol_g[b] = (spread[2] + near * abs(k)) * per[a], (spread[2] + near * abs(k)) * per[b]
    if grad:
        each = lambda v: np.repeat(v, t_len)
        dref, tol = R.gradient(each(slopes), np.zeros(R.n), each(tol_g))
        # a pair with a sequence that has no number has none in any of its rows
        bad = each(np.repeat(~np.isfinite(slopes[0::2]), 2)) & R.live
        dref[bad] = np.nan
        dref[~R.live] = 0.0
        assert got.dtype == z.dtype
        assert_close(got, dref, tol, z.dtype, "gradient")
    else:
        assert got is None
    return logp, margin, loss, got


PAIRS = [(2 * max(1, a // 2), b, c, d, e) for a, b, c, d, e in SHAPES]


@pytest.mark.parametrize("n_seq,t_len,V,dtype,T", PAIRS, ids=[f"{a}x{b}x{c}-{str(d)[6:]}-T{e}" for a, b, c, d, e in PAIRS])
def test_preference_loss_matches_the_definition(n_seq, t_len, V, dtype, T):
    run_preference(*make_rows(n_seq, t_len, V, dtype, seed=V + 4), T)


@pytest.mark.parametrize("kind,smoothing", [("sigmoid", 0.0), ("sigmoid", 0.2), ("hinge", 0.0), ("ipo", 0.0)])
@pytest.mark.parametrize("average", [False, True])
@pytest.mark.parametrize("V,dtype", [(5003, F32), (40008, BF16)])
def test_preference_kinds(V, dtype, kind, smoothing, average):
    z, x = make_rows(8, 9, V, dtype, seed=V + 5)
    for beta, move in ((0.1, 2.0), (2.0, 2.0)):
        run_preference(z, x, 0.9, beta, kind, smoothing, average, move=move)
    run_preference(z, x, 0.9, 0.1, kind, smoothing, average, grad=False)


def test_preference_of_empty_sequences():
    z, x = make_rows(6, 4, 3001, F32, seed=1)
    x[0], x[1], x[2] = -1, -1, -1
    for average in (False, True):
        run_preference(z, x, average=average)


def test_preference_of_many_long_pairs():
    z, x = make_rows(6, 300, 1500, BF16, seed=2, absent=0.3)
    run_preference(z, x)
    z, x = make_rows(260, 3, 700, F32, seed=3)
    run_preference(z, x)


# ---------------------------------------------------------------------------
# Rows that are masked, invalid, or far from 0
# ---------------------------------------------------------------------------

def odd_rows(V, dtype):
    """Rows and tokens of every unusual kind."""
    g = gen(V)
    base = torch.randn(V, generator=g)
    low = float(torch.finfo(dtype).min)
    rows, toks = [], []

    def put(z, x):
        rows.append(z.clone()), toks.append(x)

    z = base.clone()
    z[2:] = -INF
    put(z, 1), put(z, 0), put(z, V - 1)                     # masked but for two; the token masked
    z = base.clone()
    z[3:] = low
    put(z, 2), put(z, V - 1)                                # the type's lowest value for a mask
    put(torch.full((V,), -INF), 0)                          # nothing left
    put(torch.full((V,), low), 1)                           # masked whole with the lowest value
    z = torch.full((V,), -INF)
    z[V // 2] = 3.0
    put(z, V // 2), put(z, 0)                               # one token left
    for bad in (NAN, INF):
        for at in (0, V // 2, V - 1):
            z = base.clone()
            z[at] = bad
            put(z, 1), put(z, at)
    put(base, V), put(base, 2 ** 31 - 1), put(base, -1), put(base, -2 ** 31)
    for level in (1e4, -1e4):
        put(base + level, 1)
    z = base.clone()
    z[1] = 1e30
    put(z, 1), put(z, 0)                                    # a token forced
    z = base.clone()
    z[0], z[1] = -low * 0.9, low * 0.9                      # a difference past the range
    put(z, 0)
    put(torch.zeros(V), V - 1), put(torch.full((V,), -0.0), 0)
    z = torch.full((V,), NAN)
    put(z, 0), put(z, -1)
    return torch.stack(rows)[:, None].to(dtype), torch.tensor(toks, dtype=torch.int64).to(torch.int32)[:, None]


ODD = [(40, F32), (40, BF16), (5003, F32), (5003, BF16), (40008, BF16), (140001, F32)]


@pytest.mark.parametrize("V,dtype", ODD, ids=[f"{v}-{str(d)[6:]}" for v, d in ODD])
@pytest.mark.parametrize("T", [1.0, 0.6, 1.7])
def test_logp_of_masked_and_invalid_rows(V, dtype, T):
    check_logp(*odd_rows(V, dtype), T, True)
    check_logp(*odd_rows(V, dtype), T, False)


@pytest.mark.parametrize("V,dtype", ODD, ids=[f"{v}-{str(d)[6:]}" for v, d in ODD])
def test_policy_loss_of_masked_and_invalid_rows(V, dtype):
    z, x = odd_rows(V, dtype)
    R = Rows(z, x, 1.0)
    keep = torch.from_numpy(~R.ok | (R.logp > -1e4))      # a log-probability of -inf: the test below
    for over in (dict(), dict(ent=0.01, per_token=True), dict(kl=0.1)):
        run_policy(z[keep].contiguous(), x[keep].contiguous(), **over)


@pytest.mark.parametrize("V,dtype", ODD, ids=[f"{v}-{str(d)[6:]}" for v, d in ODD])
def test_preference_loss_of_masked_and_invalid_rows(V, dtype):
    z, x = odd_rows(V, dtype)
    R = Rows(z, x, 1.0)
    keep = torch.from_numpy(~R.ok | (R.logp > -1e4))
    z, x = z[keep], x[keep]
    n = len(z) // 2 * 2
    run_preference(z[:n].contiguous(), x[:n].contiguous())


def test_a_token_that_the_policy_cannot_say():
    """log p = -inf: r = 0, so nothing is to be learnt for A > 0 and the clipped
    term holds for A < 0; a divergence is infinite and has no gradient."""
    z = torch.randn(3, 1, 100)
    z[:, :, 7] = -INF
    x = torch.full((3, 1), 7, dtype=torch.int32)
    A = torch.tensor([1.0, -1.0, 0.0])
    args = [t.to(DEV) for t in (z, x, A, torch.ones(3))]
    old = torch.full((3, 1), -1.0, device=DEV)
    logp, _, row, loss, grad = svp.policy_loss(*args, old_logp=old)
    assert (logp == -INF).all() and torch.allclose(row[:, 0].cpu(), torch.tensor([0.0, 0.8, 0.0]))
    assert (grad == 0).all()
    logp, _, row, loss, grad = svp.policy_loss(*args, old_logp=old, ref_logp=old, kl_coef=0.1)
    assert (row == INF).all() and (loss == INF).all() and grad.isnan().all()


def test_a_derivative_past_the_range_has_no_gradient():
    z, x = make_rows(2, 1, 50, F32, absent=0.0)
    old = torch.full((2, 1), -200.0, device=DEV)      # r = e^(200 + log p): past the range
    A = torch.tensor([-1.0, 1.0], device=DEV)
    _, _, row, _, grad = svp.policy_loss(z.to(DEV), x.to(DEV), A, torch.ones(2, device=DEV), old_logp=old)
    assert row[0, 0] == INF and grad[0].isnan().all()
    assert abs(row[1, 0].item() + 1.2) < 1e-6 and (grad[1] == 0).all()


def test_gradients_are_the_losses_differences():
    """Along random directions, in 64 bits outside the kernels: a central
    difference of step e is off by e^2 times the third derivative, and the
    float32 losses by 2e-6 of themselves over e."""
    n_seq, t_len, V, e = 4, 5, 300, 0.02
    z, x = make_rows(n_seq, t_len, V, F32, seed=9)
    z, x = z.to(DEV), x.to(DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    R = torch.randn(n_seq, t_len, device=DEV, generator=g)
    old = svp.token_logp(z, x)[0] + R * 0.05
    ref = old + R * 0.1
    w = torch.rand(n_seq, device=DEV, generator=g) + 0.5
    A = torch.randn(n_seq, device=DEV, generator=g)
    s = svp.token_logp(z, x)[0].sum(1) + torch.randn(n_seq, device=DEV, generator=g)
    calls = {
        "policy": lambda t, grad=True: svp.policy_loss(t, x, A, w, old_logp=old, ref_logp=ref, clip_low=0.9,
                                                       clip_high=9.0, kl_coef=0.3, entropy_coef=0.05, grad=grad)[3:],
        "preference": lambda t, grad=True: svp.preference_loss(t, x, s, w[:2], beta=0.3, grad=grad)[2:],
    }
    for name, call in calls.items():
        _, d = call(z)
        for k in range(4):
            way = torch.randn(z.shape, device=DEV, generator=g)
            up, down = (call(z + f * e * way, False)[0].double().sum() for f in (1, -1))
            slope = (d.double() * way.double()).sum().item()
            size = (d.double().abs() * way.double().abs()).sum().item()
            assert abs((up - down).item() / (2 * e) - slope) < 2e-3 * size + 1e-4, (name, k)


# ---------------------------------------------------------------------------
# Layouts, places, streams and graphs
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("V,dtype", [(1003, F32), (1001, BF16), (20001, BF16), (70001, F32), (151936, BF16)])
@pytest.mark.parametrize("by,out_by", [(1, 0), (0, 1), (3, 3), (1, 2)])
def test_rows_at_any_alignment(V, dtype, by, out_by):
    z, x = make_rows(3, 2, V, dtype, seed=V + by)
    out = lambda: shifted(torch.full_like(z, 7.0), out_by)
    check_logp(z, x, 1.0, True, dev=shifted(z, by))
    o = out()
    assert run_policy(z, x, ent=0.01, out=o, dev=shifted(z, by))[4] is o
    o = out()
    z4, x4 = torch.cat([z, z[:1]]), torch.cat([x, x[:1]])
    o = shifted(torch.full_like(z4, 7.0), out_by)
    assert run_preference(z4, x4, out=o, dev=shifted(z4, by))[3] is o


@pytest.mark.parametrize("V,dtype", [(7, F32), (1003, F32), (16384, BF16), (20001, BF16), (128256, BF16), (151936, F32)])
def test_gradients_in_place_of_the_logits(V, dtype):
    z, x = make_rows(4, 3, V, dtype, seed=V)
    a = z.to(DEV)
    run_policy(z, x, kl=0.1, out=a, dev=a)
    a = z.to(DEV)
    run_preference(z, x, out=a, dev=a)
    a, xd = z.to(DEV), x.to(DEV)
    logp, H, lse = svp.token_logp(a, xd, entropy=True)
    d = torch.randn(x.shape, generator=gen(2)).to(DEV)
    apart = svp.token_logp_grad(a, xd, logp, lse, d, entropy=H, d_entropy=d)
    here = svp.token_logp_grad(a, xd, logp, lse, d, entropy=H, d_entropy=d, out=a)
    assert here is a and torch.equal(apart, here)


def test_overlaps_are_refused():
    z, x = make_rows(2, 2, 64, F32)
    flat = torch.zeros(2 * z.numel(), device=DEV)
    a, b = flat[:z.numel()].view(z.shape).copy_(z), flat[64:64 + z.numel()].view(z.shape)
    w = torch.ones(2, device=DEV)
    with pytest.raises(svp.SpecVerifyError, match="INVALID_ARG"):
        svp.policy_loss(a, x.to(DEV), w, w, out=b)
    with pytest.raises(svp.SpecVerifyError, match="INVALID_ARG"):
        svp.preference_loss(a, x.to(DEV), w, w[:1], out=b)
    with pytest.raises(ValueError, match="pairs"):
        svp.preference_loss(a[:1], x[:1].to(DEV), w[:1], w[:0])
    with pytest.raises(ValueError, match="ref_logp"):
        svp.policy_loss(a, x.to(DEV), w, w, kl_coef=0.1)
    with pytest.raises(ValueError, match="contiguous"):
        svp.token_logp(a.transpose(0, 1), x.to(DEV))
    with pytest.raises(ValueError, match="shape"):
        svp.policy_loss(a, x.to(DEV), w[:1], w)
    with pytest.raises(ValueError, match="grad=False"):
        svp.policy_loss(a, x.to(DEV), w, w, grad=False, out=b)


def test_what_lies_around_the_outputs_stays():
    V, dtype = 5003, BF16
    z, x = make_rows(4, 3, V, dtype)
    n = z.numel()
    for by in (1, 8):
        flat = torch.full((n + 64,), 9.0, dtype=dtype, device=DEV)
        out = flat[by:by + n].view(z.shape)
        run_policy(z, x, out=out)
        assert (flat[:by] == 9).all() and (flat[by + n:] == 9).all()
        flat.fill_(9.0)
        run_preference(z, x, out=out)
        assert (flat[:by] == 9).all() and (flat[by + n:] == 9).all()


def everything(z, x, stream=None):
    w = torch.ones(z.shape[0], device=DEV)
    d = torch.linspace(-1, 1, x.numel(), device=DEV).view(x.shape)
    if stream is not None:
        stream.wait_stream(torch.cuda.current_stream())
    logp, H, lse = svp.token_logp(z, x, 0.9, entropy=True, stream=stream)
    g = svp.token_logp_grad(z, x, logp, lse, d, entropy=H, d_entropy=d, temperature=0.9, stream=stream)
    p = svp.policy_loss(z, x, w, w, old_logp=logp, ref_logp=lse, temperature=0.9, kl_coef=1e-3, entropy_coef=0.1, stream=stream)
    q = svp.preference_loss(z, x, lse.new_zeros(z.shape[0]) if stream is None else torch.zeros_like(w), w[::2].contiguous(),
                            temperature=0.9, stream=stream)
    return [logp, H, lse, g, *p, *q]


@pytest.mark.parametrize("V,dtype", [(3001, F32), (128256, BF16)])
def test_the_same_bits_on_any_stream_and_in_graphs(V, dtype):
    z, x = (t.to(DEV) for t in make_rows(4, 6, V, dtype, seed=3))
    want = everything(z, x)
    again = everything(z, x)
    side = torch.cuda.Stream()
    on_side = everything(z, x, side)
    side.synchronize()
    graphs, outs = [], []
    for _ in range(2):                        # two graphs, each with a workspace of its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(everything(z, x))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(5)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):     # side by side
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got in (again, on_side, *outs):
            for a, b in zip(want, got):
                assert torch.equal(a, b)


def test_many_rows():
    """More rows than a grid's other dimensions would take; short ones, of
    which only a few are compared."""
    n = 70000
    z = torch.randn(n, 1, 24, generator=gen(1), dtype=F32).to(DEV)
    x = torch.randint(-1, 24, (n, 1), generator=gen(2)).to(torch.int32).to(DEV)
    w = torch.ones(n, device=DEV)
    _, _, _, loss, grad = svp.policy_loss(z, x, w, w)
    lp = torch.log_softmax(z.double(), 2)
    want = lp.exp()
    want.scatter_add_(2, x.clamp(min=0).long()[..., None], -torch.ones(n, 1, 1, dtype=torch.float64, device=DEV))
    want = torch.where((x >= 0)[..., None], want, 0.0)
    assert (grad.double() - want).abs().max() < 4 * REL
    assert torch.equal(loss, -(x[:, 0] >= 0).float())


def test_offsets_past_32_bits():
    """Rows of 1 MiB whose bytes lie past 2^32 and whose elements lie past 2^31."""
    V, n = 524288, 4200
    z = torch.empty(2, n // 2, V, dtype=BF16, device=DEV)
    z.fill_(1.0)
    x = torch.full((2, n // 2), -1, dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    z[1, -1] = torch.randn(V, device=DEV, generator=g) * 3
    x[1, -1] = V - 1
    w = torch.ones(2, device=DEV)
    R = Rows(z[1:, -1:].cpu(), x[1:, -1:].cpu(), 1.0)
    logp, _, lse = svp.token_logp(z, x)
    assert_close(logp[1:, -1:], R.logp, R.tol_logp)
    for grad in (svp.policy_loss(z, x, w, w)[4], svp.preference_loss(z, x, w, w[:1], beta=1e-9, kind="hinge", grad=True)[3] / 1e-9):
        ref, tol = R.gradient(-np.ones(1), np.zeros(1), np.zeros(1))
        if (grad[1, -1, -1] > 0):             # the rejected sequence's gradient has the other sign
            ref = -ref
        assert_close(grad[1:, -1:], ref, tol + 2.0 ** -7 * np.abs(ref), BF16)
        assert (grad[0, 0] == 0).all() and (grad[1, -2] == 0).all()
        del grad


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("V,dtype", [(17000, BF16), (9001, F32)])
def test_more_rows_than_are_looked_at_together(V, dtype, entropy):
    """Padded rollouts of more rows than a window of tokens holds, on rows that
    are streamed: every row's numbers, and every gradient, in 64 bits."""
    n_seq, t_len = 3, 6700
    g = torch.Generator(device=DEV).manual_seed(1)
    z = (torch.randn(n_seq, t_len, V, device=DEV, generator=g, dtype=F32) * 2).to(dtype)
    x = torch.randint(0, V, (n_seq, t_len), device=DEV, generator=g).to(torch.int32)
    x[0, 1500:] = -1
    x[1, :4000] = -1
    x[2][torch.rand(t_len, device=DEV, generator=g) < 0.5] = -1
    A = torch.randn(n_seq, t_len, device=DEV, generator=g)
    w = torch.ones(n_seq, device=DEV)
    logp, H, row_loss, loss, grad = svp.policy_loss(z, x, A, w, entropy_coef=0.1 if entropy else 0.0)
    again = svp.token_logp(z, x, entropy=entropy)
    have = x >= 0
    for b in range(n_seq):
        for a in range(0, t_len, 500):
            at = slice(a, a + 500)
            zz, live = z[b, at].double(), have[b, at]
            lp = torch.log_softmax(zz, 1)
            p = lp.exp()
            tok = x[b, at].long().clamp(min=0)[:, None]
            lpx = torch.where(live, lp.gather(1, tok)[:, 0], 0.0)
            ent = torch.where(live, -(p * lp).sum(1), 0.0)
            assert (logp[b, at] - lpx).abs().max() < 2 * REL and (again[0][b, at] - lpx).abs().max() < 2 * REL
            lse = torch.where(live, torch.logsumexp(zz, 1), -INF)
            assert (again[2][b, at].double() - lse).nan_to_num(0.0).abs().max() < 2 * REL
            gg = -A[b, at].double()
            d = -p * gg[:, None]
            d.scatter_add_(1, tok, gg[:, None])
            if entropy:
                assert (H[b, at] - ent).abs().max() < 10 * REL * (1 + ent.abs().max())
                d = d + 0.1 * p * (lp + ent[:, None])
            d = torch.where(live[:, None], d, 0.0)
            got = grad[b, at].double()
            # float32: 4 REL of the two parts' sizes; bf16 half a step more
            size = p * gg.abs()[:, None] + (0.1 * p * (lp.abs() + ent[:, None] + 1) if entropy else 0.0)
            size.scatter_add_(1, tok, gg.abs()[:, None] * (1 - p.gather(1, tok)))
            assert ((got - d).abs() <= 4 * REL * size + (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * d.abs() * 1.001 + 1e-37).all()
    assert torch.equal(loss, row_loss.double().sum(1).float()) or (loss - row_loss.double().sum(1)).abs().max() < 1e-3


@pytest.mark.parametrize("V,dtype,n", [(128256, BF16, 8500), (60001, F32, 9000)])
def test_a_row_is_the_same_whatever_rows_lie_around_it(V, dtype, n):
    """Rows of clusters of several CTAs, more of them than a window of tokens
    holds, against the same rows in calls of their own: the same bits."""
    g = torch.Generator(device=DEV).manual_seed(2)
    z = torch.empty(n, 1, V, dtype=dtype, device=DEV)
    for a in range(0, n, 500):
        z[a:a + 500] = torch.randn(min(500, n - a), 1, V, device=DEV, generator=g)
    x = torch.randint(0, V, (n, 1), device=DEV, generator=g).to(torch.int32)
    x[torch.rand(n, 1, device=DEV, generator=g) < 0.3] = -1
    x[:40] = -1
    A, w = torch.randn(n, device=DEV, generator=g), torch.ones(n, device=DEV)
    whole = svp.policy_loss(z, x, A, w, entropy_coef=0.01)
    sums = svp.token_logp(z, x, entropy=True)
    m = n // 2 + 7
    for at in (slice(0, m), slice(m, n)):
        part = svp.policy_loss(z[at], x[at], A[at], w[at], entropy_coef=0.01)
        for a, b in zip(whole, part):
            assert torch.equal(a[at], b)
        for a, b in zip(sums, svp.token_logp(z[at], x[at], entropy=True)):
            assert torch.equal(a[at], b)
    d = torch.randn(n, 1, device=DEV, generator=g)
    logp, H, lse = sums
    grad = svp.token_logp_grad(z, x, logp, lse, d, entropy=H, d_entropy=d, out=whole[4])
    here = svp.token_logp_grad(z, x, logp, lse, d, entropy=H, d_entropy=d, out=z)
    assert torch.equal(grad, here)


# ---------------------------------------------------------------------------
# Waits that expire
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("V,dtype", [(20000, BF16), (128256, BF16), (151936, F32)])
def test_an_expired_wait_gives_nan_and_leaves_the_next_call_alone(V, dtype):
    z, x = make_rows(6, 30, V, dtype, seed=1)
    zd, xd, w = z.to(DEV), x.to(DEV), torch.ones(6, device=DEV)
    want = svp.policy_loss(zd, xd, w, w)
    lib = svp.load_library()
    live = (x >= 0).to(DEV)
    try:
        assert lib.spec_kd_set_wait_limit_ns(0) == svp.SV_OK
        logp, _, row_loss, loss, grad = svp.policy_loss(zd, xd, w, w)
        alone = svp.token_logp(zd, xd, entropy=True)
        torch.cuda.synchronize()
    finally:
        lib.spec_kd_set_wait_limit_ns(-1)
    for t in (logp, row_loss, *alone):
        assert t[live].isnan().all()
    assert (logp[~live] == 0).all() and (row_loss[~live] == 0).all() and (alone[2][~live] == -INF).all()
    assert loss[live.any(1)].isnan().all()
    assert grad[live].isnan().all() and (grad[~live] == 0).all()
    for a, b in zip(want, svp.policy_loss(zd, xd, w, w)):
        assert (a is None and b is None) or torch.equal(a, b)


def test_a_first_call_can_be_captured():
    """In a process of its own: nothing has been launched before the capture."""
    import subprocess
    import sys
    code = """
import torch, speculative_decoding_verification_71_gb300 as svp
z = torch.randn(3, 4, 70001, device="cuda"); x = torch.randint(0, 70001, (3, 4), device="cuda").to(torch.int32)
w = torch.ones(3, device="cuda"); y = z[:2, :, :3001].contiguous(); g = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(g):
    a = svp.policy_loss(z, x, w, w, entropy_coef=0.1)
    b = svp.preference_loss(y, x[:2] % 3001, w[:2], w[:1])
    c = svp.clip_gradients([z], 1e9)
g.replay(); torch.cuda.synchronize()
d = svp.policy_loss(z, x, w, w, entropy_coef=0.1)
assert all(torch.equal(p, q) for p, q in zip(a, d)) and a[4].abs().max() > 0 and b[3].abs().max() > 0 and c.item() > 0
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=root)
    assert "captured" in out.stdout, out.stderr[-2000:]
