"""kd_top and kd_top_loss against their definitions in 64 bits.

Tolerances, from the arithmetic: exponentials are ex2.approx (2^-22) of an
argument rounded once, sums are fp32, at most a few hundred terms long per
thread and then pairwise (1e-6 to 1e-5 of the sum); c = fl(log2(e) / T) shifts
log p(x) by 2^-24 |z - z'| / T.
  * logp, lse: 1e-5 + 5e-7 |value|;  the listed ids are exact;
  * the row KL: 1e-5 (1 + sum p |log p - log q|) + 2e-6 (1 + |log r - log(1 - Q)|)
    + 1e-6: the second part is r = 1 - P, whose sum of up to 256 fp32 terms is
    off by up to 2e-6;
  * the gradient: w / T times 1e-5 (p + q + q r / (1 - Q)) + 2e-6 q / (1 - Q),
    bf16 one step (2^-7 of the value) more.
"""
import math

import numpy as np
import pytest
import torch

import speculative_decoding_verification_71_gb300 as svp
from speculative_decoding_verification_71_gb300 import build as svbuild

pytestmark = pytest.mark.gpu
DEV = "cuda"
INF = float("inf")
FLT_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _built():
    svbuild.build()
    svp.load_library()


# ---------------------------------------------------------------------------
# kd_top
# ---------------------------------------------------------------------------

def top_reference(row, K, T):
    z = row.double().numpy()
    if np.isnan(z).any() or (z == np.inf).any():
        return [-1] * K, [math.nan] * K, math.nan
    if (z == -np.inf).all():
        return [-1] * K, [math.nan] * K, -math.inf
    m = z.max()
    log_sum = math.log(np.exp((z - m) / T).sum())
    order = np.lexsort((np.arange(len(z)), -z))[:K]
    ids = [int(i) if z[i] > -np.inf else -1 for i in order] + [-1] * (K - len(order))
    logp = [(z[i] - m) / T - log_sum if i >= 0 else -np.inf for i in ids]
    return ids, logp, m / T + log_sum


def check_top(t, K, T=1.0, n_rows=None, dev=None):
    n_seq, t_len, V = t.shape
    ids, logp, lse = svp.kd_top(t.to(DEV) if dev is None else dev, K, T,
                                n_rows=None if n_rows is None else torch.tensor(n_rows, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert ids.shape == logp.shape == (n_seq, t_len, K) and lse.shape == (n_seq, t_len)
    ids, logp, lse = ids.cpu().numpy(), logp.cpu().double().numpy(), lse.cpu().double().numpy()
    for b in range(n_seq):
        for i in range(t_len):
            if n_rows is not None and i >= n_rows[b]:
                want = [-1] * K, [-math.inf] * K, -math.inf
            else:
                want = top_reference(t[b, i], K, T)
            assert ids[b, i].tolist() == want[0], (b, i)
            for got, ref in ((logp[b, i], np.array(want[1])), (lse[b, i:i + 1], np.array([want[2]]))):
                fin = np.isfinite(ref)
                assert np.array_equal(got[~fin], ref[~fin], equal_nan=True), (b, i)
                assert (np.abs(got - ref)[fin] <= 1e-5 + 5e-7 * np.abs(ref[fin])).all(), (b, i, np.abs(got - ref)[fin].max())


def randn(*shape, seed=0, scale=3.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype)


TOP_CASES = [  # n_seq, t_len, V, dtype, K, T
    (1, 1, 1, torch.float32, 1, 1.0),
    (2, 2, 5, torch.bfloat16, 8, 1.0),          # more places than tokens
    (3, 1, 100, torch.float32, 100, 0.7),       # every token
    (2, 3, 1000, torch.bfloat16, 1, 1.0),
    (2, 2, 4099, torch.float32, 20, 0.6),
    (2, 2, 4099, torch.bfloat16, 256, 1.3),
    (1, 3, 20000, torch.bfloat16, 64, 1.0),
    (1, 1, 151936, torch.bfloat16, 20, 1.0),
    (2, 2, 128256, torch.bfloat16, 256, 1.0),
    (1, 2, 50001, torch.float32, 255, 0.8),
    (1, 1, 600001, torch.float32, 33, 1.0),
    (40, 8, 3000, torch.bfloat16, 64, 1.0),     # more rows than SMs
    (400, 2, 777, torch.float32, 17, 1.0),
]


@pytest.mark.parametrize("n_seq,t_len,V,dtype,K,T", TOP_CASES,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-{str(c[3])[6:]}-K{c[4]}" for c in TOP_CASES])
def test_top_matches_the_definition(n_seq, t_len, V, dtype, K, T):
    check_top(randn(n_seq, t_len, V, seed=V, dtype=dtype), K, T)


@pytest.mark.parametrize("V,dtype,K", [(262147, torch.float32, 256), (262147, torch.float32, 64),
                                       (200003, torch.bfloat16, 256), (140001, torch.float32, 200)])
def test_top_of_long_rows_that_are_not_split(V, dtype, K):
    check_top(randn(6, 3 if K > 128 else 26, V, seed=V + K, dtype=dtype), K)


@pytest.mark.parametrize("V,dtype,K,rows", [(300001, torch.float32, 64, 90), (300001, torch.float32, 200, 90),
                                            (700001, torch.float32, 256, 2), (700001, torch.bfloat16, 128, 40)])
def test_top_of_long_rows_that_are_split(V, dtype, K, rows):
    check_top(randn(rows, 1, V, seed=V + K, dtype=dtype), K)


@pytest.mark.parametrize("V,dtype,K", [(262147, torch.float32, 256), (262147, torch.float32, 65), (140001, torch.float32, 200),
                                       (200003, torch.bfloat16, 256), (200003, torch.bfloat16, 64)])
def test_top_of_more_long_rows_than_are_split(V, dtype, K):
    check_top_rows(randn(7, V, seed=V + K, dtype=dtype), K, 1.0, times=23)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [129, 200, 256])
@pytest.mark.parametrize("V", [257, 1100, 4001, 8190])
def test_top_of_short_rows_with_long_lists(V, K, dtype):
    check_top(randn(7, 3, V, seed=V + K, dtype=dtype), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("K", [1, 20, 64, 256])
@pytest.mark.parametrize("V", [300, 9001, 70000])
def test_top_of_rows_in_every_order(V, K, dtype):
    r = torch.arange(V, dtype=torch.float32)
    rows = [
        r / V * 30,                                     # ascending: every tile beats the ones before
        -r / V * 30,                                    # descending
        torch.zeros(V),                                 # one value: ties go to the lowest ids
        (r % 7).round(),                                # seven values
        torch.where(r < V // 2, 0.0, -0.0),             # 0 and -0 are one value
        randn(V, seed=1).round(),
        torch.where(r == V - 1, 5.0, -3.0),             # the largest comes last
        torch.cat([torch.full((V - V // 3,), -20.0), randn(V // 3, seed=2)]),   # all the mass at the end
    ]
    check_top(torch.stack(rows)[:, None].to(dtype), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [50, 5001, 140001])
def test_top_of_masked_and_invalid_rows(V, dtype):
    low = torch.finfo(dtype).min
    z = randn(12, 1, V, seed=3, dtype=dtype)
    z[0] = -INF                                          # nothing is left
    z[1, 0, 1:] = -INF                                   # one token
    z[2, 0, :-1] = -INF                                  # one token, the last
    z[3, 0, 7:] = -INF                                   # fewer than K
    z[4, 0, 3:] = low                                    # the type's lowest value in place of -inf
    z[5, 0, V // 2] = float("nan")
    z[6, 0, V - 1] = INF
    z[7] = low
    z[8, 0, ::2] = -INF
    z[9, 0, 0], z[9, 0, -1] = INF, -INF
    z[10, 0, : V - 10] = low
    z[11, 0, 0] = float("nan")
    z[11, 0, 1:] = -INF
    for K in (1, 16, 64):
        check_top(z, K)


# Rows far from 0.  The sum is of 2^((z - M) c) at any level, so the bounds at
# the head of this file hold; a value that passes float32's range is infinite.
LEVELS = [x * s for x in (1e6, 2e7, 1e8, 1e9, 1e10, 1e12, 1e30, 2.4e38, 3e38) for s in (1.0, -1.0)] + ["lowest"]


def rows_at(level, V, dtype):
    """[7, V]: rows of one level, of levels near it, and with ordinary logits
    beside it."""
    at = torch.finfo(dtype).min if level == "lowest" else level
    r = torch.arange(V, dtype=torch.float32)
    z = randn(7, V, seed=V, dtype=dtype)
    z[0] = at                                                # everything
    z[1, V // 3] = at                                        # one token: forced, or alone masked
    z[2, V // 4:V // 2] = at                                 # a block
    z[3] = at if level == "lowest" else (at * (1 + (r * 7 % 13).floor() / 128)).to(dtype)
    z[4] = at                                                # all but a few, as behind a narrow mask
    few = (torch.arange(5) * 2357 + 11) % V
    z[4, few] = randn(5, seed=8, dtype=dtype)
    z[5] = torch.finfo(dtype).min if abs(at) < 1e31 else 0.0  # a token at that level, the rest masked
    z[5, V - 1] = at
    z[6] = -INF
    z[6, ::2] = at
    return z


def check_top_rows(z, K, T, times=1):
    """Rows [n, V], `times` times over in one call, against the definition rounded to float32."""
    n, V = z.shape
    ids, logp, lse = (x.cpu().numpy() for x in svp.kd_top(z.repeat(times, 1)[:, None].to(DEV), K, T))
    for i in range(n):
        x = z[i].double().numpy()
        m = x.max()
        log_sum = math.log(np.exp((x - m) / T).sum())
        order = np.argsort(-x, kind="stable")[:K]
        kept = x[order] > -np.inf
        want_ids = np.concatenate([np.where(kept, order, -1), np.full(K - len(order), -1)])
        want = np.concatenate([np.where(kept, (x[order] - m) / T - log_sum, -np.inf), np.full(K - len(order), -np.inf)])
        for j in range(i, n * times, n):
            assert np.array_equal(ids[j, 0], want_ids), (i, j)
            with np.errstate(over="ignore"):
                for got, ref in ((logp[j, 0], want), (lse[j], np.array([m / T + log_sum]))):
                    near = np.isfinite(ref.astype(np.float32)) & np.isfinite(got)
                    same = got == ref.astype(np.float32)
                    off = np.abs(np.where(near, got.astype(np.float64) - np.where(near, ref, 0), 0))
                    assert (same | near).all() and (off <= 1e-5 + 5e-7 * np.abs(np.where(near, ref, 0))).all(), (i, j, got[:4], ref[:4])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.6, 0.7, 0.8, 1.0, 1.3, 1.5, 2.0, 4.0])
def test_top_of_rows_at_any_level(T, dtype):
    for V in (50, 1003, 20001):
        for level in LEVELS:
            check_top_rows(rows_at(level, V, dtype), 20, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,level", [(0.6, -1e9), (0.8, -1e10), (1.0, -1e30), (1.0, 1e10), (1.0, 3e38), (1.5, "lowest"),
                                     (1.5, -1e30), (4.0, "lowest"), (2.0, -1e12)])
def test_top_of_long_rows_at_any_level(T, level, dtype):
    z = rows_at(level, 140001, dtype)
    check_top_rows(z, 20, T)                 # a cluster of 8 CTAs to a row
    check_top_rows(z, 200, T, times=4)       # of 4
    check_top_rows(z, 64, T, times=24)       # a CTA to a row


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1.0, 1.7, 2.0, 4.0, 100.0])
def test_top_of_rows_as_wide_as_the_type(T, dtype):
    # z - M passes the range, (z - M) / T need not
    for V in (9, 3000):
        z = torch.zeros(3, V, dtype=dtype)
        z[0], z[0, 2] = torch.finfo(dtype).min, 3e38
        z[1, ::2], z[1, 1::2] = -2e38, 2e38
        z[2, 0], z[2, 1] = torch.finfo(dtype).max, torch.finfo(dtype).min
        check_top_rows(z, 9, T)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_top_of_invalid_rows_at_any_level(dtype):
    for V in (50, 20001, 140001):
        z = torch.stack([torch.full((V,), x) for x in (1e10, -1e30, 3e38, -3e38, 0.0)]).to(dtype)
        z[0, V // 2] = z[1, V - 1] = z[2, 0] = float("nan")
        z[3, V // 3] = z[4, V - 1] = INF
        ids, logp, lse = svp.kd_top(z[:, None].contiguous().to(DEV), 10)
        assert (ids == -1).all() and logp.isnan().all() and lse.isnan().all()


def test_top_rows_past_a_sequences_own_are_not_read():
    z = randn(5, 4, 2003, seed=4, dtype=torch.bfloat16)
    n = [0, 1, 4, 2, 9]
    for b in range(5):
        z[b, min(n[b], 4):] = float("nan")
    check_top(z, 30, n_rows=n)
    check_top(z[:1, :1], 30, n_rows=[-3])


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1), (torch.float32, 3), (torch.bfloat16, 1), (torch.bfloat16, 6)])
def test_top_of_rows_off_the_16_byte_boundary(dtype, shift):
    z = randn(3, 2, 6000, seed=5, dtype=dtype)
    dev = torch.full((z.numel() + 16,), INF, dtype=dtype, device=DEV)[shift:shift + z.numel()].view(z.shape)
    dev.copy_(z)
    check_top(z, 50, dev=dev)


def test_top_is_deterministic_and_stream_ordered():
    z = randn(64, 2, 30011, seed=6, dtype=torch.bfloat16).to(DEV)
    want = svp.kd_top(z, 100)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s, s):
        got = svp.kd_top(z, 100, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.slow
def test_top_of_rows_past_32_bit_offsets():
    z = torch.zeros(16800, 1, 128256, dtype=torch.bfloat16, device=DEV)
    tail = randn(2, 1, 128256, seed=7, dtype=torch.bfloat16)
    z[-2:] = tail.to(DEV)
    ids, logp, _ = svp.kd_top(z, 40)
    torch.cuda.synchronize()
    for b in range(2):
        want = top_reference(tail[b, 0], 40, 1.0)
        assert ids[b - 2, 0].tolist() == want[0]
    assert ids[5, 0].tolist() == list(range(40))


# ---------------------------------------------------------------------------
# kd_top_loss
# ---------------------------------------------------------------------------

def loss_reference(ids, lp, z, w, T, tail):
    """One row in 64 bits: (KL, gradient, KL tolerance, gradient tolerance)."""
    z = z.double().numpy()
    V = len(z)
    lp = lp.double().numpy()
    ids = ids.numpy()
    nan = math.nan, np.full(V, math.nan), 0.0, np.zeros(V)
    if np.isnan(lp).any() or (lp == np.inf).any() or (ids >= V).any():
        return nan
    used = ids >= 0
    x, lp = ids[used], lp[used]
    if not used.any():
        return 0.0, np.zeros(V), 0.0, np.zeros(V)
    if len(set(x.tolist())) < len(x) or np.isnan(z).any() or (z == np.inf).any() or (z == -np.inf).all():
        return nan
    m = z.max()
    lq = (z - m) / T - math.log(np.exp((z - m) / T).sum())
    q = np.exp(lq)
    p = np.exp(lp)
    r = 0.0
    if tail:
        r = 1 - p.sum()
        r = 0.0 if r < 2.0 ** -20 else r
    else:
        lp = lp - math.log(p.sum()) if p.sum() > 0 else lp
        p = p / p.sum() if p.sum() > 0 else p
    others = np.ones(V, bool)
    others[x] = False
    lrest = -math.inf                     # log(1 - Q), also where 1 - Q underflows
    if others.any() and lq[others].max() > -np.inf:
        top = lq[others].max()
        lrest = top + math.log(np.exp(lq[others] - top).sum())
    on = p > 0
    kl = float((p[on] * (lp[on] - lq[x][on])).sum())
    spread = float((p[on] * np.abs(lp[on] - lq[x][on])).sum())
    grad, share, odds = q.copy(), np.zeros(V), 0.0
    if r > 0:
        kl = kl + r * (math.log(r) - lrest)
        odds = abs(math.log(r) - lrest)
    if lrest > -math.inf:
        share[others] = np.exp(lq[others] - lrest)
    with np.errstate(over="ignore"):
        kl = math.inf if np.isinf(np.float32(kl)) else kl
    grad -= r * share
    grad[x] -= p
    s = w / T
    gt = 1e-5 * (q + r * share) + 2e-6 * share
    gt[x] += 1e-5 * p
    return kl, s * grad, (1e-5 * (1 + spread) + 2e-6 * (1 + odds) + 1e-6) if math.isfinite(kl) else 0.0, s * gt + 1e-30


def check_loss(ids, lp, z, w, T=1.0, tail=True, dev=None):
    n_seq, t_len, V = z.shape
    d = z.to(DEV) if dev is None else dev
    kl, loss, grad = svp.kd_top_loss(ids.to(DEV), lp.to(DEV), d, w.to(DEV), T, tail=tail)
    kl2, loss2, none = svp.kd_top_loss(ids.to(DEV), lp.to(DEV), d, w.to(DEV), T, tail=tail, grad=False)
    torch.cuda.synchronize()
    assert none is None
    assert torch.equal(kl.nan_to_num(1e9), kl2.nan_to_num(1e9)) and torch.equal(loss.nan_to_num(1e9), loss2.nan_to_num(1e9))
    kl, loss, g = kl.cpu().double().numpy(), loss.cpu().double().numpy(), grad.cpu().double().numpy()
    for b in range(n_seq):
        total, slack = 0.0, 1e-6
        for i in range(t_len):
            ref, rg, tol, gt = loss_reference(ids[b, i], lp[b, i], z[b, i], float(w[b]), T, tail)
            if math.isfinite(ref):
                assert abs(kl[b, i] - ref) <= tol, (b, i, kl[b, i], ref, tol)
            else:
                assert np.array_equal(kl[b, i], ref, equal_nan=True), (b, i, kl[b, i], ref)
            if z.dtype == torch.bfloat16:
                gt = gt + np.abs(rg) * 2.0 ** -7 + 1e-37
            bad = np.isnan(rg)
            assert np.array_equal(np.isnan(g[b, i]), bad), (b, i)
            assert (np.abs(g[b, i] - rg)[~bad] <= gt[~bad]).all(), (b, i, (np.abs(g[b, i] - rg) - gt)[~bad].max())
            total, slack = total + ref, slack + tol
        want = float(w[b]) * total
        if abs(want) <= FLT_MAX:
            assert abs(loss[b] - want) <= float(w[b]) * slack + 1e-6
        else:
            assert not math.isfinite(loss[b])
    return kl, loss, g


def lists(teacher, K, T):
    z = teacher.float().double() / T
    top = z.sort(dim=2, descending=True, stable=True)
    lp = top.values[:, :, :K] - torch.logsumexp(z, 2, keepdim=True)
    return top.indices[:, :, :K].to(torch.int32).contiguous(), lp.float().contiguous()


def pair(n_seq, t_len, V, dtype, K, T, seed=0, noise=0.7):
    t = randn(n_seq, t_len, V, seed=seed)
    z = (t + randn(n_seq, t_len, V, seed=seed + 1, scale=noise)).to(dtype)
    w = torch.rand(n_seq, generator=torch.Generator().manual_seed(seed + 2)) * 2
    return (*lists(t, K, T), z, w)


LOSS_CASES = [  # n_seq, t_len, V, dtype, K, T
    (1, 1, 2, torch.float32, 1, 1.0),
    (2, 3, 9, torch.bfloat16, 4, 1.0),
    (1, 2, 64, torch.float32, 64, 1.0),          # the list is complete
    (2, 2, 1000, torch.float32, 20, 0.7),
    (2, 2, 4099, torch.bfloat16, 256, 1.3),
    (1, 3, 4099, torch.float32, 33, 1.0),
    (2, 2, 20000, torch.bfloat16, 64, 1.0),
    (1, 2, 151936, torch.bfloat16, 64, 1.0),
    (1, 2, 128256, torch.bfloat16, 1, 0.6),
    (1, 2, 50001, torch.float32, 128, 0.8),
    (1, 1, 151936, torch.float32, 20, 1.0),
    (1, 1, 524288, torch.bfloat16, 100, 1.0),
    (60, 6, 1500, torch.bfloat16, 16, 1.0),      # more rows than SMs
    (170, 2, 613, torch.float32, 40, 1.0),
]


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("n_seq,t_len,V,dtype,K,T", LOSS_CASES,
                         ids=[f"{c[0]}x{c[1]}x{c[2]}-{str(c[3])[6:]}-K{c[4]}" for c in LOSS_CASES])
def test_loss_matches_the_definition(n_seq, t_len, V, dtype, K, T, tail):
    check_loss(*pair(n_seq, t_len, V, dtype, K, T, seed=V), T, tail)


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, V) for V in (4072, 4073, 8175, 8177, 16360, 16367, 16369)] +
                         [(torch.float32, V) for V in (2035, 2041, 4085, 4091, 8181, 8185)])
def test_loss_where_the_row_length_changes_the_kernel(dtype, V, tail):
    check_loss(*pair(3, 3, V, dtype, 70, 0.9, seed=V), 0.9, tail)


# the longest rows of a kernel and the shortest of the next: 512, 1024 and 2048
# vectors with the two that a row off the 16-byte boundary takes more
@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("dtype,V", [(torch.bfloat16, V) for V in (4087, 4088, 8183, 8184, 16375, 16376, 16377)] +
                         [(torch.float32, V) for V in (2043, 2044, 4091, 4092, 8187, 8188, 8189)])
def test_loss_on_both_sides_of_a_change_of_kernel(dtype, V, tail):
    check_loss(*pair(3, 3, V, dtype, 70, 0.9, seed=V), 0.9, tail)


@pytest.mark.parametrize("n_seq,t_len", [(1, 1500), (3, 257), (9, 256), (300, 1)])
def test_loss_of_few_and_many_positions(n_seq, t_len):
    check_loss(*pair(n_seq, t_len, 130, torch.float32, 8, 1.0, seed=n_seq), 1.0, True)


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [333, 40001])
def test_loss_of_unusual_rows(V, dtype, tail):
    K = 24
    ids, lp, z, w = pair(16, 1, V, dtype, K, 1.0, seed=50)
    low = torch.finfo(dtype).min
    ids[0], lp[0] = -1, -INF                              # no list
    ids[1, 0, 5:], lp[1, 0, 5:] = -1, -INF                # a short one
    ids[2, 0, ::2] = -1                                   # holes
    lp[3, 0, 4:] = -INF                                   # listed, without mass
    z[4, 0, 1::2] = -INF                                  # half the draft masked
    z[5, 0, :] = -INF                                     # nothing left: invalid
    z[6, 0, int(ids[6, 0, 3])] = float("nan")             # NaN in a listed place
    z[7, 0, V - 1] = INF
    lp[8, 0, 2] = float("nan")
    ids[9, 0, 1] = ids[9, 0, 0]                           # listed twice
    ids[10, 0, 0] = V                                     # no such token
    mask = torch.ones(V, dtype=torch.bool)
    mask[ids[11, 0].long()] = False
    z[11, 0, mask] = -INF                                 # the draft has nothing else
    z[12, 0, mask] = low                                  # ... and with the lowest value
    z[13, 0, int(ids[13, 0, 0])] = 60.0                   # the draft is sure of one
    z[14, 0, ~mask] -= 200.0                              # listed tokens underflow against the others
    ids[15, 0, 1:], lp[15, 0, 1:] = -1, -INF              # one token, all the mass
    lp[15, 0, 0] = 0.0
    check_loss(ids, lp, z, w, 1.0, tail)


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [60, 40001])
def test_loss_of_rows_as_wide_as_the_type(V, dtype, tail):
    # a draft logit and the row's maximum whose difference passes the range,
    # which a T above 1 brings back into it
    T, K = 8.0, 6
    ids, lp, z, w = pair(4, 1, V, dtype, K, T, seed=130)
    low = torch.finfo(dtype).min
    z[0], z[0, 0, int(ids[0, 0, 0])] = low, 3e38          # one listed token, the rest far below
    z[1, 0, int(ids[1, 0, 1])] = low                      # a listed token far below an unlisted one
    z[1, 0, next(x for x in range(V) if x not in ids[1, 0].tolist())] = 3e38
    z[2, 0, int(ids[2, 0, 0])], z[2, 0, int(ids[2, 0, 1])] = -2e38, 2e38
    kl, _, grad = (x.cpu().double().numpy() for x in svp.kd_top_loss(ids.to(DEV), lp.to(DEV), z.to(DEV), w.to(DEV), T, tail=tail))
    for b in range(4):
        ref, _, tol, _ = loss_reference(ids[b, 0], lp[b, 0], z[b, 0], float(w[b]), T, tail)
        assert math.isfinite(ref) and abs(kl[b, 0] - ref) <= tol, (b, kl[b, 0], ref, tol)
        # the others' shares about their own maximum: log q of -1e38 has no digits left for them
        x, v = ids[b, 0].numpy(), z[b, 0].double().numpy()
        p = np.exp(lp[b, 0].double().numpy())
        r = 1 - p.sum() if tail else 0.0
        p = p if tail else p / p.sum()
        q, share = np.exp((v - v.max()) / T), np.exp(np.minimum(v - np.delete(v, x).max(), 0) / T)
        q, share[x] = q / q.sum(), 0.0
        share /= share.sum()
        want, bound = q - r * share, 1e-5 * (q + r * share) + 2e-6 * share
        want[x] -= p
        bound[x] += 1e-5 * p
        if dtype == torch.bfloat16:
            bound = bound + np.abs(want) * 2.0 ** -7
        s = float(w[b]) / T
        assert (np.abs(grad[b, 0] - s * want) <= s * bound + 1e-30).all(), (b, (np.abs(grad[b, 0] - s * want) - s * bound).max())


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [0.3, 0.6, 1.0, 2.0])
@pytest.mark.parametrize("V", [60, 40001])
def test_loss_of_a_draft_masked_with_the_lowest_value(V, T, dtype, tail):
    # (z - m) / T passes the range where T is below 1, its share of the KL does not
    K = 12
    ids, lp, z, w = pair(4, 1, V, dtype, K, 1.0, seed=180)
    lp = torch.log_softmax(torch.arange(K, 0, -1) * 0.9, 0).expand_as(lp).contiguous() - 0.1   # a tail of 0.1
    low = torch.finfo(dtype).min
    z[0, 0, ids[0, 0, 4:].long()] = low                   # some of the listed, with 0.03 of the mass
    z[1, 0, int(ids[1, 0, K - 1])] = low
    z[1, 0, int(ids[1, 0, K - 2])] = -INF                 # ... where nothing helps
    others = torch.ones(V, dtype=torch.bool)
    others[ids[2, 0].long()] = False
    z[2, 0, others] = low                                 # all the others, with a tenth of it
    lp[3, 0, 6:] = -300.0                                 # probability 0 in float32
    z[3, 0, ids[3, 0, 6:].long()] = low
    if T < 1:
        z[3, 0, ids[3, 0].long()] = 3e38                  # both far above 0
        z[3, 0, int(ids[3, 0, 5])] = 1.5e38               # probability 0.004
    kl, _, _ = (x.cpu().double().numpy() for x in svp.kd_top_loss(ids.to(DEV), lp.to(DEV), z.to(DEV), w.to(DEV), T, tail=tail))
    for b in range(4):
        with np.errstate(over="ignore"):
            ref, _, tol, _ = loss_reference(ids[b, 0], lp[b, 0], z[b, 0], float(w[b]), T, tail)
        assert math.isfinite(ref) == (b != 1)
        assert kl[b, 0] == ref if b == 1 else abs(kl[b, 0] - ref) <= tol, (b, kl[b, 0], ref, tol)


def test_rows_without_a_list_are_not_read():
    ids, lp, z, w = pair(4, 3, 2001, torch.bfloat16, 10, 1.0, seed=60)
    for b, n in enumerate((0, 1, 2, 3)):
        ids[b, n:], lp[b, n:], z[b, n:] = -1, -INF, float("nan")
    kl, loss, g = check_loss(ids, lp, z, w)
    assert (kl[0] == 0).all() and loss[0] == 0 and (g[0] == 0).all()


def test_the_full_list_is_the_full_divergence():
    t = randn(2, 3, 200, seed=70)
    z = t + randn(2, 3, 200, seed=71, scale=0.5)
    w = torch.tensor([1.0, 0.5])
    ids, lp = lists(t, 200, 0.9)
    kl, loss, g = svp.kd_top_loss(ids.to(DEV), lp.to(DEV), z.to(DEV), w.to(DEV), 0.9)
    kl2, loss2, g2 = svp.kd_loss(t.to(DEV), z.to(DEV), w.to(DEV), 0.9)
    torch.testing.assert_close(kl, kl2, rtol=0, atol=2e-5)
    torch.testing.assert_close(g, g2, rtol=0, atol=2e-5)


@pytest.mark.parametrize("tail", [True, False], ids=["tail", "renorm"])
@pytest.mark.parametrize("V,K", [(37, 5), (600, 12)])
def test_the_gradient_is_the_slope_of_the_loss(V, K, tail):
    # central differences of the operator's own loss along random directions of
    # size 1 a token: their truncation is h^2 / 6 of a third derivative below
    # 2 w / T^3 a row, the losses' rounding 1e-5 w / h
    T, h, rows = 1.3, 0.05, 3
    ids, lp, z, w = pair(1, rows, V, torch.float32, K, T, seed=80)
    w = torch.tensor([1.0])
    run = lambda x: svp.kd_top_loss(ids.to(DEV), lp.to(DEV), x.contiguous(), w.to(DEV), T, tail=tail)
    zd = z.to(DEV)
    g = run(zd)[2].double()
    for seed in range(6):
        d = (torch.rand(z.shape, generator=torch.Generator().manual_seed(seed)) * 2 - 1).to(DEV)
        up, down = run(zd + h * d)[1].double(), run(zd - h * d)[1].double()
        slope = ((up - down) / (2 * h)).item()
        assert abs(slope - (g * d).sum().item()) <= rows * (h * h / 3 / T ** 3 + 2e-5 / h)


@pytest.mark.parametrize("dtype,shift", [(torch.float32, 1), (torch.bfloat16, 1), (torch.bfloat16, 5)])
def test_loss_of_rows_off_the_16_byte_boundary(dtype, shift):
    ids, lp, z, w = pair(2, 2, 5003, dtype, 30, 1.0, seed=90)
    dev = torch.full((z.numel() + 16,), INF, dtype=dtype, device=DEV)[shift:shift + z.numel()].view(z.shape)
    dev.copy_(z)
    check_loss(ids, lp, z, w, dev=dev)


def test_loss_is_deterministic_and_stream_ordered():
    ids, lp, z, w = (x.to(DEV) for x in pair(8, 40, 20011, torch.bfloat16, 64, 1.0, seed=100))
    want = svp.kd_top_loss(ids, lp, z, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (None, s, s):
        got = svp.kd_top_loss(ids, lp, z, w, stream=stream)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.fixture
def wait_limit():
    lib = svp.load_library()
    yield lambda ns: lib.spec_kd_set_wait_limit_ns(ns)
    lib.spec_kd_set_wait_limit_ns(-1)


# rows of 8, 2 and 1 CTAs
@pytest.mark.parametrize("n_seq,t_len,V,dtype", [(3, 5, 140001, torch.bfloat16), (50, 8, 140001, torch.bfloat16),
                                                 (130, 3, 9001, torch.float32)])
@pytest.mark.parametrize("grad", [True, False], ids=["grad", "loss"])
def test_loss_where_every_wait_expires(n_seq, t_len, V, dtype, grad, wait_limit):
    g = torch.Generator(device=DEV).manual_seed(140)
    z = (torch.randn(n_seq, t_len, V, generator=g, device=DEV) * 3).to(dtype)
    ids, lp, _ = svp.kd_top(z.flip(2).contiguous(), 12)
    ids[1, 0], lp[1, 0] = -1, -INF                       # no list: nothing is waited for
    w = torch.ones(n_seq, device=DEV)
    want = svp.kd_top_loss(ids, lp, z, w, grad=grad)
    wait_limit(0)
    kl, loss, gr = svp.kd_top_loss(ids, lp, z, w, grad=grad)
    wait_limit(-1)
    again = svp.kd_top_loss(ids, lp, z, w, grad=grad)
    torch.cuda.synchronize()
    assert kl[1, 0] == 0 and loss.isnan().all()
    kl[1, 0] = math.nan
    assert kl.isnan().all()
    if grad:
        assert (gr[1, 0] == 0).all()
        gr[1, 0] = math.nan
        assert gr.isnan().all()
    assert all(x is y is None or torch.equal(x, y) for x, y in zip(again, want))


@pytest.mark.parametrize("ns", [1, 3000, 20000])
@pytest.mark.parametrize("n_seq,t_len,V,dtype", [(3, 5, 140001, torch.bfloat16), (130, 3, 70001, torch.bfloat16)])
def test_loss_where_some_waits_expire(n_seq, t_len, V, dtype, ns, wait_limit):
    # which ones is not known; what is not NaN is right
    g = torch.Generator(device=DEV).manual_seed(150)
    z = (torch.randn(n_seq, t_len, V, generator=g, device=DEV) * 3).to(dtype)
    ids, lp, _ = svp.kd_top(z.flip(2).contiguous(), 12)
    w = torch.ones(n_seq, device=DEV)
    want = svp.kd_top_loss(ids, lp, z, w)
    wait_limit(ns)
    kl, loss, gr = svp.kd_top_loss(ids, lp, z, w)
    torch.cuda.synchronize()
    assert (kl.isnan() | (kl == want[0])).all()
    assert torch.equal(loss.isnan(), kl.isnan().any(1)) and (loss.isnan() | (loss == want[1])).all()
    assert (gr.isnan() | (gr == want[2])).all()
    assert not gr[~kl.isnan()].isnan().any()


def test_captured_calls_replay():
    ids, lp, z, w = (x.to(DEV) for x in pair(2, 2, 3000, torch.float32, 16, 1.0, seed=110))
    want = svp.kd_top(z, 16) + svp.kd_top_loss(ids, lp, z, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = svp.kd_top(z, 16) + svp.kd_top_loss(ids, lp, z, w)
    for x in got:
        x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.slow
def test_loss_of_rows_past_32_bit_offsets():
    n, V = 16800, 128256
    z = torch.zeros(n, 1, V, dtype=torch.bfloat16, device=DEV)
    ids, lp, tail, _ = pair(2, 1, V, torch.bfloat16, 20, 1.0, seed=120)
    z[-2:] = tail.to(DEV)
    all_ids = torch.full((n, 1, 20), -1, dtype=torch.int32, device=DEV)
    all_lp = torch.full((n, 1, 20), -INF, device=DEV)
    all_ids[-2:], all_lp[-2:] = ids.to(DEV), lp.to(DEV)
    kl, _, g = svp.kd_top_loss(all_ids, all_lp, z, torch.ones(n, device=DEV))
    torch.cuda.synchronize()
    for b in range(2):
        ref, rg, tol, gt = loss_reference(ids[b, 0], lp[b, 0], tail[b, 0], 1.0, 1.0, True)
        assert abs(kl[b - 2, 0].item() - ref) <= tol
        assert (np.abs(g[b - 2, 0].double().cpu().numpy() - rg) <= gt + np.abs(rg) * 2.0 ** -7 + 1e-37).all()
    assert (g[:100] == 0).all()


def test_refusals():
    z = torch.zeros(2, 3, 64, device=DEV)
    ids = torch.zeros(2, 3, 4, dtype=torch.int32, device=DEV)
    lp, w = torch.zeros(2, 3, 4, device=DEV), torch.ones(2, device=DEV)
    for k in (0, -1, svp.SV_KD_TOP_MAX + 1):
        with pytest.raises(ValueError):
            svp.kd_top(z, k)
    with pytest.raises(TypeError):
        svp.kd_top(z.double(), 4)
    with pytest.raises(ValueError):
        svp.kd_top(z[0], 4)
    with pytest.raises(ValueError):
        svp.kd_top(z.cpu(), 4)
    with pytest.raises(ValueError):
        svp.kd_top(z.transpose(0, 1), 4)
    with pytest.raises(TypeError):
        svp.kd_top(z, 4, n_rows=torch.ones(2, device=DEV))
    for T in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(svp.SpecVerifyError):
            svp.kd_top(z, 4, T)
        with pytest.raises(svp.SpecVerifyError):
            svp.kd_top_loss(ids, lp, z, w, T)
    with pytest.raises(TypeError):
        svp.kd_top_loss(ids.long(), lp, z, w)
    with pytest.raises(TypeError):
        svp.kd_top_loss(ids, lp.bfloat16(), z, w)
    with pytest.raises(ValueError):
        svp.kd_top_loss(ids, lp[:, :, :3], z, w)
    with pytest.raises(ValueError):
        svp.kd_top_loss(ids[:, :2], lp, z, w)
    with pytest.raises(ValueError):
        svp.kd_top_loss(ids, lp, z, w[:1])
    with pytest.raises(svp.SpecVerifyError):
        svp.kd_top_loss(torch.zeros(1, 1, 300, dtype=torch.int32, device=DEV), torch.zeros(1, 1, 300, device=DEV),
                        z[:1, :1], w[:1])
    with pytest.raises(svp.SpecVerifyError):
        svp.kd_top_loss(ids[:1, :1].contiguous(), lp[:1, :1].contiguous(),
                        torch.zeros(1, 1, 524289, dtype=torch.bfloat16, device=DEV), w[:1])
