"""The operators of a policy's update in 64 bits, and how far float32 kernels
may be off them.

Where the tolerances come from: an exponential is ex2.approx (2^-22) of
(z - m) log2(e) / T, rounded three times, so off by up to 2^-22 + 2^-22 |z - m| / T
of itself; sums are float32, a few hundred terms long per thread and then
pairwise.  What lies 40 below the maximum no longer counts, so a sum over the
row, or over all tokens but one, is off by up to REL = 2e-5 of itself.
"""
import math

import numpy as np

REL = 2e-5
HALF_STEP = {"torch.float32": 2.0 ** -24, "torch.bfloat16": 2.0 ** -8}


class Rows:
    """logp, entropy, lse and p of [n, V] rows and their tokens, with the
    tolerances of each.  ``ok`` marks rows with numbers, ``live`` those with a
    token."""

    def __init__(self, logits, tokens, T):
        z = logits.double().cpu().numpy()
        shape = z.shape[:-1]
        z = z.reshape(-1, z.shape[-1])
        x = tokens.cpu().numpy().reshape(-1).astype(np.int64)
        n, V = z.shape
        self.live = x >= 0
        self.ok = self.live & (x < V) & ~np.isnan(z).any(1) & ~(z == np.inf).any(1) & (z > -np.inf).any(1)
        at = np.where(self.ok, x, 0)
        z = np.where(self.ok[:, None], z, 0.0)
        m = z.max(1)
        with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
            u = (z - m[:, None]) / T
            e = np.exp(u)
            others = e.copy()
            others[np.arange(n), at] = 0.0
            s, ex = others.sum(1), e[np.arange(n), at]
            Z = s + ex
            ux = u[np.arange(n), at]
            top = ux == 0.0
            self.logp = np.where(top, -np.log1p(s), ux - np.log(Z))
            self.lse = m / T + np.log(Z)
            self.p = e / Z[:, None]
            self.rest = s / Z
            self.logp_v = u - np.log(Z)[:, None]
            ue = np.where(e > 0, u * e, 0.0)
            self.H = np.log1p(Z - 1) - ue.sum(1) / Z
            self.spread = -ue.sum(1) / Z
            self.tol_logp = np.where(top, REL * self.rest + 2.0 ** -22 * np.abs(self.logp),
                                     REL + 2.0 ** -22 * np.abs(np.where(np.isfinite(ux), ux, 0.0)))
            self.tol_lse = REL + 2.0 ** -22 * np.abs(self.lse)
            self.tol_H = np.where(top, 3 * REL * (self.rest + self.H), 3 * REL * (1 + self.spread))
        self.x, self.n, self.V, self.shape, self.T = at, n, V, shape, T
        for a, empty in ((self.logp, 0.0), (self.H, 0.0), (self.lse, -np.inf)):
            a[~self.live] = empty
            a[self.live & ~self.ok] = np.nan

    def gradient(self, g, h, tol_g, tol_h=None):
        """The gradient in the logits from the derivatives g of the
        log-probabilities and h of the entropies ([n]), and its tolerance in
        float32, for derivatives that are off by up to tol_g and tol_h."""
        n, T = self.n, self.T
        rows = np.arange(n)
        g, h = np.where(self.ok, g, 0.0), np.where(self.ok, h, 0.0)
        tol_g = np.where(self.ok, tol_g, 0.0)
        tol_h = np.zeros(n) if tol_h is None else np.where(self.ok, tol_h, 0.0)
        with np.errstate(invalid="ignore", over="ignore"):
            bend = np.where(self.p > 0, self.p * (self.logp_v + np.where(self.ok, self.H, 0.0)[:, None]), 0.0)
            d = -g[:, None] * self.p - h[:, None] * bend
            own = np.where(self.p[rows, self.x] > 0, bend[rows, self.x], 0.0)
            d[rows, self.x] = g * self.rest - h * own
            width = np.where(self.p > 0, self.p * (np.abs(self.logp_v) + 1 + np.where(self.ok, self.H, 0.0)[:, None]), 0.0)
            tol = (np.abs(g) * 2 * REL + tol_g)[:, None] * self.p + (np.abs(h) * 3 * REL + tol_h)[:, None] * width
            tol[rows, self.x] = ((np.abs(g) * 2 * REL + tol_g) * self.rest
                                 + (np.abs(h) * 3 * REL + tol_h) * width[rows, self.x])
        d, tol = d / T, tol / T + 1e-37
        d[~self.live] = 0.0
        d[self.live & ~self.ok] = np.nan
        return d, tol


def policy(R, A, w, old=None, ref=None, low=0.2, high=0.2, dual=None, kl=0.0, ent=0.0):
    """(row loss, its tolerance, derivative in logp, its tolerance, in H), with
    A, w, old, ref as [n] arrays (w repeated for a sequence's rows)."""
    with np.errstate(invalid="ignore", over="ignore"):
        logp = np.where(R.ok, R.logp, 0.0)
        r = np.exp(logp - old) if old is not None else np.ones(R.n)
        gained, held = r * A, np.clip(r, 1 - low, 1 + high) * A
        gain = np.minimum(gained, held)
        slope = np.where(gained <= held, -gained, 0.0)
        if dual:
            cut = (A < 0) & (gain < dual * A)
            gain, slope = np.where(cut, dual * A, gain), np.where(cut, 0.0, slope)
        loss = -gain
        off = (R.tol_logp + 4e-7 * (1 + np.abs(logp))) if old is not None else 0 * R.tol_logp
        tol_loss = np.abs(gained) * off + 2e-7 * np.abs(gain)
        tol_slope = np.abs(slope) * (off + 2e-7)
        if ref is not None and kl:
            d = ref - logp
            loss = loss + kl * np.where(np.abs(d) < 1e-3, d * d * (0.5 + d / 6 + d * d / 24), np.expm1(d) - d)
            slope = slope - kl * np.expm1(d)
            off = R.tol_logp + 4e-7 * (1 + np.abs(logp))
            tol_loss = tol_loss + abs(kl) * (np.abs(np.expm1(d)) * off + off * off + 4e-7 * np.abs(np.expm1(d) - d))
            tol_slope = tol_slope + abs(kl) * (np.exp(d) * off + 4e-7 * np.abs(np.expm1(d)))
        if ent:
            loss = loss - ent * np.where(R.ok, R.H, 0.0)
            tol_loss = tol_loss + abs(ent) * R.tol_H
    loss = np.where(R.ok, loss, np.where(R.live, np.nan, 0.0))
    tol_loss = tol_loss + 4e-7 * np.abs(loss) + 1e-37
    return loss, tol_loss, w * slope, np.abs(w) * tol_slope, -ent * w * np.ones(R.n)


def preference(s, ref, w, beta, kind, smoothing):
    """(margin, loss, derivative of the loss in s_0 - s_1) of one pair."""
    h = (s[0] - s[1]) - (float(ref[0]) - float(ref[1]))
    m = beta * h
    soft = lambda v: max(v, 0.0) + math.log1p(math.exp(-abs(v)))
    up = lambda v: 1 / (1 + math.exp(-v)) if v > 0 else math.exp(v) / (1 + math.exp(v))
    if kind == "sigmoid":
        loss, slope = (1 - smoothing) * soft(-m) + smoothing * soft(m), beta * (smoothing * up(m) - (1 - smoothing) * up(-m))
    elif kind == "hinge":
        loss, slope = max(0.0, 1 - m), -beta if m < 1 else 0.0
    else:
        off = h - 0.5 / beta
        loss, slope = off * off, 2 * off
    return m, w * loss, w * slope


def assert_close(got, ref, tol, dtype="torch.float32", what=""):
    """got (a tensor) against ref within tol and half a step of its type; NaN
    and infinities have to agree."""
    g = got.detach().double().cpu().numpy().reshape(ref.shape)
    ref = np.where(np.abs(ref) > np.finfo(np.float32).max, np.copysign(np.inf, ref), ref)   # past float32's range
    fin = np.isfinite(ref)
    assert np.array_equal(g[~fin], ref[~fin], equal_nan=True), (what, g[~fin][:5], ref[~fin][:5])
    off = np.abs(g[fin] - ref[fin])
    lim = np.broadcast_to(tol, ref.shape)[fin]
    step = HALF_STEP[str(dtype)] * (np.abs(ref[fin]) + lim)
    bad = ~(off <= lim + step)
    if bad.any():
        i = int(np.argmax(np.where(bad, off - lim - step, -np.inf)))
        raise AssertionError(f"{what}: {bad.sum()} of {bad.size} off, worst {g[fin][i]} for {ref[fin][i]}, "
                             f"{off[i] / (lim + step)[i]:.2f} of what is allowed")
