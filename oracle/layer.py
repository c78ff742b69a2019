"""Projections, the gated feed-forward block, rotary positions and the policy
objective, in fp64 (test infrastructure only).

Plain NumPy from the definitions; shares no code with the library.  Each
``*_mag`` value beside a result is the same sum over magnitudes, from which
the tests derive their tolerances.
"""
import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])


def act(z, name):
    """(act(z), act'(z))."""
    if name in (None, "none"):
        return z, np.ones_like(z)
    if name == "gelu":
        phi = 0.5 * (1.0 + _erf(z / math.sqrt(2.0)))
        return z * phi, phi + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if name == "silu":
        with np.errstate(over="ignore"):
            s = 1.0 / (1.0 + np.exp(-z))
        return z * s, s * (1.0 + z * (1.0 - s))
    t = np.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    slope = math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z * z)
    return 0.5 * z * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * slope


def linear(x, w, bias=None, name="none", residual=None):
    z = x @ w.T if bias is None else x @ w.T + bias
    y = act(z, name)[0]
    return y if residual is None else y + residual


def linear_bwd(x, w, dy, bias=None, name="none"):
    """(dx, dw, db)."""
    z = x @ w.T if bias is None else x @ w.T + bias
    dz = dy * act(z, name)[1]
    return dz @ w, dz.T @ x, dz.sum(0)


def gated_ffn(x, w_in, w_out, name="silu", residual=None):
    """(y, g | u, a)."""
    gu = x @ w_in.T
    half = w_in.shape[0] // 2
    a = act(gu[:, :half], name)[0] * gu[:, half:]
    y = a @ w_out.T
    return (y if residual is None else y + residual), gu, a


def gated_ffn_bwd(x, w_in, w_out, dy, name="silu"):
    """(dx, dw_in, dw_out)."""
    gu = x @ w_in.T
    half = w_in.shape[0] // 2
    g, u = gu[:, :half], gu[:, half:]
    value, slope = act(g, name)
    da = dy @ w_out
    d = np.concatenate([da * u * slope, da * value], axis=1)
    return d @ w_in, d.T @ x, dy.T @ (value * u)


def rope(t, depth, freqs, interleaved=False, factor=1.0, inverse=False):
    """t [F, H, d] rotated, pair by pair."""
    out = np.array(t, dtype=np.float64)
    n = len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        angle = depth.astype(np.float64) * f * (-1.0 if inverse else 1.0)
        c, s = factor * np.cos(angle)[:, None], factor * np.sin(angle)[:, None]
        out[:, :, a] = t[:, :, a] * c - t[:, :, b] * s
        out[:, :, b] = t[:, :, a] * s + t[:, :, b] * c
    return out


def policy_loss(loss, old, adv, weight, index, ref=None, lo=0.2, hi=0.2, dual=0.0, kl_coef=0.0, offsets=None):
    """(stats, dloss, magnitudes of the terms of both), token by token."""
    R, F = len(old), len(loss)
    grad, mag = np.zeros(F), np.zeros(F)
    stats, smag = np.zeros(5), np.zeros(5)
    bounds = [(r, r + 1) for r in range(R)] if offsets is None else list(zip(offsets[:-1], offsets[1:]))
    for b, e in bounds:
        on = [r for r in range(b, e) if weight[r] != 0]
        if not on:
            continue
        d = sum(-loss[index[r]] - old[r] for r in on) / len(on)
        ratio = math.exp(d)
        pull, pull_mag = 0.0, 0.0
        for r in on:
            A, w, logp = adv[r], weight[r], -loss[index[r]]
            plain, band = ratio * A, min(max(ratio, 1.0 - lo), 1.0 + hi) * A
            s, held = min(plain, band), plain > band
            if dual and A < 0 and dual * A > s:
                s, held = dual * A, True
            if not held:
                pull += w * A * ratio
            pull_mag += abs(w * A * ratio)
            kl = 0.0
            if ref is not None:
                t = ref[r] - logp
                kl = math.expm1(t) - t
                grad[index[r]] += w * kl_coef * math.expm1(t)
                mag[index[r]] += abs(w) * kl_coef * (math.exp(t) + 1.0)
            terms = np.array([kl_coef * kl - s, kl, float(held), ratio, 1.0])
            stats += w * terms
            smag += abs(w) * np.array([kl_coef * kl + abs(s), kl, float(held), ratio, 1.0])
        for r in on:
            grad[index[r]] += pull / len(on)
            mag[index[r]] += pull_mag / len(on)
    return stats, grad, smag, mag
