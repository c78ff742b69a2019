"""The operators around the token mixers, in fp64 (test infrastructure only).

Plain NumPy from the definitions: embedding lookup and its table's gradient,
the norms around a block with gate and residual and their gradients, softmax
cross entropy over the vocabulary and its gradients.  Shares no code with the
library.
"""
import numpy as np


def embed(table, tokens, scale=1.0):
    out = np.zeros((len(tokens), table.shape[1]))
    for f, t in enumerate(tokens):
        if 0 <= t < table.shape[0]:
            out[f] = scale * table[t]
    return out


def embed_bwd(tokens, dout, vocab, scale=1.0):
    g = np.zeros((vocab, dout.shape[1]))
    for f, t in enumerate(tokens):
        if 0 <= t < vocab:
            g[t] += scale * dout[f]
    return g


def _rstd(a, eps):
    return 1.0 / np.sqrt(np.mean(a * a, axis=1, keepdims=True) + eps)


def _sig(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def block_norm(res, w_pre, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6):
    r = np.array(res, dtype=np.float64)
    if y is not None:
        u = y if w_post is None else y * _rstd(y, eps) * w_post
        r = r + scale * (u if gate is None else _sig(gate) * u)
    return r, r * _rstd(r, eps) * w_pre


def _norm_grad(a, w, d, eps):
    """d/da and d/dw of sum(d * a * rstd(a) * w)."""
    s = _rstd(a, eps)
    n = a * s
    dn = d * w
    return s * (dn - n * np.mean(dn * n, axis=1, keepdims=True)), np.sum(d * n, axis=0)


def block_norm_bwd(res, w_pre, dx, dres_out=None, y=None, w_post=None, gate=None, scale=1.0, eps=1e-6):
    """(dres, dy, dgate, dw_post, dw_pre); None where the input is None."""
    r, _ = block_norm(res, w_pre, y, w_post, gate, scale, eps)
    dr, dw_pre = _norm_grad(r, w_pre, dx, eps)
    if dres_out is not None:
        dr = dr + dres_out
    if y is None:
        return dr, None, None, None, dw_pre
    u = y if w_post is None else y * _rstd(y, eps) * w_post
    d, dgate, dw_post = scale * dr, None, None
    if gate is not None:
        s = _sig(gate)
        dgate = d * u * s * (1.0 - s)
        d = d * s
    if w_post is not None:
        d, dw_post = _norm_grad(y, w_post, d, eps)
    return dr, d, dgate, dw_post, dw_pre


def lm_loss(h, w, target, scale=1.0):
    """(loss, lse), zero where the target is outside the vocabulary."""
    n, v = len(h), len(w)
    loss, lse = np.zeros(n), np.zeros(n)
    on = np.flatnonzero((target >= 0) & (target < v))
    z = scale * (h[on] @ w.T)
    m = z.max(axis=1, keepdims=True) if len(on) else z
    lse[on] = (m + np.log(np.sum(np.exp(z - m), axis=1, keepdims=True)))[:, 0] if len(on) else 0.0
    loss[on] = lse[on] - z[np.arange(len(on)), target[on]]
    return loss, lse


def lm_loss_bwd(h, w, target, dloss, scale=1.0):
    """(dh, dw) of sum(dloss * loss) over the positions with a target."""
    n, v = len(h), len(w)
    dh = np.zeros(h.shape)
    on = np.flatnonzero((target >= 0) & (target < v))
    dz = score_grads(h, w, target, dloss, scale)
    dh[on] = dz @ w
    return dh, dz.T @ h[on]


def score_grads(h, w, target, dloss, scale=1.0):
    """dz of the positions with a target, in order."""
    v = len(w)
    on = np.flatnonzero((target >= 0) & (target < v))
    _, lse = lm_loss(h, w, target, scale)
    p = np.exp(scale * (h[on] @ w.T) - lse[on, None])
    p[np.arange(len(on)), target[on]] -= 1.0
    return p * (dloss[on, None] * scale)
