"""A whole training step of a layer over a packed tree, tight enough that a lost
term shows.

Tolerance, in 2-norms: a tensor rounded to bf16 is off by b / sqrt 3 = 2.3e-3 of its
norm at most (b = 2^-8).  Some 32 results, operands and kept values of the step are
rounded on the way to a gradient, independently; with a gain of at most 2 each they
come to 2 sqrt(32) 2.3e-3 = 2.6e-2; 2^-5 is allowed.  On the CPU the reference is
computed again with one ingredient left out or changed at a time: each moves some
gradient by three times that or more.
"""
import math

import numpy as np
import pytest
import torch

BF = 2.0 ** -8
TOL = 2.0 ** -5

HQ, HKV, D, V, I = 4, 2, 64, 304, 328
C = HQ * D
KL, LOW, HIGH, FACTOR, STRETCH, ROT = 0.5, 0.2, 0.28, 1.25, 2.0, 32


def _rnd(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def _sequences():
    rng = np.random.default_rng(11)
    head = rng.integers(0, 300, 60)
    return [np.concatenate([head, rng.integers(0, 300, k)]).astype(np.int32) for k in (40, 75, 22, 90)]


def _weights():
    one = lambda seed: 1 + _rnd(seed, C, std=0.1, dtype=torch.float32)
    return {"table": _rnd(1, V, C), "wqkv": _rnd(2, (HQ + 2 * HKV) * D, C, std=C ** -0.5),
            "bqkv": _rnd(3, (HQ + 2 * HKV) * D, std=0.1, dtype=torch.float32), "wo": _rnd(4, C, C, std=C ** -0.5),
            "w_in": _rnd(5, 2 * I, C, std=C ** -0.5), "w_out": _rnd(6, C, I, std=I ** -0.5), "n1": one(7), "n2": one(8),
            "n3": one(9), "head": _rnd(10, V, C, std=C ** -0.5)}


def _policy(logp):
    """(old, ref, advantage) of raw tokens: a third each at the sampled ratio, well above and well below the clip."""
    R = len(logp)
    step = torch.tensor([0.0, 0.6, -0.6], dtype=torch.float32)[torch.arange(R) % 3]
    return (logp + step + 0.02 * _rnd(13, R, dtype=torch.float32), logp + 0.7 * _rnd(14, R, dtype=torch.float32),
            _rnd(12, R, dtype=torch.float32))


def _loss(p, batch, policy=None, change=None):
    """(log-probabilities of the raw tokens, objective) in fp64; change: what is left out or done otherwise."""
    depth, end, index, target, ids, weight = batch
    F = len(ids)

    def norm(t, s):
        return t * torch.rsqrt(t.square().mean(1, keepdim=True) + 1e-6) * s

    freqs = 1e4 ** (-torch.arange(0, ROT, 2, dtype=torch.float64) / ROT) / (1.0 if change == "stretch" else STRETCH)
    factor = 1.0 if change == "factor" else FACTOR

    def turn(t):
        angle = depth.double()[:, None] * freqs
        c, s = (factor * torch.cos(angle))[:, None], (factor * torch.sin(angle))[:, None]
        if change == "pairs":
            a, b = t[..., :ROT // 2], t[..., ROT // 2:ROT]
            return torch.cat([a * c - b * s, a * s + b * c, t[..., ROT:]], 2)
        a, b = t[..., 0:ROT:2], t[..., 1:ROT:2]
        return torch.cat([torch.stack([a * c - b * s, a * s + b * c], 3).flatten(2), t[..., ROT:]], 2)
    e = p["table"][ids.long()]
    z = norm(e, p["n1"]) @ p["wqkv"].T
    if change != "bias":
        z = z + p["bqkv"]
    q = turn(z[:, :C].unflatten(1, (HQ, D))).transpose(0, 1)
    k = turn(z[:, C:C + HKV * D].unflatten(1, (HKV, D))).repeat_interleave(HQ // HKV, 1).transpose(0, 1)
    v = z[:, C + HKV * D:].unflatten(1, (HKV, D)).repeat_interleave(HQ // HKV, 1).transpose(0, 1)
    i = torch.arange(F)
    sees = i[None] <= i[:, None]
    if change != "tree":
        sees = sees & (i[:, None] < end.long()[None])
    scores = (q @ k.transpose(1, 2) / D ** 0.5).masked_fill(~sees[None], float("-inf"))
    m = (torch.softmax(scores, 2) @ v).transpose(0, 1).flatten(1) @ p["wo"].T
    if change != "residual":
        m = m + e
    gu = norm(m, p["n2"]) @ p["w_in"].T
    act = torch.nn.functional.gelu if change == "act" else torch.nn.functional.silu
    y = (act(gu[:, :I]) * gu[:, I:]) @ p["w_out"].T
    if change != "ffn residual":
        y = y + m
    logp = torch.log_softmax(norm(y, p["n3"]) @ p["head"].T, 1).gather(1, target.long().clamp(min=0)[:, None])[:, 0]
    raw = logp[index.long()]
    if policy is None:
        return raw, None
    on = torch.nonzero(weight)[:, 0]
    old, ref, adv = (t[on].double() for t in policy)
    ratio, t = torch.exp(raw[on] - old), ref - raw[on]
    s = ratio * adv
    if change != "clip":
        s = torch.minimum(s, ratio.clamp(1 - LOW, 1 + HIGH) * adv)
    kl = 0.0 if change == "kl" else KL * (torch.expm1(t) - t)
    return raw, (weight[on].double() * (kl - s)).sum()


def _plan(ops):
    seqs = _sequences()
    plan = ops.Plan.from_sequences(seqs, row_capacity=1024, min_shared=8)
    nxt = np.concatenate([np.append(s[1:], -1) for s in seqs]).astype(np.int32)
    weight = torch.from_numpy((nxt >= 0).astype(np.float32) / plan.info["n_raw"])
    return plan, np.concatenate(seqs), nxt, weight


def _host_batch(ops):
    """The batch's arrays from the host plan: positions in packed order."""
    plan, ids, nxt, weight = _plan(ops)
    host = {k: torch.from_numpy(v) for k, v in plan.export().items()}
    begin, raw = plan.raw_of_forwarded()
    first = raw[begin[:-1]]
    return (host["depth"], host["subtree_end"], host["token_index"], torch.from_numpy(nxt[first]),
            torch.from_numpy(ids[first]), weight)


def test_every_ingredient_moves_some_gradient(lib):
    from prefix_tree_packed_dfs_gb300 import ops
    batch = _host_batch(ops)
    p = {k: t.double().requires_grad_() for k, t in _weights().items()}
    policy = _policy(_loss(p, batch)[0].detach().float())
    grads = lambda change: torch.autograd.grad(_loss(p, batch, policy, change)[1], list(p.values()), allow_unused=True)
    want = grads(None)
    for change in ("stretch", "factor", "pairs", "bias", "tree", "residual", "act", "ffn residual", "clip", "kl"):
        moved = max(float((torch.zeros_like(w) if g is None else g).sub(w).norm() / w.norm())
                    for g, w in zip(grads(change), want))
        assert moved >= 3 * TOL, (change, moved)


@pytest.mark.gpu
def test_a_training_step_keeps_every_ingredient():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops
    plan, raw_ids, nxt, weight = _plan(ops)
    dp = plan.to_device()
    p = {k: t.cuda() for k, t in _weights().items()}
    ids = ops.gather_to_forwarded(dp, torch.from_numpy(raw_ids).cuda())
    target = ops.gather_to_forwarded(dp, torch.from_numpy(nxt).cuda())
    freqs = ops.rope_freqs(ROT, 1e4, stretch=STRETCH)
    rope = dict(interleaved=True, factor=FACTOR)
    # forward
    emb = ops.embed(p["table"], ids)
    _, x1 = ops.block_norm(emb, p["n1"])
    qkv = ops.linear(x1, p["wqkv"], bias=p["bqkv"])
    q, k = qkv[:, :C].unflatten(1, (HQ, D)), qkv[:, C:C + HKV * D].unflatten(1, (HKV, D))
    v = qkv[:, C + HKV * D:].unflatten(1, (HKV, D)).contiguous()
    rq, rk = ops.rope_by_depth_ex(q, k, dp.depth, freqs, **rope)
    o, lse = ops.tree_attn_fwd(dp, rq, rk, v, precise=False)
    mid = ops.linear(o.flatten(1), p["wo"], residual=emb)
    _, x2 = ops.block_norm(mid, p["n2"])
    out, pre, a = ops.gated_ffn(x2, p["w_in"], p["w_out"], residual=mid, save=True)
    _, x3 = ops.block_norm(out, p["n3"])
    loss, lse_v = ops.lm_loss(x3, p["head"], target)
    raw = -ops.scatter_token_index(dp.token_index, lse_src=loss[None])[1][0]
    policy = _policy(raw.cpu())
    old, ref, adv = (t.cuda() for t in policy)
    stats, dloss = ops.policy_loss(loss, old, adv, weight.cuda(), dp.token_index, dp.fwd_raw_begin, dp.fwd_raw,
                                   ref_logp=ref, clip_low=LOW, clip_high=HIGH, kl_coef=KL)
    # backward
    dx3, dhead = ops.lm_loss_bwd(x3, p["head"], target, lse_v, dloss)
    dout, _, _, _, dn3 = ops.block_norm_bwd(out, p["n3"], dx3)
    dx2, dw_in, dw_out = ops.gated_ffn_bwd(x2, p["w_in"], p["w_out"], dout, pre, a)
    dmid, _, _, _, dn2 = ops.block_norm_bwd(mid, p["n2"], dx2, dres_out=dout)
    do, dwo, _ = ops.linear_bwd(o.flatten(1), p["wo"], dmid)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = ops.tree_attn_bwd(dp, rq, rk, v, o, lse, do.unflatten(1, (HQ, D)))
    ops.rope_by_depth_ex(dq, dk, dp.depth, freqs, inverse=True, q_out=dqkv[:, :C].unflatten(1, (HQ, D)),
                         k_out=dqkv[:, C:C + HKV * D].unflatten(1, (HKV, D)), **rope)
    dqkv[:, C + HKV * D:] = dv.flatten(1)
    dx1, dwqkv, dbqkv = ops.linear_bwd(x1, p["wqkv"], dqkv, bias=p["bqkv"])
    demb, _, _, _, dn1 = ops.block_norm_bwd(emb, p["n1"], dx1, dres_out=dmid)
    dtable = ops.embed_bwd(ids, demb, V)
    got = dict(table=dtable, wqkv=dwqkv, bqkv=dbqkv, wo=dwo, w_in=dw_in, w_out=dw_out, n1=dn1, n2=dn2, n3=dn3, head=dhead)

    w = {n: t.double().cpu().requires_grad_() for n, t in p.items()}
    batch = tuple(t.cpu() for t in (dp.depth, dp.subtree_end, dp.token_index, target, ids)) + (weight,)
    total = _loss(w, batch, policy)[1]
    grads = dict(zip(w, torch.autograd.grad(total, list(w.values()))))
    off = {n: float((got[n].double().cpu() - g).norm() / g.norm()) for n, g in grads.items()}
    assert max(off.values()) <= TOL, off
    assert math.isfinite(float(stats[0])) and abs(float(stats[0]) - float(total.detach())) <= \
        TOL * float((weight * adv.cpu().abs() + weight * KL).sum())
