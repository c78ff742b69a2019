"""Parity of the projections, the feed-forward block, the rotary forms and the
policy objective with their fp64 oracle.

Tolerances.  u = 2^-24 is half a step of fp32, b = 2^-8 half a step of bf16 (of
the power of two below a value; 2^-9 of most).
 * A product's sum of K terms: the tensor core truncates, so each addition is
   off by at most 2u of the running magnitude: K 2^-23 sum |terms| (e_z below).
 * Activations: |act'| <= 1.13, |act''| <= 1.2 for all of them; their own
   arithmetic within 2^-20 (|z| + 1) (gelu: Phi within 1.5e-7 = 2^-22.7 times z).
 * linear: b |y| + 1.13 e_z + 2^-20 (|z| + 1)[activation] + 2u (|z| + |residual|).
 * linear_bwd: dz off by e_d = |dy| (1.2 e_z + 2^-19) and, in its products, by
   b |dz| more; dx, dw: the sums of those times the other factor's magnitude,
   the products' own e, and b of the result.  db: sum e_d + N u sum |dz|.
 * gated_ffn: a off by e_a = 1.13 e_g |u| + |act| e_u + 2^-19 (|g| + 1) |u| + b |a|;
   its backward works on a rounded to bf16 and on g and u kept as scaled fp16,
   which adds 2^-11 of their value (and 2^-38 of the largest of 32 neighbours: half
   the step of fp16's smallest numbers, 2^-25, against 2^14) to e_g, e_u.
 * rope: fp32 products of sin and cos within 2^-21: 2^-20 factor (|a| + |b|), and b.
 * policy: a share is a product of few fp32 factors and one exponential of
   |argument| < 8 (relative error below 8u + 2^-22): 2^-19 of the terms'
   magnitudes covers it and sums of up to 16 in a row.
"""
import numpy as np
import pytest
import torch

from oracle import layer as ol

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8
ACTS = ["none", "silu", "gelu", "gelu_tanh"]


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _f64(t):
    return t.detach().double().cpu().numpy()


def _rnd(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def _within(got, ref, tol, what):
    err = np.abs(_f64(got) - ref)
    assert np.isfinite(err).all(), "%s: not finite" % what
    over = err - tol
    i = np.unravel_index(np.argmax(over), over.shape)
    assert over[i] <= 0, "%s: off by %.3g at %s, allowed %.3g" % (what, err[i], i, np.broadcast_to(tol, err.shape)[i])


def _err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# rows: one, few (all three token widths, both ends), below and above a tile, ragged; odd widths
LINEAR = [(1, 64, 64), (1, 2048, 4096), (3, 8, 8), (16, 1000, 552), (17, 136, 1032), (32, 4096, 264), (33, 72, 2048),
          (64, 520, 776), (65, 64, 128), (128, 256, 256), (200, 2048, 512), (257, 1000, 520), (1001, 552, 1000),
          (700, 4096, 136), (3000, 64, 2056), (1000, 4096, 1000), (130, 8, 8),
          (66, 24, 4104), (2600, 328, 1032)]


def _linear_ref(x, w, bias, act, residual):
    z = x @ w.T
    mag = np.abs(x) @ np.abs(w).T
    if bias is not None:
        z, mag = z + bias, mag + np.abs(bias)
    e_z = (x.shape[1] + 2) * 2.0 ** -23 * mag
    y = ol.linear(x, w, bias, act, residual)
    tol = BF * np.abs(y) + 1.13 * e_z + 2 * U * (np.abs(z) + (0 if residual is None else np.abs(residual)))
    if act != "none":
        tol = tol + 2.0 ** -20 * (np.abs(z) + 1)
    return y, tol, z, e_z


@pytest.mark.parametrize("n,c,o", LINEAR)
@pytest.mark.parametrize("act,bias,res", [("none", False, False), ("silu", True, True), ("gelu", True, False),
                                          ("gelu_tanh", False, True)])
def test_linear(ops, n, c, o, act, bias, res):
    x, w = _rnd(1, n, 3 * c)[:, c:2 * c], _rnd(2, o, c, std=c ** -0.5)
    b = _rnd(3, o, std=0.5, dtype=torch.float32) if bias else None
    r = _rnd(4, n, 2 * o, std=2.0)[:, o:] if res else None
    err = _err()
    y = ops.linear(x, w, bias=b, act=act, residual=r, dev_err=err)
    f = lambda t: None if t is None else _f64(t)
    ref, tol, _, _ = _linear_ref(f(x), f(w), f(b), act, f(r))
    _within(y, ref, tol, "y")
    assert int(err) == 0
    # into a column slice of a wider tensor, whose other columns stay
    wide = torch.full((n, o + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.linear(x, w, bias=b, act=act, residual=r, out=wide[:, 8:8 + o])
    assert torch.equal(wide[:, 8:8 + o], y) and (wide[:, :8] == 7).all() and (wide[:, 8 + o:] == 7).all()
    if res:   # in place on the residual
        r2 = r.clone()
        ops.linear(x, w, bias=b, act=act, residual=r2, out=r2)
        assert torch.equal(r2, y)


@pytest.mark.parametrize("n,c,o", LINEAR)
@pytest.mark.parametrize("act,bias", [("none", False), ("none", True), ("silu", True), ("gelu", True),
                                      ("gelu_tanh", False)])
def test_linear_bwd(ops, n, c, o, act, bias):
    x, w = _rnd(1, n, c + 8)[:, :c], _rnd(2, o, c, std=c ** -0.5)
    b = _rnd(3, o, std=0.5, dtype=torch.float32) if bias else None
    dy = _rnd(5, n, 2 * o)[:, o:]
    err = _err()
    dirty = torch.full((o, c), float("nan"), dtype=torch.bfloat16, device="cuda")
    dx, dw, db = ops.linear_bwd(x, w, dy, bias=b, act=act, dw=dirty, dev_err=err)
    assert int(err) == 0
    X, W, D, Bv = _f64(x), _f64(w), _f64(dy), None if b is None else _f64(b)
    _, _, z, e_z = _linear_ref(X, W, Bv, act, None)
    rx, rw, rb = ol.linear_bwd(X, W, D, Bv, act)
    dz = D * ol.act(z, act)[1]
    e_d = 0.0 * dz if act == "none" else np.abs(D) * (1.2 * e_z + 2.0 ** -19)
    e_p = e_d if act == "none" else e_d + BF * np.abs(dz)
    _within(dx, rx, BF * np.abs(rx) + e_p @ np.abs(W) + (o + 2) * 2.0 ** -23 * (np.abs(dz) @ np.abs(W)), "dx")
    _within(dw, rw, BF * np.abs(rw) + e_p.T @ np.abs(X) + (n + 2) * 2.0 ** -23 * (np.abs(dz).T @ np.abs(X)), "dw")
    if bias:
        _within(db, rb, e_d.sum(0) + (n + 2) * U * np.abs(dz).sum(0) + 1e-30, "db")
    else:
        assert db is None
    again = ops.linear_bwd(x, w, dy, bias=b, act=act)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1])
    # dx into a column slice
    wide = torch.full((n, c + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.linear_bwd(x, w, dy, bias=b, act=act, dx=wide[:, 8:8 + c])
    assert torch.equal(wide[:, 8:8 + c], dx) and (wide[:, :8] == 7).all() and (wide[:, 8 + c:] == 7).all()


FFN = [(1, 64, 64, 64), (1, 2048, 1024, 2048), (5, 8, 8, 8), (16, 136, 200, 136), (32, 1000, 328, 1000),
       (40, 256, 1032, 512), (64, 520, 136, 520), (65, 64, 128, 64), (129, 128, 264, 72), (257, 1000, 520, 1000),
       (1003, 264, 1096, 264), (300, 2048, 256, 2048), (130, 8, 8, 8), (70, 24, 2056, 8)]


def _ffn_parts(X, WI, WO, act):
    i = WO.shape[1]
    gu = X @ WI.T
    e = (X.shape[1] + 2) * 2.0 ** -23 * (np.abs(X) @ np.abs(WI).T)
    g, u, e_g, e_u = gu[:, :i], gu[:, i:], e[:, :i], e[:, i:]
    v, slope = ol.act(g, act)
    e_a = 1.13 * e_g * (np.abs(u) + e_u) + np.abs(v) * e_u + 2.0 ** -19 * (np.abs(g) + 1) * np.abs(u)
    e_a = e_a + BF * (np.abs(v * u) + e_a)
    return g, u, e_g, e_u, v, slope, e_a


@pytest.mark.parametrize("n,c,i,o", FFN)
@pytest.mark.parametrize("act,res", [("silu", True), ("gelu", False), ("gelu_tanh", True), ("none", False)])
def test_gated_ffn(ops, n, c, i, o, act, res):
    x, w_in, w_out = _rnd(1, n, c + 8)[:, 8:], _rnd(2, 2 * i, c, std=c ** -0.5), _rnd(3, o, i, std=i ** -0.5)
    r = _rnd(4, n, 2 * o, std=2.0)[:, o:] if res else None
    err = _err()
    y, pre, a = ops.gated_ffn(x, w_in, w_out, act=act, residual=r, save=True, dev_err=err)
    X, WI, WO = _f64(x), _f64(w_in), _f64(w_out)
    R = None if r is None else _f64(r)
    ry, rgu, ra = ol.gated_ffn(X, WI, WO, act, R)
    g, u, e_g, e_u, v, _, e_a = _ffn_parts(X, WI, WO, act)
    keep = lambda t, e: 2.0 ** -11 * (np.abs(t) + e) + 2.0 ** -38 * (np.abs(t) + e).max(1, keepdims=True)
    k_g, k_u = keep(g, e_g), keep(u, e_u)
    ip = -(-i // 64) * 64
    half = pre[:4 * n * ip].view(torch.float16).view(n, 2, ip)[:, :, :i].double().cpu().numpy()
    groups, rows = -(-i // 32), -(-n // 128) * 128
    exps = pre[4 * n * ip:].view(2, groups, rows)[:, :, :n].cpu().numpy().astype(np.int64)
    unscale = np.repeat(2.0 ** (exps - 141), 32, 1)[:, :i].transpose(2, 0, 1)
    got = (half * unscale).reshape(n, 2 * i)
    err_pre = np.abs(got - rgu)
    assert (err_pre <= np.concatenate([k_g + e_g, k_u + e_u], 1)).all(), "pre: off by %.3g" % err_pre.max()
    _within(a, ra, e_a, "a")
    tol = BF * np.abs(ry) + e_a @ np.abs(WO).T + (i + 2) * 2.0 ** -23 * (np.abs(ra) @ np.abs(WO).T) * 1.01
    tol = tol + 2 * U * (0 if R is None else np.abs(R) + np.abs(ry))
    _within(y, ry, tol, "y")
    y2 = ops.gated_ffn(x, w_in, w_out, act=act, residual=r)   # nothing kept
    _within(y2, ry, tol, "y with nothing kept")
    if res:
        r2 = r.clone()
        ops.gated_ffn(x, w_in, w_out, act=act, residual=r2, out=r2)
        assert torch.equal(r2, y2)
    dy = _rnd(6, n, 2 * o)[:, :o]
    dx, dwi, dwo = ops.gated_ffn_bwd(x, w_in, w_out, dy, pre, a, act=act, dev_err=err)
    assert int(err) == 0
    D = _f64(dy)
    rx, rwi, rwo = ol.gated_ffn_bwd(X, WI, WO, D, act)
    slope = ol.act(g, act)[1]
    da, e_da = D @ WO, (o + 2) * 2.0 ** -23 * (np.abs(D) @ np.abs(WO))
    q_g, q_u = e_g + k_g, e_u + k_u     # of g, u as kept
    top = np.abs(da) + e_da
    curve = 0.0 if act == "none" else 1.2
    e_dg = e_da * (np.abs(u) + q_u) * 1.13 + np.abs(da) * (q_u * 1.13 + (np.abs(u) + q_u) * (curve * q_g + 2.0 ** -19))
    e_du = e_da * (np.abs(v) + 1.13 * q_g) + np.abs(da) * (1.13 * q_g + 2.0 ** -19 * (np.abs(g) + 1))
    e_d = np.concatenate([e_dg + BF * (np.abs(da * u * slope) + e_dg), e_du + BF * (np.abs(da * v) + e_du)], 1)
    d = np.concatenate([np.abs(da * u * slope), np.abs(da * v)], 1)
    k = 2.0 ** -23 * 1.05
    assert top.shape == da.shape
    _within(dx, rx, BF * np.abs(rx) + e_d @ np.abs(WI) * 1.01 + (2 * i + 2) * k * (d @ np.abs(WI)), "dx")
    _within(dwi, rwi, BF * np.abs(rwi) + e_d.T @ np.abs(X) * 1.01 + (n + 2) * k * (d.T @ np.abs(X)), "dw_in")
    _within(dwo, rwo, BF * np.abs(rwo) + np.abs(D).T @ e_a * 1.01 + (n + 2) * k * (np.abs(D).T @ np.abs(ra)), "dw_out")


ROPE = [(1, 1, 1, 16, 16), (1, 16, 8, 128, 128), (5, 4, 2, 64, 32), (100, 3, 1, 96, 48), (33, 8, 8, 256, 256),
        (77, 1, 4, 40, 32), (1000, 16, 8, 128, 64), (3, 64, 8, 512, 256)]


@pytest.mark.parametrize("f,hq,hkv,d,rot", ROPE)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_forms(ops, f, hq, hkv, d, rot, interleaved, inverse):
    qkv = _rnd(1, f, (hq + 2 * hkv) * d)
    q, k = qkv[:, :hq * d].unflatten(1, (hq, d)), qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
    g = np.random.default_rng(5)
    depth = g.integers(0, 2 ** 31 - 1, f).astype(np.int32) if f % 2 else g.integers(-50, 5000, f).astype(np.int32)
    dp = torch.from_numpy(depth).cuda()
    freqs = ops.rope_freqs(rot, 1e4, stretch=4.0, trained=4096)
    kw = dict(interleaved=interleaved, factor=1.25, inverse=inverse)
    before = qkv.clone()
    oq, ok = ops.rope_by_depth_ex(q, k, dp, freqs, **kw)
    assert torch.equal(qkv, before)
    n = rot // 2
    for got, src in ((oq, q), (ok, k)):
        s = _f64(src)
        ref = ol.rope(s, depth, freqs, interleaved, 1.25, inverse)
        mag = np.abs(s)
        part = mag[..., :rot]
        sw = part.reshape(part.shape[:2] + (n, 2))[..., ::-1].reshape(part.shape) if interleaved else \
            np.concatenate([part[..., n:], part[..., :n]], -1)
        tol = BF * np.abs(ref)
        # the oracle's own angle: |depth freq| 2^-53 radians; the library's 2^-53 turns per position
        far = np.abs(depth.astype(np.float64))[:, None, None] * 16.0 * 2.0 ** -53
        tol[..., :rot] += (2.0 ** -20 + far) * 1.25 * (part + sw)
        tol[..., rot:] = 0.0
        _within(got, ref, tol, "rotated")
    only, none = ops.rope_by_depth_ex(q, None, dp, freqs, **kw)
    assert none is None and torch.equal(only, oq)
    only, none = ops.rope_by_depth_ex(None, k, dp, freqs, **kw)[::-1]
    assert none is None and torch.equal(only, ok)
    ops.rope_by_depth_ex(q, k, dp, freqs, q_out=q, k_out=k, **kw)      # in place, on the slices
    assert torch.equal(q, oq) and torch.equal(k, ok) and torch.equal(qkv[:, (hq + hkv) * d:], before[:, (hq + hkv) * d:])


def test_rope_form_of_the_plain_call(ops):
    q, k = _rnd(1, 301, 4, 128), _rnd(2, 301, 2, 128)
    depth = torch.arange(301, dtype=torch.int32, device="cuda") * 100
    oq, ok = ops.rope_by_depth_ex(q, k, depth, ops.rope_freqs(128, 1e6))
    pq, pk = ops.rope_by_depth(q.clone(), k.clone(), depth, 1e6)
    for a, b in ((oq, pq), (ok, pk)):   # both round the same fp32 value, up to its last bits
        assert ((a.float() - b.float()).abs() <= 2 * BF * b.float().abs() + 2.0 ** -18).all()


def _tree(seed, seqs, shared, least, most):
    """token_index, CSR and offsets of sequences over one shared prefix, pairs sharing a little more."""
    g = np.random.default_rng(seed)
    at, index, offsets = shared, [], [0]
    common = None
    for k in range(seqs):
        n = int(g.integers(least, most + 1))
        if k % 2 == 0:
            c = min(least, n) // 2
            common = np.arange(at, at + c)
            at += c
        own = np.arange(at, at + n - len(common))
        at += n - len(common)
        index += [np.arange(shared), common, own]
        offsets.append(offsets[-1] + shared + n)
    index = np.concatenate(index).astype(np.int32)
    begin = np.zeros(at + 1, dtype=np.int32)
    begin[1:] = np.cumsum(np.bincount(index, minlength=at))
    return index, begin, np.argsort(index, kind="stable").astype(np.int32), np.asarray(offsets, np.int32)


@pytest.mark.parametrize("seqs,shared,least,most", [(1, 0, 1, 1), (2, 1, 2, 2), (4, 128, 64, 128), (64, 40, 3, 90),
                                                   (700, 3, 1, 9), (3, 10, 700, 1500)])
@pytest.mark.parametrize("level", ["token", "sequence"])
@pytest.mark.parametrize("kl,dual", [(0.0, 0.0), (0.05, 0.0), (0.04, 3.0)])
@pytest.mark.parametrize("prefix_on", [False, True])
def test_policy_loss(ops, seqs, shared, least, most, level, kl, dual, prefix_on):
    index, begin, raw, offsets = _tree(seqs, seqs, shared, least, most)
    F, R = len(begin) - 1, len(index)
    g = np.random.default_rng(7)
    loss = (0.05 + 3 * g.random(F)).astype(np.float32)
    old = (-loss[index] + 0.4 * g.normal(size=R)).astype(np.float32)
    ref = (-loss[index] + 0.7 * g.normal(size=R)).astype(np.float32)
    adv = g.normal(size=R).astype(np.float32)
    adv[g.random(R) < 0.05] = 0.0
    weight = (g.random(R) / R).astype(np.float32)
    off = np.zeros(R, bool)
    if not prefix_on:
        for b in offsets[:-1]:
            off[b:b + shared] = True
    off[g.random(R) < 0.1] = True
    weight[off] = 0.0
    for a in (old, ref, adv):
        a[off] = np.nan                     # nothing of a token without weight is read
    lo, hi = (0.2, 0.28) if level == "token" else (0.01, 0.02)
    stats, dl, smag, mag = ol.policy_loss(loss.astype(float), old.astype(float), adv.astype(float),
                                          weight.astype(float), index, ref.astype(float) if kl else None, lo, hi, dual,
                                          kl, offsets if level == "sequence" else None)
    t = lambda a: torch.from_numpy(a).cuda()
    args = (t(loss), t(old), t(adv), t(weight), t(index), t(begin), t(raw))
    kw = dict(ref_logp=t(ref) if kl else None, clip_low=lo, clip_high=hi, dual_clip=dual, kl_coef=kl,
              seq_offsets=t(offsets) if level == "sequence" else None)
    gs, gd = ops.policy_loss(*args, **kw)
    _within(gs, stats, 2.0 ** -19 * smag + 1e-30, "stats")
    _within(gd, dl, 2.0 ** -19 * mag + 1e-30, "dloss")
    ws = torch.full((int(4 * R + 512 + 40 * max(seqs, 2000)),), 0xFF, dtype=torch.uint8, device="cuda")
    s2, d2 = ops.policy_loss(*args, workspace=ws, **kw)
    assert torch.equal(gs, s2) and torch.equal(gd, d2)


def test_policy_through_a_plan_reaches_the_loss(ops):
    """The objective's gradient by the chain policy_loss -> lm_loss_bwd, against fp64 on the unpacked tokens."""
    rng = np.random.default_rng(3)
    head = rng.integers(0, 500, 40)
    seqs = [np.concatenate([head, rng.integers(0, 500, n)]).astype(np.int32) for n in (17, 30, 25)]
    plan = ops.Plan.from_sequences(seqs, row_capacity=512, min_shared=8)
    dp = plan.to_device()
    F, R, C, V = plan.info["n_fwd"], plan.info["n_raw"], 64, 504
    h, w = _rnd(1, F, C), _rnd(2, V, C, std=0.3)
    nxt = np.concatenate([np.append(s[1:], -1) for s in seqs]).astype(np.int32)
    target = ops.gather_to_forwarded(dp, torch.from_numpy(nxt).cuda())
    loss, lse = ops.lm_loss(h, w, target)
    raw_loss = ops.scatter_token_index(dp.token_index, lse_src=loss[None])[1][0]
    weight = torch.from_numpy((nxt >= 0).astype(np.float32) / R).cuda()
    adv = _rnd(3, R, dtype=torch.float32)
    old = -raw_loss + _rnd(4, R, std=0.3, dtype=torch.float32)
    stats, dloss = ops.policy_loss(loss, old, adv, weight, dp.token_index, dp.fwd_raw_begin, dp.fwd_raw)
    dh, dw = ops.lm_loss_bwd(h, w, target, lse, dloss)
    # fp64, raw token by raw token
    H = h.double()[dp.token_index.long()].requires_grad_()
    W = w.double().requires_grad_()
    on = torch.nonzero(weight)[:, 0]
    logp = torch.log_softmax(H[on] @ W.T, 1).gather(1, torch.from_numpy(nxt).cuda()[on].long()[:, None])[:, 0]
    ratio = torch.exp(logp - old[on].double())
    A = adv[on].double()
    obj = -(weight[on].double() * torch.minimum(ratio * A, ratio.clamp(0.8, 1.2) * A)).sum()
    gH, gW = torch.autograd.grad(obj, (H, W))
    want = torch.zeros(F, C, dtype=torch.float64, device="cuda").index_add_(0, dp.token_index.long(), gH)
    assert abs(float(stats[0]) - float(obj)) <= 1e-5 * float((weight * adv.abs()).sum())
    for got, ref in ((dh, want), (dw, gW)):   # dz and the result in bf16
        assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -8
