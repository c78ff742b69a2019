"""Parity of the operators around the token mixers with their fp64 oracle.

Tolerances.  u = 2^-24 is fp32's rounding (half a step), b = 2^-8 bf16's.
 * embed: one fp32 product and one bf16 rounding: (b + 2u) |ref|.
 * embed_bwd: an fp32 sum of n terms and one product: (n + 2) u sum|terms|,
   plus b |ref| where the table's gradient is bf16.
 * block_norm: a row's statistic is a sum of C <= 16384 squares, at most 16 in
   a row per thread and then trees: its relative error is below 64 u; rsqrtf
   adds 2 ulp, the sigmoid (exp, add, divide; |gate| < 16) below 64 u, the
   products a few u.  So every factor of u, r, x is within 256 u = 2^-16 of
   its magnitude, and a result within 2^-16 of the sum of its terms'
   magnitudes, plus b |ref| for the bf16 outputs.  Its weights' gradients are
   fp32 sums over rows; with N <= 4096 rows no more than 256 are added in a
   row (the groups of rows in one thread, then the groups): 2^-16 again, so
   2^-15 of the sum of magnitudes.
 * lm_loss: a score is an fp32 sum of C products, each addition off by at most
   2u (truncation) of the running magnitude: C 2^-23 sum|h w|.  The softmax
   sum adds at most 256 * 16 + 512 terms in a row with exponentials of
   relative error 2^-22 (and of arguments |z| u): (4608 + 4) 2^-24 < 2^-11.8
   worst case for its logarithm with 16 tiles per unit; the shapes here have
   one tile per unit (up to 1,024 additions: 2^-14).
 * lm_loss_bwd: dz carries b (its bf16 form) plus the error of p, which is the
   score's and lse's absolute error times p; dh and dw add their own b.  The
   2-norm: two independent roundings, each at most b and b / sqrt(3) in the
   root mean square: 2^-8 sqrt(2/3) = 3.2e-3.  That mean needs many
   roundings.  With a handful of positions one element of dz, the target's
   (near -1, every other element 1e-4 of it or less), carries all but a
   vanishing share of dw's norm: dw = dz h^T is then that one rounded number
   times h, and its relative error is that number's, up to b in the worst
   case, plus the output's: b + b / sqrt(3) <= 6.2e-3.
"""
import ctypes

import numpy as np
import pytest
import torch

import workloads
from oracle import operators as oo

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8


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
    d = np.abs(_f64(got) - ref)
    at = np.argmax(d - tol) if d.size else 0
    assert np.all(d <= tol), "%s: off by %.3g where %.3g is allowed" % (what, d.flat[at],
                                                                       np.broadcast_to(tol, d.shape).flat[at])


# ---- embedding ------------------------------------------------------------------

EMBED = [(1, 8, 1), (1, 2048, 50), (33, 64, 7), (257, 120, 255), (1000, 1000, 256), (2049, 136, 65535),
         (5000, 264, 65536), (70, 4104, 40000)]


def _tokens(n, v, seed, kind):
    g = np.random.default_rng(seed)
    if kind == "uniform":
        t = g.integers(0, v, n)
    else:
        t = np.minimum(v - 1, np.exp(g.random(n) * np.log(v + 1.0)) - 1).astype(np.int64)
    t[g.random(n) < 0.1] = -1
    if n > 4:
        t[1], t[2] = v, -2 ** 31
    return t.astype(np.int32)


@pytest.mark.parametrize("n,c,v", EMBED)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embed(ops, n, c, v, dtype):
    table, tok = _rnd(1, v, c, dtype=dtype), _tokens(n, v, 2, "zipf")
    out = ops.embed(table, torch.from_numpy(tok).cuda(), scale=3.3)
    s = float(np.float32(3.3))
    ref = oo.embed(_f64(table), tok, s)
    _within(out, ref, (BF + 2 * U) * np.abs(ref), "embed")


@pytest.mark.parametrize("n,c,v", EMBED)
@pytest.mark.parametrize("kind", ["uniform", "zipf"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_embed_bwd(ops, n, c, v, kind, dtype):
    tok, dout = _tokens(n, v, 3, kind), _rnd(4, n, c)
    t = torch.from_numpy(tok).cuda()
    dirty = torch.full((v, c), float("nan"), dtype=dtype, device="cuda")   # every row is written
    got = ops.embed_bwd(t, dout, v, scale=0.7, dtable=dirty)
    s = float(np.float32(0.7))
    ref = oo.embed_bwd(tok, _f64(dout), v, s)
    mag = oo.embed_bwd(tok, np.abs(_f64(dout)), v, s)
    most = np.bincount(tok[(tok >= 0) & (tok < v)], minlength=1).max()
    tol = (most + 2) * U * mag + (BF * np.abs(ref) if dtype == torch.bfloat16 else 0)
    _within(got, ref, tol, "dtable")
    assert torch.equal(got, ops.embed_bwd(t, dout, v, scale=0.7, dtype=dtype))   # deterministic


@pytest.mark.parametrize("n,v", [(2048, 300), (2049, 300), (16383, 70), (16384, 5000), (1_048_576, 70000),
                                 (1_048_577, 70000)])
def test_embed_bwd_sizes_where_the_plan_changes(ops, n, v):
    """One sort tile and two, both piece lengths, both tile lengths; fp64 sums on the GPU."""
    tok, dout = torch.from_numpy(_tokens(n, v, 8, "zipf")).cuda(), _rnd(9, n, 8)
    got = ops.embed_bwd(tok, dout, v)
    at = torch.where((tok >= 0) & (tok < v), tok, v).long()
    ref = torch.zeros(v + 1, 8, dtype=torch.float64, device="cuda").index_add_(0, at, dout.double())[:v]
    mag = torch.zeros(v + 1, 8, dtype=torch.float64, device="cuda").index_add_(0, at, dout.double().abs())[:v]
    # additions in a row: a piece's 64, then the pieces of the longest run
    most = 64 + int(torch.bincount(at)[:v].max()) // 16 + 2
    assert ((got.double() - ref).abs() <= most * U * mag).all()


@pytest.mark.parametrize("n", [63, 64, 65, 128, 129, 5000])
def test_embed_bwd_one_id(ops, n):
    """A single run over every piece, alone and beside one other id at either end."""
    dout = _rnd(5, n, 72)
    for other in (None, 0, n - 1):
        tok = np.full(n, 4, np.int32)
        if other is not None:
            tok[other] = 2 if other == 0 else 6
        got = ops.embed_bwd(torch.from_numpy(tok).cuda(), dout, 9)
        _within(got, oo.embed_bwd(tok, _f64(dout), 9), (n + 2) * U * oo.embed_bwd(tok, np.abs(_f64(dout)), 9), "run")


def test_embed_bwd_masked_nan_and_empty(ops):
    # NaN rows of padding reach nothing; no positions at all: zeros
    dout = _rnd(6, 100, 64)
    tok = np.arange(100, dtype=np.int32) % 7
    tok[50:] = -1
    dout[50:] = float("nan")
    got = ops.embed_bwd(torch.from_numpy(tok).cuda(), dout, 7)
    assert torch.isfinite(got).all()
    z = ops.embed_bwd(torch.zeros(0, dtype=torch.int32, device="cuda"), _rnd(1, 0, 64), 5,
                      dtable=torch.ones(5, 64, device="cuda"))
    assert not z.any()
    assert ops.embed(_rnd(1, 5, 64), torch.zeros(0, dtype=torch.int32, device="cuda")).shape == (0, 64)
    all_pad = ops.embed_bwd(torch.full((300,), -1, dtype=torch.int32, device="cuda"), _rnd(7, 300, 64), 5)
    assert not all_pad.any()


# ---- norms around a block ----------------------------------------------------------

NORM = [(1, 8), (3, 64), (130, 264), (257, 512), (65, 520), (1000, 1000), (4096, 128), (300, 2048), (67, 2056),
        (40, 4096), (19, 8192), (9, 16384)]
FORMS = [(True, True, True), (True, False, True), (False, True, True), (False, False, True), (False, False, False)]


def _norm_inputs(n, c, post, gate, y, strided):
    a = {"res": _rnd(11, n, c, std=2.0), "w_pre": 1 + _rnd(12, c, std=0.2, dtype=torch.float32)}
    if y:
        a["y"] = _rnd(13, n, 3 * c)[:, c:2 * c] if strided else _rnd(13, n, c)
    if gate:
        a["gate"] = _rnd(14, n, 2 * c, std=3.0)[:, c:] if strided else _rnd(14, n, c, std=3.0)
    if post:
        a["w_post"] = 1 + _rnd(15, c, std=0.2, dtype=torch.float32)
    return a


@pytest.mark.parametrize("n,c", NORM)
@pytest.mark.parametrize("post,gate,y", FORMS)
def test_block_norm(ops, n, c, post, gate, y):
    a = _norm_inputs(n, c, post, gate, y, strided=c % 16 == 0)
    r, x = ops.block_norm(scale=0.5, eps=1e-5, **a)
    d = {k: _f64(t) for k, t in a.items()}
    eps = float(np.float32(1e-5))
    rr, rx = oo.block_norm(scale=0.5, eps=eps, **d)
    mag = np.abs(d["res"]) + np.abs(rr - d["res"])
    if y:
        _within(r, rr, BF * np.abs(rr) + 2.0 ** -16 * mag, "r")
    else:
        assert r is a["res"]
    rstd = 1 / np.sqrt(np.mean(rr * rr, axis=1, keepdims=True) + eps)
    _within(x, rx, BF * np.abs(rx) + 2.0 ** -15 * mag * rstd * np.abs(d["w_pre"]), "x")
    if y:   # in place
        r2, x2 = ops.block_norm(scale=0.5, eps=1e-5, **dict(a, res=a["res"].clone()), res_out=None)
        res = a["res"].clone()
        r3, x3 = ops.block_norm(scale=0.5, eps=1e-5, **dict(a, res=res), res_out=res)
        assert torch.equal(r3, r2) and torch.equal(x3, x2) and r3 is res


@pytest.mark.parametrize("n,c", NORM)
@pytest.mark.parametrize("post,gate,y", FORMS)
@pytest.mark.parametrize("with_dr", [True, False])
def test_block_norm_bwd(ops, n, c, post, gate, y, with_dr):
    a = _norm_inputs(n, c, post, gate, y, strided=c % 16 == 0)
    dx, dr = _rnd(16, n, c), _rnd(17, n, c) if with_dr else None
    kw = {}
    if y and c % 16 == 0:   # dy and dgate as column slices of one gradient
        wide = torch.full((n, 3 * c), 7.0, dtype=torch.bfloat16, device="cuda")
        kw["dy"] = wide[:, c:2 * c]
        if gate:
            kw["dgate"] = wide[:, 2 * c:]
    got = ops.block_norm_bwd(dx=dx, dres_out=dr, scale=0.5, eps=1e-5, **a, **kw)
    d = {k: _f64(t) for k, t in a.items()}
    eps = float(np.float32(1e-5))
    args = dict(dx=_f64(dx), dres_out=None if dr is None else _f64(dr), scale=0.5, eps=eps, **d)
    ref = oo.block_norm_bwd(**args)
    if kw:
        assert (wide[:, :c] == 7).all() and (gate or (wide[:, 2 * c:] == 7).all())   # the rest is left as it was
    # magnitudes of the terms
    r, _ = oo.block_norm(d["res"], d["w_pre"], d.get("y"), d.get("w_post"), d.get("gate"), 0.5, eps)
    rmag = np.abs(d["res"]) + np.abs(r - d["res"])
    rstd = 1 / np.sqrt(np.mean(r * r, axis=1, keepdims=True) + eps)
    rh = rmag * rstd
    dn = np.abs(args["dx"] * d["w_pre"])
    m_dr = rstd * (dn + rh * np.mean(dn * rh, axis=1, keepdims=True)) + (0 if dr is None else np.abs(args["dres_out"]))
    tol = 2.0 ** -15
    _within(got[0], ref[0], BF * np.abs(ref[0]) + tol * m_dr, "dres")
    _within(got[4], ref[4], tol * np.sum(np.abs(args["dx"]) * rh, axis=0), "dw_pre")
    if not y:
        assert got[1] is None and got[2] is None and got[3] is None
        return
    s = 1 / (1 + np.exp(-d["gate"])) if gate else 1.0
    yr = 1 / np.sqrt(np.mean(d["y"] ** 2, axis=1, keepdims=True) + eps) if post else 1.0
    yh = np.abs(d["y"]) * yr
    wp = np.abs(d["w_post"]) if post else 1.0
    m_d = 0.5 * m_dr
    if gate:
        # 1 - s is formed from s: its error is u, not relative to it
        _within(got[2], ref[2], BF * np.abs(ref[2]) + m_d * yh * wp * s * (tol * (1 - s) + 4 * U), "dgate")
    m_du = m_d * s
    if post:
        _within(got[3], ref[3], tol * np.sum(m_du * yh, axis=0), "dw_post")
        m_dy = yr * (m_du * wp + yh * np.mean(m_du * wp * yh, axis=1, keepdims=True))
    else:
        assert got[3] is None
        m_dy = m_du
    _within(got[1], ref[1], BF * np.abs(ref[1]) + tol * m_dy, "dy")
    again = ops.block_norm_bwd(dx=dx, dres_out=dr, scale=0.5, eps=1e-5, **a)
    assert all(p is None and q is None or torch.equal(p, q) for p, q in zip(got, again))


def test_block_norm_zero_rows_and_extremes(ops):
    """A row of zeros (eps alone under the root), saturated gates, no rows at all."""
    c = 256
    res, y = torch.zeros(2, 2, c, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(c, device="cuda")
    gate = torch.full((2, c), 1e4, dtype=torch.bfloat16, device="cuda")
    gate[1] = -1e4
    r, x = ops.block_norm(res, w, y=y, w_post=w, gate=gate)
    assert not r.any() and not x.any()
    y = _rnd(21, 2, c)
    r, _ = ops.block_norm(res, w, y=y, gate=gate)
    assert torch.equal(r[0], y[0]) and not r[1].any()
    g = ops.block_norm_bwd(res, w, _rnd(22, 2, c), y=y, gate=gate, w_post=w)
    assert all(torch.isfinite(t.float()).all() for t in g)
    e = _rnd(1, 0, c)
    assert ops.block_norm(e, w, y=e, w_post=w)[1].shape == (0, c)
    g = ops.block_norm_bwd(e, w, e, y=e, w_post=w, dw_pre=torch.ones(c, device="cuda"))
    assert not g[3].any() and not g[4].any()


# ---- loss over the vocabulary ---------------------------------------------------------

# (N, V, C, share of positions with a target)
LOSS = [(1, 1, 8, 1.0), (1, 32000, 64, 1.0), (3, 257, 8, 1.0), (255, 1000, 72, 0.5), (256, 256, 64, 1.0),
        (257, 5003, 128, 0.3), (700, 129, 1000, 0.9), (1030, 2049, 520, 0.02), (5, 4096, 2048, 0.8),
        (2600, 300, 64, 0.7), (600, 7000, 264, 0.0),
        # a few positions: one read of w (up to 16,384 values of h), and just above
        (2, 5003, 4096, 1.0), (2, 3, 8, 1.0), (3, 1000, 2048, 0.7), (4, 77, 4096, 1.0), (4, 20011, 64, 0.5),
        (2, 300, 8200, 1.0), (3, 100, 5464, 1.0), (1, 100, 16384, 1.0), (5, 1000, 64, 1.0)]


def _loss_inputs(n, v, c, on, seed=31):
    h, w = _rnd(seed, n, c), _rnd(seed + 1, v, c, std=2.0 / np.sqrt(c))
    g = np.random.default_rng(seed)
    t = g.integers(0, v, n)
    off = g.random(n) >= on
    t[off] = np.where(g.random(off.sum()) < 0.5, -1, v + g.integers(0, 1000, off.sum()))
    # what sits in positions without a target reaches nothing
    h[torch.from_numpy(np.flatnonzero(off)).cuda()] = float("nan")
    dl = g.normal(size=n).astype(np.float32)
    dl[off] = np.nan
    return h, w, t.astype(np.int32), dl


@pytest.mark.parametrize("n,v,c,on", LOSS)
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_lm_loss_and_gradients(ops, n, v, c, on, scale):
    h, w, t, dl = _loss_inputs(n, v, c, on)
    tt = torch.from_numpy(t).cuda()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    loss, lse = ops.lm_loss(h, w, tt, scale=scale, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    sc = float(np.float32(scale))
    hd, wd = np.nan_to_num(_f64(h)), _f64(w)
    r_loss, r_lse = oo.lm_loss(hd, wd, t, sc)
    valid = (t >= 0) & (t < v)
    e_z = c * 2.0 ** -23 * sc * (np.abs(hd) @ np.abs(wd).T).max(axis=1)        # a score's error
    tol = (e_z + 2.0 ** -14 + np.abs(r_lse) * 2.0 ** -21) * valid
    _within(lse, r_lse, tol, "lse")
    _within(loss, r_loss, 2 * tol, "loss")
    dh = torch.full_like(h, float("nan"))
    dw = torch.full_like(w, float("nan"))
    ops.lm_loss_bwd(h, w, tt, lse, torch.from_numpy(dl).cuda(), scale=scale, dh=dh, dw=dw, dev_err=err)
    torch.cuda.synchronize()
    assert int(err) == 0
    dl0 = np.where(valid, dl, 0).astype(np.float64)
    r_dh, r_dw = oo.lm_loss_bwd(hd, wd, t, dl0, sc)
    dz = np.zeros((n, v))
    dz[valid] = oo.score_grads(hd, wd, t, dl0, sc)
    hot = np.zeros((n, v))
    hot[valid, t[valid]] = 1.0
    p = dz + hot * (dl0 * sc)[:, None]                                          # coef * p
    e_dz = 2 * BF * np.abs(dz) + np.abs(p) * (2 * tol + 2.0 ** -20)[:, None]
    k = 2.0 ** -23
    _within(dh, r_dh, BF * np.abs(r_dh) + (1 + BF) * (e_dz @ np.abs(wd) + v * k * (np.abs(dz) @ np.abs(wd))), "dh")
    _within(dw, r_dw, BF * np.abs(r_dw) + (1 + BF) * (e_dz.T @ np.abs(hd) + n * k * (np.abs(dz).T @ np.abs(hd))), "dw")
    for got, ref in ((dh, r_dh), (dw, r_dw)):
        off = np.linalg.norm(_f64(got) - ref)
        # with one id the exact gradients vanish: what is left is the error of p alone
        few = 6.2e-3 if valid.sum() < 16 else 3.2e-3
        assert off <= few * np.linalg.norm(ref) + np.linalg.norm(np.abs(p) * (2 * tol)[:, None]) * np.sqrt(c) * 8, off
    again = ops.lm_loss_bwd(h, w, tt, lse, torch.from_numpy(dl).cuda(), scale=scale)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dw)              # deterministic


def test_lm_loss_scores_do_not_drift_with_the_width(ops):
    """Products of one sign, 16,384 channels: an accumulator that is truncated
    1,024 times drifts by up to 1024 * 2^-23.  A score is added up in chunks of
    512 channels: at most 32 truncations of one unit (2^-23) each, then 32
    roundings (2^-24) of the running sum; lse adds the logarithm and its own
    roundings of |lse| (2^-22)."""
    n, c = 300, 16384
    h, w = _rnd(55, n, c).abs(), _rnd(56, 3, c, std=0.01).abs()
    lse = ops.lm_loss(h, w, torch.zeros(n, dtype=torch.int32, device="cuda"))[1].double()
    ref = torch.logsumexp(h.double() @ w.double().T, 1)
    assert ((lse - ref).abs() <= (32 * 2.0 ** -23 + 32 * 2.0 ** -24 + 2.0 ** -22) * ref).all()


def test_lm_loss_pieces(ops):
    """More than one piece of the vocabulary: dz would take more than 4 GiB.
    Sampled rows of dh and dw against fp64."""
    n, v, c = 16384, 140003, 64
    h, w = _rnd(41, n, c), _rnd(42, v, c, std=0.25)
    g = np.random.default_rng(43)
    t = g.integers(0, v, n).astype(np.int32)
    t[::7] = -1
    tt = torch.from_numpy(t).cuda()
    dl = _rnd(44, n, dtype=torch.float32)
    loss, lse = ops.lm_loss(h, w, tt)
    dh, dw = ops.lm_loss_bwd(h, w, tt, lse, dl)
    rows = np.concatenate([g.integers(0, n, 16), [0, 1, n - 1]])
    cols = np.concatenate([g.integers(0, v, 16), [0, v - 1, 69999, 70000, 70143, 70144], t[t >= 0][:4]])
    hd, wd = h.double(), w.double()
    z = hd[rows] @ wd.T
    r_lse = torch.logsumexp(z, 1)
    on = tt[rows] >= 0
    want = torch.where(on, r_lse - z.gather(1, tt[rows].long().clamp(min=0)[:, None])[:, 0], 0.0)
    assert (loss[rows].double() - want).abs().max() <= 2 * (64 * 2.0 ** -23 * 64 + 2.0 ** -12)
    d = torch.softmax(z, 1)
    one = torch.ones(len(rows), 1, dtype=torch.float64, device="cuda")
    d.scatter_add_(1, tt[rows].long().clamp(min=0)[:, None], -one)
    d = d * torch.where(on, dl[rows].double(), 0.0)[:, None]
    ref = d @ wd
    assert (dh[rows].double() - ref).norm() <= 3.2e-3 * ref.norm()
    assert not dh[tt < 0].any()
    full_lse = torch.cat([torch.logsumexp(x @ wd.T, 1) for x in hd.split(2048)])
    p = torch.exp(hd @ wd[cols].T - full_lse[:, None])
    p = p - (tt[:, None] == torch.from_numpy(cols).cuda()[None]).double()
    p = p * torch.where(tt >= 0, dl.double(), 0.0)[:, None]
    ref = p.T @ hd
    assert (dw[cols].double() - ref).norm() <= 3.2e-3 * ref.norm()


def test_lm_loss_infinite_and_masked_everything(ops):
    # a score of +inf poisons its own row alone; no target anywhere: all zero
    h, w = _rnd(51, 300, 64), _rnd(52, 500, 64)
    h[7] = float("inf")
    t = torch.zeros(300, dtype=torch.int32, device="cuda")
    loss, lse = ops.lm_loss(h, w, t)
    assert torch.isnan(lse[7]) and torch.isfinite(lse[:7]).all() and torch.isfinite(lse[8:]).all()
    t.fill_(-1)
    loss, lse = ops.lm_loss(h, w, t)
    dh, dw = ops.lm_loss_bwd(h, w, t, lse, torch.full((300,), float("nan"), device="cuda"))
    assert not loss.any() and not lse.any() and not dh.any() and not dw.any()
    e = torch.zeros(0, dtype=torch.int32, device="cuda")
    f = torch.zeros(0, device="cuda")
    assert ops.lm_loss(_rnd(1, 0, 64), w, e)[0].numel() == 0
    assert not ops.lm_loss_bwd(_rnd(1, 0, 64), w, e, f, f, dw=torch.ones_like(w))[1].any()


# ---- streams, graphs, offsets ---------------------------------------------------------

def _all_ops(ops, s, out):
    out["emb"] = ops.embed(s["table"], s["tok"], scale=2.0)
    out["r"], out["x"] = ops.block_norm(out["emb"], s["w"], y=s["y"], w_post=s["w"], gate=s["gate"])
    out["loss"], out["lse"] = ops.lm_loss(out["x"], s["table"], s["tok"])
    out["dh"], out["dw"] = ops.lm_loss_bwd(out["x"], s["table"], s["tok"], out["lse"], s["dl"])
    out["g"] = ops.block_norm_bwd(out["emb"], s["w"], out["dh"], y=s["y"], w_post=s["w"], gate=s["gate"])
    out["dt"] = ops.embed_bwd(s["tok"], out["g"][0], 900)
    return out


def _state(seed, n=600, c=128, v=900):
    tok = torch.from_numpy(_tokens(n, v, seed, "zipf")).cuda()
    return {"table": _rnd(seed, v, c), "tok": tok, "y": _rnd(seed + 1, n, c), "gate": _rnd(seed + 2, n, c),
            "w": 1 + _rnd(seed + 3, c, std=0.1, dtype=torch.float32), "dl": _rnd(seed + 4, n, dtype=torch.float32)}


def _same(a, b):
    for k in a:
        xs, ys = (a[k], b[k]) if isinstance(a[k], tuple) else ((a[k],), (b[k],))
        for x, y in zip(xs, ys):
            assert torch.equal(x, y), k


def test_on_another_stream_and_in_a_graph(ops):
    s = _state(61)
    want = _all_ops(ops, s, {})
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = _all_ops(ops, s, {})
    side.synchronize()
    _same(got, want)
    graph, static = torch.cuda.CUDAGraph(), {}
    with torch.cuda.graph(graph):
        _all_ops(ops, s, static)
    for seed in (62, 63):
        other = _state(seed)
        for k in s:
            s[k].copy_(other[k])
        graph.replay()
        torch.cuda.synchronize()
        _same(static, _all_ops(ops, s, {}))


def test_two_calls_at_once(ops):
    """Two streams, each with its own workspaces, run the same calls together."""
    a, b = _state(71), _state(72)
    wa, wb = _all_ops(ops, a, {}), _all_ops(ops, b, {})
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ga, gb = [], []
    for _ in range(5):
        with torch.cuda.stream(s1):
            ga.append(_all_ops(ops, a, {}))
        with torch.cuda.stream(s2):
            gb.append(_all_ops(ops, b, {}))
    torch.cuda.synchronize()
    for x in ga:
        _same(x, wa)
    for x in gb:
        _same(x, wb)


def test_offsets_past_32_bits(ops):
    """Element offsets above 2^31: the last rows of a long table and of long activations."""
    v, c = 1_100_000, 2048
    table = torch.zeros(v, c, dtype=torch.bfloat16, device="cuda")
    table[-5:] = _rnd(81, 5, c)
    tok = torch.tensor([v - 1, 0, v - 5, v - 2], dtype=torch.int32, device="cuda")
    out = ops.embed(table, tok)
    assert torch.equal(out, table[tok.long()])
    g = ops.embed_bwd(tok, out, v, dtype=torch.bfloat16)
    assert torch.equal(g[[v - 1, v - 5, v - 2]], out[[0, 2, 3]]) and not g[v - 4].any() and not g[1].any()
    del g
    w = torch.ones(c, device="cuda")
    r, x = ops.block_norm(table, w, y=table)
    r5, x5 = ops.block_norm(table[-5:].contiguous(), w, y=table[-5:].contiguous())
    assert torch.equal(r[-5:], r5) and torch.equal(x[-5:], x5)
    del r, x
    got = ops.block_norm_bwd(table, w, table, y=table)
    one = ops.block_norm_bwd(table[-5:].contiguous(), w, table[-5:].contiguous(), y=table[-5:].contiguous())
    assert torch.equal(got[0][-5:], one[0]) and torch.equal(got[1][-5:], one[1])
    del got
    h = _rnd(82, 3, c, std=0.05)
    t = torch.tensor([v - 1, 5, v - 2], dtype=torch.int32, device="cuda")
    loss, lse = ops.lm_loss(h, table, t)
    z = h.double() @ table[-5:].double().T
    want = torch.log(torch.exp(z).sum(1) + (v - 5))
    assert (lse.double() - want).abs().max() <= 2.0 ** -11
    dh, dw = ops.lm_loss_bwd(h, table, t, lse, torch.ones(3, device="cuda"))
    ref = (torch.exp(z - want[:, None]).T @ h.double())
    ref[4] -= h[0].double()
    ref[3] -= h[2].double()
    assert (dw[-5:].double() - ref).norm() <= 3.2e-3 * ref.norm()


# ---- together, as a training step uses them ------------------------------------------------

def test_training_step_over_a_packed_tree(ops):
    """Token ids of a packed tree -> embedding -> norm -> tree attention ->
    norm, gate and residual -> loss weighted per raw token, and back, against
    fp64 automatic differentiation of the same layers over dense ancestor
    masks.  About ten bf16 roundings lie between the ids and a gradient, each
    at most 2^-8 and 2^-8/sqrt(3) in the root mean square: 7.2e-3, and the
    attention's own (P, dS): twice that bounds the sum."""
    w = workloads.get("tiny_fit")
    plan = ops.Plan.from_sequences(w.sequences, group_ids=w.group_ids, row_capacity=w.row_capacity,
                                   min_shared=w.min_shared)
    dp = plan.to_device()
    F, V, H, d = plan.info["n_fwd"], workloads.VOCAB, 2, 64
    C = H * d
    table = _rnd(91, V, C, std=0.5)
    w1, w2 = (1 + _rnd(s, C, std=0.1, dtype=torch.float32) for s in (92, 93))
    wp = 1 + _rnd(94, C, std=0.1, dtype=torch.float32)
    gate = _rnd(95, F, C)
    raw = torch.from_numpy(w.flat_tokens()).cuda()
    nxt = np.concatenate([np.append(s[1:], -1) for s in w.sequences]).astype(np.int32)   # next token, none at the end
    weight = _rnd(96, 1, plan.info["n_raw"], dtype=torch.float32)
    tok = ops.gather_to_forwarded(dp, raw)
    tgt = ops.gather_to_forwarded(dp, torch.from_numpy(nxt).cuda())
    _, dl = ops.sum_to_forwarded(dp, lse_src=weight)
    dl = dl[0]

    emb = ops.embed(table, tok)
    _, x = ops.block_norm(emb, w1)
    qkv = x.view(F, H, d)
    q, k = ops.rope_by_depth(qkv.clone(), qkv.clone(), dp.depth, 1e4)
    o, lse_a = ops.tree_attn_fwd(dp, q, k, qkv)
    r, xo = ops.block_norm(emb, w2, y=o.view(F, C), w_post=wp, gate=gate, scale=0.7)
    loss, lse = ops.lm_loss(xo, table, tgt)
    dxo, dout_w = ops.lm_loss_bwd(xo, table, tgt, lse, dl)
    demb, do, dgate, dwp, dw2 = ops.block_norm_bwd(emb, w2, dxo, y=o.view(F, C), w_post=wp, gate=gate, scale=0.7)
    dq, dk, dv = ops.tree_attn_bwd(dp, q, k, qkv, o, lse_a, do.view(F, H, d), rope_base=1e4)
    dx = (dq.float() + dk.float() + dv.float()).bfloat16().view(F, C)
    demb2, _, _, _, dw1 = ops.block_norm_bwd(emb, w1, dx, dres_out=demb)
    dtable = ops.embed_bwd(tok, demb2, V)

    T = table.double().requires_grad_(True)
    G, W1, W2, WP = (a.double().requires_grad_(True) for a in (gate, w1, w2, wp))
    To = table.double().requires_grad_(True)

    def norm(a):
        return a / (a.square().mean(1, keepdim=True) + 1e-6).sqrt()
    E = T[tok.long()]
    X = (norm(E) * W1).view(F, H, d)
    ang = dp.depth.double()[:, None] * 1e4 ** (-torch.arange(0, d, 2, device="cuda").double() / d)
    cs, sn = ang.cos()[:, None], ang.sin()[:, None]
    R = torch.cat([X[..., :d // 2] * cs - X[..., d // 2:] * sn, X[..., d // 2:] * cs + X[..., :d // 2] * sn], -1)
    i = torch.arange(F, device="cuda")
    seen = (i[None] <= i[:, None]) & (i[:, None] < dp.subtree_end.long()[None])
    S = torch.einsum("fhd,ghd->hfg", R, R) / d ** 0.5
    O = torch.einsum("hfg,ghd->fhd", torch.softmax(S.masked_fill(~seen, float("-inf")), -1), X).reshape(F, C)
    XO = norm(E + 0.7 * torch.sigmoid(G) * norm(O) * WP) * W2
    on = tgt >= 0
    Z = XO @ To.T
    L = torch.where(on, torch.logsumexp(Z, 1) - Z.gather(1, tgt.long().clamp(min=0)[:, None])[:, 0], 0.0)
    (L * dl.double()).sum().backward()
    for got, ref, name in ((loss, L, "loss"), (dtable, T.grad, "dtable"), (dout_w, To.grad, "projection"),
                           (dgate, G.grad, "dgate"), (dw1, W1.grad, "dw1"), (dw2, W2.grad, "dw2"),
                           (dwp, WP.grad, "dw_post")):
        off = float((got.double() - ref.detach()).norm() / ref.detach().norm())
        assert off <= 1.5e-2, (name, off)
    # the loss of the packed positions weighted by sums over their raw tokens
    # is the loss of the raw tokens
    raw_loss, total = loss[dp.token_index.long()].double(), (loss.double() * dl.double()).sum()
    assert torch.isclose((raw_loss * weight[0].double()).sum(), total, rtol=1e-5, atol=1e-4)


# ---- nothing but the outputs is written, nothing but the inputs is read ----------------------

def _inside(rows, cols, dtype, fill):
    """(view of rows x cols, whole buffer): five guard rows of ``fill`` on either side."""
    buf = torch.full((rows + 10, cols), fill, dtype=dtype, device="cuda")
    return buf[5:5 + rows], buf


def _guards_whole(buf, rows, fill):
    return bool((buf[:5] == fill).all()) and bool((buf[5 + rows:] == fill).all())


def _dirty(need):
    """A workspace of exactly ``need`` bytes of 0xFF (NaN, -1), and what lies behind it."""
    buf = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    return buf[:need], buf[need:]


@pytest.mark.parametrize("n,v,c", [(3, 300, 64), (700, 1000, 72), (257, 513, 264), (2100, 333, 520), (4100, 900, 40),
                                   (5000, 9000, 264)])
def test_outputs_and_workspaces_keep_to_their_bounds(ops, n, v, c):
    from prefix_tree_packed_dfs_gb300 import binding
    lib = binding.load()
    tok = torch.from_numpy(_tokens(n, v, 101, "zipf")).cuda()
    table, y, gate = _rnd(102, v, c), _rnd(103, n, c), _rnd(104, n, c)
    w = 1 + _rnd(105, c, std=0.1, dtype=torch.float32)
    dl = _rnd(106, n, dtype=torch.float32)

    def both(fn, shapes, need):
        """fn into guarded outputs with a dirty workspace of the least size, and plainly."""
        outs = [_inside(r, k, t, 3.0) for r, k, t in shapes]
        ws, behind = _dirty(need)
        fn([o[0] for o in outs], ws if need else None)
        plain = [torch.empty(r, k, dtype=t, device="cuda") for r, k, t in shapes]
        fn(plain, None)
        for (o, buf), p, (r, _, _) in zip(outs, plain, shapes):
            assert _guards_whole(buf, r, 3.0) and torch.equal(o, p)
        assert (behind == 255).all()
        return plain

    bf, f32 = torch.bfloat16, torch.float32
    (emb,) = both(lambda o, ws: ops.embed(table, tok, out=o[0]), [(n, c, bf)], 0)
    both(lambda o, ws: ops.embed_bwd(tok, y, v, dtable=o[0], workspace=ws), [(v, c, f32)],
         lib.tpk_embed_bwd_workspace_bytes(n, v, c))
    r, x = both(lambda o, ws: ops.block_norm(emb, w, y=y, w_post=w, gate=gate, res_out=o[0], out=o[1]),
                [(n, c, bf), (n, c, bf)], 0)
    both(lambda o, ws: ops.block_norm_bwd(emb, w, x, dres_out=r, y=y, w_post=w, gate=gate, dres=o[0], dy=o[1],
                                          dgate=o[2], dw_post=o[3].view(c), dw_pre=o[4].view(c), workspace=ws),
         [(n, c, bf), (n, c, bf), (n, c, bf), (1, c, f32), (1, c, f32)], lib.tpk_block_norm_bwd_workspace_bytes(n, c))
    loss, lse = both(lambda o, ws: ops.lm_loss(x, table, tok, loss=o[0].view(n), lse=o[1].view(n), workspace=ws),
                     [(n, 1, f32), (n, 1, f32)], lib.tpk_lm_loss_workspace_bytes(n, v, c, 0))
    both(lambda o, ws: ops.lm_loss_bwd(x, table, tok, lse.view(n), dl, dh=o[0], dw=o[1], workspace=ws),
         [(n, c, bf), (v, c, bf)], lib.tpk_lm_loss_workspace_bytes(n, v, c, 1))


def test_ids_and_weights_of_one_element_alignment(ops):
    """Ids, targets, lse and loss weights need no more than their own alignment."""
    n, v, c = 1500, 700, 64
    whole = torch.from_numpy(_tokens(n + 1, v, 111, "uniform")).cuda()
    tok = whole[1:]
    assert tok.data_ptr() % 16
    table, h = _rnd(112, v, c), _rnd(113, n, c)
    assert torch.equal(ops.embed(table, tok), ops.embed(table, tok.clone()))
    assert torch.equal(ops.embed_bwd(tok, h, v), ops.embed_bwd(tok.clone(), h, v))
    a, b = ops.lm_loss(h, table, tok), ops.lm_loss(h, table, tok.clone())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    dl = _rnd(114, n + 1, dtype=torch.float32)[1:]
    lse = torch.cat([a[1][:1], a[1]])[1:]
    p, q = ops.lm_loss_bwd(h, table, tok, lse, dl), ops.lm_loss_bwd(h, table, tok.clone(), a[1], dl.clone())
    assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])
    # the norms' weights are read 16 bytes at a time: other addresses are refused
    from prefix_tree_packed_dfs_gb300.binding import TpkError
    with pytest.raises(TpkError):
        ops.block_norm(h, torch.ones(c + 1, device="cuda")[1:])


def test_the_same_position_sets_in_any_company(ops):
    """A position's loss and gradient do not depend on how many others have no
    target: the same rows alone, and scattered among rows without one."""
    n, v, c = 900, 1200, 128
    h, w = _rnd(121, n, c), _rnd(122, v, c, std=0.2)
    t = torch.from_numpy((np.random.default_rng(123).integers(0, v, n)).astype(np.int32)).cuda()
    dl = _rnd(124, n, dtype=torch.float32)
    loss, lse = ops.lm_loss(h, w, t)
    dh, dw = ops.lm_loss_bwd(h, w, t, lse, dl)
    at = torch.sort(torch.randperm(5 * n, generator=torch.Generator().manual_seed(125))[:n]).values.cuda()
    hs = torch.full((5 * n, c), float("nan"), dtype=torch.bfloat16, device="cuda")
    ts = torch.full((5 * n,), -7, dtype=torch.int32, device="cuda")
    ds = torch.full((5 * n,), float("inf"), device="cuda")
    hs[at], ts[at], ds[at] = h, t, dl
    loss2, lse2 = ops.lm_loss(hs, w, ts)
    dh2, dw2 = ops.lm_loss_bwd(hs, w, ts, lse2, ds)
    assert torch.equal(loss2[at], loss) and torch.equal(lse2[at], lse)
    assert torch.equal(dh2[at], dh) and torch.equal(dw2, dw)
    rest = torch.ones(5 * n, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert not loss2[rest].any() and not lse2[rest].any() and not dh2[rest].any()


def test_lm_loss_long_batch(ops):
    """600,000 positions of width 3,600: more than 2^31 elements of h, of dh and
    of a piece's dz, two pieces, rows that are copied to be aligned.  Sampled
    rows of dh and dw against fp64 (dw by the lse under test, sampled too)."""
    n, v, c = 600_000, 8000, 3600
    w = _rnd(131, v, c, std=0.03)
    h = torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(132)
    for part in h.split(50_000):
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda"))
    g = np.random.default_rng(133)
    t = g.integers(0, v, n).astype(np.int32)
    t[g.random(n) < 0.1] = -1
    tt = torch.from_numpy(t).cuda()
    dl = _rnd(134, n, dtype=torch.float32)
    loss, lse = ops.lm_loss(h, w, tt)
    dh, dw = ops.lm_loss_bwd(h, w, tt, lse, dl)
    rows = np.concatenate([g.integers(0, n, 24), [0, 1, n - 2, n - 1]])
    cols = np.concatenate([g.integers(0, v, 8), [0, 4095, 4096, v - 1]])
    on = tt[rows] >= 0
    z = h[rows].double() @ w.double().T
    r_lse = torch.where(on, torch.logsumexp(z, 1), 0.0)
    # a score: 32 truncations (2^-23) per chunk of 512 channels and 8 roundings
    # of the sum, of sum|h w| = 3600 * 0.03 * 2 / pi = 69; the softmax sum 2^-14
    assert (lse[rows].double() - r_lse).abs().max() <= (32 * 2.0 ** -23 + 8 * 2.0 ** -24) * 80 + 2.0 ** -14
    d = torch.softmax(z, 1)
    d.scatter_add_(1, tt[rows].long().clamp(min=0)[:, None],
                   -torch.ones(len(rows), 1, dtype=torch.float64, device="cuda"))
    ref = (d * torch.where(on, dl[rows].double(), 0.0)[:, None]) @ w.double()
    assert (dh[rows].double() - ref).norm() <= 3.2e-3 * ref.norm()
    for i in np.flatnonzero(t < 0)[[0, -1]]:
        assert not dh[i].any()
    ref = torch.zeros(len(cols), c, dtype=torch.float64, device="cuda")
    wc, ids = w[cols].double(), torch.from_numpy(cols).cuda()
    for lo in range(0, n, 50_000):
        at = slice(lo, min(n, lo + 50_000))
        hd = h[at].double()
        p = torch.exp(hd @ wc.T - lse[at].double()[:, None]) - (tt[at, None] == ids[None]).double()
        ref += (p * torch.where(tt[at] >= 0, dl[at].double(), 0.0)[:, None]).T @ hd
    assert (dw[cols].double() - ref).norm() <= 3.2e-3 * ref.norm()


def test_calls_from_two_host_threads(ops):
    """Two threads, a stream each, first calls of some shapes included."""
    import threading
    states = [_state(141), _state(142, n=333, c=200, v=1111)]
    want = []
    out, errs = [None, None], []

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(4):
                    s = states[i]
                    r = {}
                    r["emb"] = ops.embed(s["table"], s["tok"])
                    r["r"], r["x"] = ops.block_norm(r["emb"], s["w"], y=s["y"], w_post=s["w"], gate=s["gate"])
                    r["loss"], r["lse"] = ops.lm_loss(r["x"], s["table"], s["tok"])
                    r["dh"], r["dw"] = ops.lm_loss_bwd(r["x"], s["table"], s["tok"], r["lse"], s["dl"])
                    r["dt"] = ops.embed_bwd(s["tok"], r["dh"], s["table"].shape[0])
                    out[i] = r
            st.synchronize()
        except Exception as e:      # reported by the test's own thread
            errs.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errs, errs
    both, out = out, [None, None]
    for i in range(2):
        work(i)
        want.append(out[i])
        _same(both[i], want[i])
