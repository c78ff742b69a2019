"""Where the operators' results are small differences or long sums of one sign,
against plain fp64 torch on the GPU.

u = 2^-24 is fp32's rounding (half a step), b = 2^-8 bf16's.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U, BF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _rnd(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


@pytest.mark.parametrize("n", [1, 4, 5, 300, 3000])
@pytest.mark.parametrize("c", [1000, 4096])
def test_lm_loss_gradient_of_confident_targets(ops, n, c):
    """Targets of probability 1 - 1e-2 to 1 - 1e-5 (scores of 15 to 22): the
    target's element of dz is the small difference p - 1.  Its error is that of
    exp(z - lse): lse is an fp32 number (|lse| u), its sum near 1 has some 20
    additions (20 u), ex2's relative error is 2^-22 (4 u); the scores
    themselves are the forward's.  dz and dh round by b each, the other
    elements (p_v > 0, together 1 - p) too, and their scores' errors stay below
    2^-12: per row of dh, with W the longest row of w,
    |dh - ref| <= W |dloss| (4 b (1 - p) + (|lse| + 24) u)."""
    v = 20000
    w = _rnd(200, v, c, std=0.05)
    g = np.random.default_rng(201)
    t = g.permutation(v)[:n].astype(np.int32)
    tt = torch.from_numpy(t).cuda()
    miss = 10.0 ** -np.linspace(2, 5, n)                       # 1 - p
    z = torch.from_numpy(np.log(v / miss)).cuda()
    wt = w[tt.long()].double()
    h = (wt * (z / (wt * wt).sum(1))[:, None]).bfloat16()      # products of one sign
    dl = _rnd(202, n, dtype=torch.float32)
    loss, lse = ops.lm_loss(h, w, tt)
    dh, _ = ops.lm_loss_bwd(h, w, tt, lse, dl)
    wd = w.double()
    logp = torch.log_softmax(h.double() @ wd.T, 1)
    at = torch.arange(n, device="cuda")
    r_loss = -logp[at, tt.long()]
    assert float(r_loss.max()) > 3e-3 and (n < 4 or float(r_loss.min()) < 4e-5)
    p = logp.exp()
    p[at, tt.long()] = torch.expm1(-r_loss)
    ref = (p * dl.double()[:, None]) @ wd
    off = (dh.double() - ref).norm(dim=1)
    most = wd.norm(dim=1).max()
    tol = most * dl.double().abs() * (4 * BF * -torch.expm1(-r_loss) + (lse.double().abs() + 24) * U)
    worst = int((off - tol).argmax())
    assert (off <= tol).all(), (worst, float(off[worst]), float(tol[worst]), float(ref[worst].norm()))


@pytest.mark.parametrize("n,v,c", [(700, 129, 1000), (257, 513, 4096), (3000, 1200, 1000), (5, 4096, 2048),
                                   (2, 5003, 4096), (4, 77, 4096), (1, 100, 16384), (300, 40, 16384)])
@pytest.mark.parametrize("scale", [1.0, 0.7])
def test_lm_loss_gradients_in_the_two_norm_at_wide_rows(ops, n, v, c, scale):
    """dz and the result each round by b at most, b / sqrt 3 in the root mean
    square: b sqrt(2/3) = 3.2e-3.  With a handful of positions the targets'
    elements carry dw, each a single rounding of dz: b + b / sqrt 3.  Scores
    (standard deviation 2) are within 1e-5: a hundredth of that."""
    h, w = _rnd(241, n, c), _rnd(242, v, c, std=2.0 / c ** 0.5)
    tt = torch.from_numpy(np.random.default_rng(243).integers(0, v, n).astype(np.int32)).cuda()
    dl = _rnd(244, n, dtype=torch.float32)
    _, lse = ops.lm_loss(h, w, tt, scale=scale)
    dh, dw = ops.lm_loss_bwd(h, w, tt, lse, dl, scale=scale)
    sc = float(np.float32(scale))
    hd, wd = h.double(), w.double()
    p = torch.softmax(sc * (hd @ wd.T), 1)
    p[torch.arange(n, device="cuda"), tt.long()] -= 1
    dz = p * (dl.double() * sc)[:, None]
    most = BF * (2 / 3) ** 0.5 if n >= 16 else BF * (1 + 3 ** -0.5)
    for got, ref in ((dh, dz @ wd), (dw, dz.T @ hd)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 1.01 * most


def test_lm_loss_gradient_of_few_positions_in_the_second_piece(ops):
    """9,000,000 ids: more than the 8,388,608 of one piece of dz.  A target of
    probability 1 - p = 1e-4 in either piece, and next to the border."""
    n, v, c = 4, 9_000_000, 8
    w = _rnd(261, v, c, std=0.1)
    tt = torch.tensor([5, 8_388_607, 8_388_608, v - 1], dtype=torch.int32, device="cuda")
    w[tt.long()] = torch.eye(8, device="cuda").bfloat16()[:4] * 8
    h = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
    h[torch.arange(4), torch.arange(4)] = 3.25                       # score 26; ln(9e6) = 16
    dl = torch.ones(n, device="cuda")
    _, lse = ops.lm_loss(h, w, tt)
    dh, dw = ops.lm_loss_bwd(h, w, tt, lse, dl)
    logp = torch.log_softmax(h.double() @ w.double().T, 1)
    at = torch.arange(n, device="cuda")
    miss = -torch.expm1(logp[at, tt.long()])
    assert 1e-5 < float(miss.min()) and float(miss.max()) < 1e-3
    p = logp.exp()
    p[at, tt.long()] = -miss
    # the bound of the confident targets above; |w| of the targets is 8
    tol = 8 * (4 * BF * miss + (lse.double().abs() + 24) * U)
    assert ((dh.double() - p @ w.double()).norm(dim=1) <= tol).all()
    # dw of a target: dz h, another rounding, and what the other positions add
    ref = p[:, tt.long()].T @ h.double()
    assert ((dw[tt.long()].double() - ref).norm(dim=1) <= 3.25 * (4 * BF * miss + (lse.double().abs() + 24) * U)).all()


def _relative_mean(got, ref):
    return float(((got.double() - ref) / ref).mean())


# A long sum of one sign: an accumulation of n truncations, each below one unit
# (2 u) of the running value, is low by at most n u of its result (half of them
# at full magnitude).  The accumulations are of 2,048 elements, 128 instructions
# of 16 products with two truncations each, added up with rounding to nearest.
# What else is not zero in the mean is small: the exponentials (2^-22) and lse
# (|lse| u).  The bf16 roundings of the results are: their mean over the M
# elements looked at is within 4 b / (2 sqrt M).
STEPS = 256


def test_lm_loss_dw_of_a_long_batch_of_one_sign(ops):
    """200,000 positions, all of one target: dw of the other ids is a sum of
    200,000 positive terms (320 tiles of dw: no split over the positions)."""
    n, v, c = 200_000, 8192, 2560
    scale = torch.rand(c, generator=torch.Generator(device="cuda").manual_seed(211), device="cuda") * 1.5 + 0.5
    h = torch.empty(n, c, dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate(h.split(50_000)):
        part.copy_(_rnd(212 + i, *part.shape, dtype=torch.float32).abs() * scale)
    w = _rnd(216, v, c, std=0.01)
    tt = torch.zeros(n, dtype=torch.int32, device="cuda")
    dl = torch.full((n,), 2.0 ** -10, device="cuda")
    _, lse = ops.lm_loss(h, w, tt)
    _, dw = ops.lm_loss_bwd(h, w, tt, lse, dl)
    ids = torch.arange(1, v, 509, device="cuda")
    ref = torch.zeros(len(ids), c, dtype=torch.float64, device="cuda")
    for lo in range(0, n, 50_000):
        hd = h[lo:lo + 50_000].double()
        ref += torch.exp(hd @ w[ids].double().T - lse[lo:lo + 50_000].double()[:, None]).T @ hd * 2.0 ** -10
    tol = STEPS * U + 2.0 ** -22 + float(lse.abs().max()) * U + 2 * BF / ref.numel() ** 0.5
    assert abs(_relative_mean(dw[ids], ref)) <= tol


def test_lm_loss_dh_of_a_large_vocabulary_of_one_sign(ops):
    """262,144 ids with positive rows and a target whose row is zero: dh is a
    sum of 262,144 positive terms (320 tiles of dh: no split over the ids)."""
    n, v, c = 8192, 262_144, 2560
    scale = torch.rand(c, generator=torch.Generator(device="cuda").manual_seed(221), device="cuda") * 1.5 + 0.5
    w = torch.empty(v, c, dtype=torch.bfloat16, device="cuda")
    for i, part in enumerate(w.split(65_536)):
        part.copy_(_rnd(222 + i, *part.shape, dtype=torch.float32).abs() * scale)
    w[7] = 0
    h = _rnd(226, n, c, std=0.01)
    tt = torch.full((n,), 7, dtype=torch.int32, device="cuda")
    _, lse = ops.lm_loss(h, w, tt)
    dh, _ = ops.lm_loss_bwd(h, w, tt, lse, torch.ones(n, device="cuda"))
    rows = torch.arange(3, n, 257, device="cuda")
    ref = torch.zeros(len(rows), c, dtype=torch.float64, device="cuda")
    for lo in range(0, v, 65_536):
        wd = w[lo:lo + 65_536].double()
        ref += torch.exp(h[rows].double() @ wd.T - lse[rows].double()[:, None]) @ wd
    tol = STEPS * U + 2.0 ** -22 + float(lse.abs().max()) * U + 2 * BF / ref.numel() ** 0.5
    assert abs(_relative_mean(dh[rows], ref)) <= tol


def test_lm_loss_of_many_small_probabilities(ops):
    """A target with score 17 against 31,999 ids with score 0: each adds e^-17,
    less than half a step of the sum that already holds the target's 1.  The
    loss may miss what is added onto that 1 element by element: the 15 other
    columns of the target's own accumulator in its tile, then an addition per
    tile of its run (16 at most), per slot (2 * 16) and in the joining tree
    (5), each off by u, 2^-22 of the exponentials and two roundings of the
    small loss itself."""
    n, v, c = 96_888, 32_000, 8
    h = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 17.0
    w = torch.zeros(v, c, dtype=torch.bfloat16, device="cuda")
    ref = float(np.log1p((v - 1) * np.exp(-17.0)))
    for target in (0, 64, 16_000):
        w.zero_()
        w[target, 0] = 1.0
        loss, _ = ops.lm_loss(h, w, torch.full((n,), target, dtype=torch.int32, device="cuda"))
        assert float((loss.double() - ref).abs().max()) <= (15 + 16 + 32 + 5) * U + ref * (2.0 ** -22 + 2 * U)


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("c", [64, 520, 2048, 16384])
def test_block_norm_gradient_of_saturated_gates(ops, post, c):
    """dgate = d u s (1 - s), s = sigmoid(gate): relative at both ends, where
    s or 1 - s is e^-|gate|.  s, 1 - s, u and d are within 2^-16 of their terms'
    magnitudes each (a row's statistics 64 u, 2^x of |gate| <= 80 another 80 u),
    their product within 2^-15 and a bf16 rounding b.  At |gate| = 80 some
    products lie below the least normal number 2^-126: there fp32 and bf16 have
    fewer bits or flush to zero, both off by less than 2^-126."""
    n = 34
    gates = torch.tensor([12.0, -12.0, 20.0, -20.0, 9.0, -9.0, 40.0, -40.0, 80.0, -80.0, 0.0, 3.0, -3.0, 16.0, 17.5,
                          30.0, -30.0], device="cuda")
    gate = gates.repeat(2)[:, None].expand(n, c).contiguous().bfloat16()
    res, y, dr = _rnd(231, n, c), _rnd(232, n, c), _rnd(233, n, c)
    one = torch.ones(c, device="cuda")
    wp = 1 + _rnd(234, c, std=0.1, dtype=torch.float32) if post else None
    # no gradient through the second norm: d = scale * dres_out alone
    got = ops.block_norm_bwd(res, one, torch.zeros_like(res), dres_out=dr, y=y, w_post=wp, gate=gate, scale=0.5)[2]
    u = y.double()
    if post:
        u = u / (u.square().mean(1, keepdim=True) + 1e-6).sqrt() * wp.double()
    g = gate.double()
    ref = 0.5 * dr.double() * u * torch.sigmoid(g) * torch.sigmoid(-g)
    assert ((got.double() - ref).abs() <= (BF + 2.0 ** -15) * ref.abs() + 2.0 ** -126).all()


@pytest.mark.parametrize("post", [True, False])
def test_block_norm_gradient_of_gates_that_are_no_numbers(ops, post):
    """A NaN gate makes its whole row NaN, as r there is NaN, and no other row;
    infinite gates are an open and a closed one."""
    n, c = 9, 264
    res, y, dr, dx = (_rnd(s, n, c) for s in (251, 252, 253, 254))
    one = torch.ones(c, device="cuda")
    wp = one if post else None
    gate = torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
    gate[3, 5] = float("nan")
    gate[6], gate[7] = float("inf"), float("-inf")
    dres, dy, dgate = ops.block_norm_bwd(res, one, dx, dres_out=dr, y=y, w_post=wp, gate=gate)[:3]
    for t in (dres, dy):
        assert torch.isnan(t[3]).all() and torch.isfinite(t[:3]).all() and torch.isfinite(t[4:]).all()
    assert torch.isnan(dgate[3]).all()
    assert not dgate[6:8].any() and not dy[7].any() and dy[6].any()
