"""The products of the projections in every form that their sizes can take: which
form a size takes (CPU), and the results of each (GPU), with bias, activation and
residual.

References in fp64 with torch on the GPU.  Tolerances as in test_gpu_layer.py and,
for the sums that stop every 8,192 elements (512 steps of 2u of the running
magnitude, the pieces and parts added in fp32), as in test_gpu_layer_use.py.
"""
import math

import pytest
import torch

U, BF = 2.0 ** -24, 2.0 ** -8

# (rows, channels, results): what the forward's product takes
FORWARD = {
    (40000, 512, 2048): ("wide", 0, 0),            # whole tiles in rounds
    (4096, 256, 5000): ("wide", 0, 0),             # ragged columns
    (2048, 4096, 12288): ("wide", 380, 4),         # whole rounds, and 4 tiles split over K
    (819, 3272, 5344): ("wide", 76, 8),            # the same, ragged both ways
    (5000, 8192, 1024): ("wide", 76, 4),
    (4922, 8016, 200): ("wide", 0, 20),            # every tile split
    (130, 9000, 256): ("narrow", 0, 0),            # a tile's K over pairs
    (700, 1000, 3000): ("narrow", 0, 0),
    (33, 1000, 3000): ("few", 0, 0),
}
# what the backward's take: (dz, dx, dw), each (form, whole tiles beside split ones, split tiles, pieces)
BACKWARD = {
    (4096, 2048, 2048): (("wide", 0, 0, 1), ("wide", 0, 0, 1), ("wide", 0, 0, 1)),
    (40000, 512, 2048): (("wide", 0, 0, 1), ("wide", 0, 0, 1), ("wide", 0, 16, 2)),
    (819, 3272, 5344): (("wide", 0, 0, 1), ("wide", 0, 0, 1), ("wide", 0, 0, 1)),
    (2048, 4096, 12288): (("wide", 0, 0, 1), ("wide", 0, 0, 2), ("wide", 0, 0, 1)),
    (16384, 2048, 2560): (("wide", 0, 0, 1), ("wide", 0, 0, 1), ("wide", 76, 4, 2)),
    (2500, 2056, 20000): (("wide", 0, 0, 1), ("wide", 76, 14, 3), ("wide", 0, 0, 1)),
    (1208, 8192, 1024): (("narrow", 0, 0, 1), ("together", 0, 0, 1), ("together", 0, 0, 1)),
    (300, 520, 1032): (("narrow", 0, 0, 1), ("together", 0, 0, 1), ("together", 0, 0, 1)),
}


def _whole(p):
    return p["tiles"] - p["split_tiles"] if p["split_tiles"] else 0


@pytest.mark.parametrize("size", FORWARD)
def test_forward_plans(lib, size):
    from prefix_tree_packed_dfs_gb300 import ops
    p = ops.linear_plan(*size)["y"]
    assert (p["form"], _whole(p), p["split_tiles"]) == FORWARD[size], p
    assert (p["splits"] > 1) == (p["split_tiles"] > 0)
    need = lib.tpk_linear_workspace_bytes(*size, 0, 0)
    assert need == (p["split_tiles"] * p["splits"] * 256 * 256 * 4 + 1023) // 1024 * 1024


@pytest.mark.parametrize("size", BACKWARD)
def test_backward_plans(lib, size):
    from prefix_tree_packed_dfs_gb300 import ops
    p = ops.linear_plan(*size, act="gelu", backward=True)
    assert list(p) == ["dz", "dx", "dw"]
    got = tuple((q["form"], _whole(q), q["split_tiles"], q["pieces"]) for q in p.values())
    assert got == BACKWARD[size], p
    assert list(ops.linear_plan(*size, backward=True)) == ["dx", "dw"]


def test_every_form_is_among_the_sizes():
    wide = {(bool(w), bool(s)) for f, w, s in FORWARD.values() if f == "wide"}
    assert wide == {(False, False), (True, True), (False, True)}
    assert {f for f, _, _ in FORWARD.values()} == {"few", "wide", "narrow"}
    dz, dx, dw = zip(*BACKWARD.values())
    assert {"wide", "narrow"} == {p[0] for p in dz}
    for product in (dx, dw):
        assert {"wide", "together"} <= {p[0] for p in product}
        assert any(p[1] and p[2] for p in product) and any(p[3] > 1 for p in product)
        assert any(p[0] == "wide" and p[3] == 1 and not p[2] for p in product)


def test_plans_refuse_what_the_calls_refuse(lib):
    from prefix_tree_packed_dfs_gb300 import binding as B, ops
    out = (B.ProductPlan * 3)()
    assert lib.tpk_linear_plan(0, 64, 64, 0, 0, out) == 0
    assert lib.tpk_linear_plan(70, 60, 64, 0, 0, out) == -1 and lib.tpk_linear_plan(70, 64, 64, 4, 0, out) == -1
    assert lib.tpk_linear_plan(70, 64, 64, 0, 0, None) == -1
    assert lib.tpk_linear_plan(70, 32776, 64, 0, 0, out) == -4
    assert lib.tpk_linear_plan((1 << 31) - 8200, 64, 1 << 20, 0, 0, out) == -3
    with pytest.raises(B.TpkError):
        ops.linear_plan(70, 60, 64)


def test_split_forward_refuses_without_its_workspace(lib):
    """A size whose tiles are split over K needs its workspace, all of it (before any launch)."""
    import ctypes
    P = ctypes.c_void_p
    for n, c, o in ((2048, 4096, 12288), (819, 3272, 5344), (4922, 8016, 200)):
        need = lib.tpk_linear_workspace_bytes(n, c, o, 0, 0)
        assert need > 0

        def call(ws, ws_bytes):
            return lib.tpk_linear(P(256), c, P(512), None, 0, None, 0, P(1024), o, n, c, o, ws, ws_bytes, None, None)
        assert call(None, 0) == -7 and call(None, need) == -7
        assert call(P(4096), need - 1) == -7 and call(P(4100), need) == -7


def test_dz_is_planned_without_the_split_that_it_does_not_have(lib):
    """Where the forward's best is wide tiles split over K, dz takes the best of what it can do: here narrow
    tiles, not wide ones on half as many pairs or in one more round."""
    from prefix_tree_packed_dfs_gb300 import ops
    for n, c, o in ((1208, 8192, 1024), (4922, 8016, 200), (2564, 5680, 1624), (78, 8152, 5248)):
        assert ops.linear_plan(n, c, o)["y"]["splits"] > 1
        dz = ops.linear_plan(n, c, o, act="silu", backward=True)["dz"]
        assert dz["form"] == "narrow" and dz["splits"] == 1, dz
    # where wide tiles are best without a split they stay
    assert ops.linear_plan(819, 3272, 5344, act="silu", backward=True)["dz"]["form"] == "wide"


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


def _rnd(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def _near(got, ref, tol, what):
    err = (got.double() - ref).abs()
    assert torch.isfinite(err).all(), what
    assert (err <= tol).all(), "%s: off by %.3g" % (what, float((err - tol).max()))


def _act(z, name):
    """(act(z), act'(z)) in fp64."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s * (1 + z * (1 - s))
    if name == "gelu":
        phi = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * phi, phi + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def _scores(x, w, b):
    """z and how far a sum that never stops may be off it."""
    z, mag = x @ w.T + b, x.abs() @ w.abs().T + b.abs()
    return z, (x.shape[1] + 2) * 2.0 ** -23 * mag


@pytest.mark.gpu
@pytest.mark.parametrize("size", FORWARD)
@pytest.mark.parametrize("act,res", [("none", True), ("silu", True), ("gelu", False), ("gelu_tanh", True)])
def test_linear_in_every_form(ops, size, act, res):
    n, c, o = size
    x, w, b = _rnd(1, n, c + 8)[:, 8:], _rnd(2, o, c, std=c ** -0.5), _rnd(3, o, std=0.5, dtype=torch.float32)
    r = _rnd(4, n, 2 * o, std=2.0)[:, o:] if res else None
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = ops.B.load().tpk_linear_workspace_bytes(n, c, o, 0, 0)
    room = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    y = ops.linear(x, w, bias=b, act=act, residual=r, dev_err=err, workspace=room[:need] if need else None)
    assert int(err) == 0 and (room[need:] == 0xFF).all()
    z, e_z = _scores(x.double(), w.double(), b.double())
    ref = _act(z, act)[0]
    if res:
        ref = ref + r.double()
    tol = BF * ref.abs() + 1.13 * e_z + 2 * U * z.abs()
    if act != "none":
        tol += 2.0 ** -20 * (z.abs() + 1)
    if res:
        tol += 2 * U * r.double().abs()
    _near(y, ref, tol, "y")
    if res:   # in place on the residual, whose other columns stay
        left = r._base[:, :o].clone()
        ops.linear(x, w, bias=b, act=act, residual=r, out=r)
        assert torch.equal(r, y) and torch.equal(r._base[:, :o], left)


@pytest.mark.gpu
@pytest.mark.parametrize("size", BACKWARD)
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
def test_linear_bwd_in_every_form(ops, size, act):
    n, c, o = size
    x, w, b = _rnd(1, n, c + 8)[:, :c], _rnd(2, o, c, std=c ** -0.5), _rnd(3, o, std=0.5, dtype=torch.float32)
    dy = _rnd(5, n, 2 * o)[:, o:]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = ops.B.load().tpk_linear_workspace_bytes(n, c, o, ops.ACTIVATIONS[act], 1)
    room = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    dx, dw, db = ops.linear_bwd(x, w, dy, bias=b, act=act, dev_err=err, workspace=room[:need])
    assert int(err) == 0 and (room[need:] == 0xFF).all()
    X, W, D = x.double(), w.double(), dy.double()
    dz, e_d = D, torch.zeros((), dtype=torch.float64, device="cuda")
    if act != "none":
        z, e_z = _scores(X, W, b.double())
        dz = D * _act(z, act)[1]
        e_d = D.abs() * (1.2 * e_z + 2.0 ** -19)
    e_p = e_d if act == "none" else e_d + BF * dz.abs()
    e_p = e_p.expand_as(dz)
    stop = lambda k: (min(k, 8192) / 16 + k / 8192 + 80) * 2.0 ** -23
    ref = dz @ W
    _near(dx, ref, BF * ref.abs() + e_p @ W.abs() + stop(o) * (dz.abs() @ W.abs()), "dx")
    ref = dz.T @ X
    _near(dw, ref, BF * ref.abs() + e_p.T @ X.abs() + stop(n) * (dz.abs().T @ X.abs()), "dw")
    _near(db, dz.sum(0), e_d.expand_as(dz).sum(0) + (n + 2) * U * dz.abs().sum(0), "db")
    again = ops.linear_bwd(x, w, dy, bias=b, act=act)
    assert all(torch.equal(p, q) for p, q in zip((dx, dw, db), again))


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [False, True])
def test_long_sums_of_one_sign_stop_often_enough(ops, spread):
    """The tensor core's truncation is a bias of up to 2^-23 of the running sum per 16 elements: a sum of 262,144 terms
    of one sign that never stopped would come out some 3e-4 low.  One that stops every 8,192 is at most 512 steps low,
    6.1e-5.  76 whole tiles in 32 pieces and 4 tiles split over K.

    The mean error of half a million results shows it, if their bf16 roundings average out.  spread: the rows of dy and
    the columns of x carry factors from 1 to 2, so that the results lie evenly over the bf16 steps (1.1e-3 of a value
    each, 2e-6 in the mean; 1e-5 is allowed).  Without the factors they do not: the results are 443,000 within some 700,
    closer together than one step of 2,048, and are all rounded by the same up to half a step, 2^-9 of the least value
    of their binade; then no more than that can be asked."""
    n, c, o = 262144, 2048, 2560
    p = ops.linear_plan(n, c, o, backward=True)["dw"]
    assert _whole(p) == 76 and p["split_tiles"] == 4 and p["pieces"] == 32, p
    x, dy = _rnd(1, n, c).abs_() + 0.5, _rnd(2, n, o).abs_() + 0.5
    if spread:
        g = torch.Generator(device="cuda").manual_seed(4)
        x *= torch.exp2(torch.rand(c, generator=g, device="cuda")).bfloat16()
        dy *= torch.exp2(torch.rand(o, generator=g, device="cuda")).bfloat16()
    dw = ops.linear_bwd(x, _rnd(3, o, c), dy)[1]
    for rows in (slice(0, 256), slice(2304, 2560)):
        ref = sum(p.double().T @ q.double() for p, q in zip(dy[:, rows].split(32768), x.split(32768)))
        off = float(((dw[rows].double() - ref) / ref).mean())
        assert abs(off) <= 512 * 2.0 ** -23 + (1e-5 if spread else 2.0 ** -9), off
