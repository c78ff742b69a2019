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
