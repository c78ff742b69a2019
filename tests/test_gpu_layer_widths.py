"""The widest rows that the projections and the feed-forward block take, with few
rows and with more, against fp64; tolerances as in test_layer_plans.py."""
import pytest
import torch

from test_layer_plans import BF, U, _act, _near, _rnd, _scores

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    assert torch.cuda.is_available()
    from prefix_tree_packed_dfs_gb300 import ops as o
    return o


@pytest.mark.parametrize("n", [1, 5, 70])
@pytest.mark.parametrize("c,o", [(8, 1 << 20), (32768, 8), (32768, 1032)])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_at_its_widest(ops, n, c, o, act):
    x, w, b = _rnd(1, n, c), _rnd(2, o, c, std=c ** -0.5), _rnd(3, o, std=0.5, dtype=torch.float32)
    r, dy = _rnd(4, n, o), _rnd(5, n, o)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = ops.linear(x, w, bias=b, act=act, residual=r, dev_err=err)
    dx, dw, db = ops.linear_bwd(x, w, dy, bias=b, act=act, dev_err=err)
    assert int(err) == 0
    X, W, D = x.double(), w.double(), dy.double()
    z, e_z = _scores(X, W, b.double())
    v, slope = _act(z, act)
    soft = 0.0 if act == "none" else 1.0
    ref = v + r.double()
    _near(y, ref, BF * ref.abs() + 1.13 * e_z + 2 * U * (z.abs() + r.double().abs()) + soft * 2.0 ** -20 * (z.abs() + 1), "y")
    dz = D * slope
    e_d = soft * D.abs() * (1.2 * e_z + 2.0 ** -19)
    e_p = e_d + soft * BF * dz.abs()
    stop = lambda k: (min(k, 8192) / 16 + k / 8192 + 80) * 2.0 ** -23
    ref = dz @ W
    _near(dx, ref, BF * ref.abs() + e_p @ W.abs() + stop(o) * (dz.abs() @ W.abs()), "dx")
    ref = dz.T @ X
    _near(dw, ref, BF * ref.abs() + e_p.T @ X.abs() + stop(n) * (dz.abs().T @ X.abs()), "dw")
    _near(db, dz.sum(0), e_d.sum(0) + (n + 2) * U * dz.abs().sum(0), "db")


@pytest.mark.parametrize("n", [1, 40, 70])
@pytest.mark.parametrize("c,i,o", [(64, 32768, 64), (32768, 64, 32768)])
def test_ffn_at_its_widest(ops, n, c, i, o):
    """2-norms: a, dg, du and the results in bf16, each b / sqrt 3 of the root mean square at most."""
    x, w_in, w_out = _rnd(1, n, c), _rnd(2, 2 * i, c, std=c ** -0.5), _rnd(3, o, i, std=i ** -0.5)
    r, dy = _rnd(4, n, o), _rnd(5, n, o)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    y, pre, a = ops.gated_ffn(x, w_in, w_out, residual=r, save=True, dev_err=err)
    y1 = ops.gated_ffn(x, w_in, w_out, residual=r, dev_err=err)
    got = ops.gated_ffn_bwd(x, w_in, w_out, dy, pre, a, dev_err=err)
    assert int(err) == 0
    leaf = [t.double().requires_grad_() for t in (x, w_in, w_out)]
    gu = leaf[0] @ leaf[1].T
    ref = (torch.nn.functional.silu(gu[:, :i]) * gu[:, i:]) @ leaf[2].T + r.double()
    want = torch.autograd.grad(ref, leaf, dy.double())
    for p, q, name in zip((y, y1) + got, (ref.detach(), ref.detach()) + want, ("y", "y alone", "dx", "dw_in", "dw_out")):
        rel = float((p.double() - q).norm() / q.norm())
        assert rel <= 3 * BF / 3 ** 0.5, (name, rel)
